"""GPU: how many bits the activation of the experts' layer keeps between its two products.

Each row of D takes the difference of two activations that agree in their first bits, so
that what the second product's operands leave out is all that is seen.

x = (1, 2^-12, 0 ...), G[i] = (1.5, 0 ...), U[i] = (1, t[i], 0 ...) with whole t[i] from 1 to 8, so g = 1.5
and u[i] = 1 + t[i] 2^-12 exactly, and with s = silu(1.5)
    a[i] = p s u[i],  y[r] = a[2 r] - a[2 r + 1] = p s (t[2 r] - t[2 r + 1]) 2^-12.
Bounds, u = 2^-24: s is the same number for all i, some 4 u of itself off; the two products by u[i] and
p round each a[i] by u each, so their difference is off by 4 u a + 4 u |y|; operands of h leave
2 h a; the sums of the second product have at most six terms that are not 0, each the size of a
at the most and cut off at 2^-23 of that.  a < 1.25 p.  Then the output's half step."""
import pytest
import torch

import hyper_connection_residual_mixes_gb300 as hcg
from hyper_connection_residual_mixes_gb300 import _lib
from hyper_connection_residual_mixes_gb300 import build as hc_build

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
T = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hc_build.build()
    _lib.load()


@pytest.mark.parametrize("x,w,h", [("bf16", "ue8m0", 2.0 ** -22), ("bf16", "fp32", 2.0 ** -22), ("bf16", "same", 0.0),
                                   ("fp16", "ue8m0", 2.0 ** -22), ("fp16", "same", 2.0 ** -22)])
@pytest.mark.parametrize("tokens", [1, 8, 33])
def test_differences_of_activations(x, w, h, tokens):
    d, inner = 16, 32
    g = torch.Generator(device="cuda").manual_seed(tokens)
    t = torch.randint(1, 9, (inner,), generator=g, device="cuda").float()
    up, down = torch.zeros((1, 2, inner, d), device="cuda"), torch.zeros((1, d, inner), device="cuda")
    up[0, 0, :, 0], up[0, 1, :, 0], up[0, 1, :, 1] = 1.5, 1.0, t
    r = torch.arange(d, device="cuda")
    down[0, r, 2 * r], down[0, r, 2 * r + 1] = 1.0, -1.0
    kw = {}
    if w == "same":
        up, down = up.to(T[x]), down.to(T[x])
    else:
        up, down = (v.to(torch.float8_e4m3fn).view(torch.uint8) for v in (up, down))
        one = lambda *s: torch.ones(s, device="cuda") if w == "fp32" else torch.full(s, 127, dtype=torch.uint8, device="cuda")
        kw = {"up_scales": one(1, 2, 1, 1), "down_scales": one(1, 1, 1)}
    rows = torch.zeros((tokens, d), device="cuda")
    rows[:, 0], rows[:, 1] = 1.0, 2.0 ** -12
    p = 0.25 + torch.rand((tokens, 1), generator=g, device="cuda")
    y = hcg.hc_moe_tokens(rows.to(T[x]), up, down, torch.zeros((tokens, 1), dtype=torch.int32, device="cuda"), p, **kw)
    ps = p.double() * 1.5 / (1 + torch.exp(torch.tensor(-1.5, dtype=torch.float64, device="cuda")))
    want = ps * ((t[0::2] - t[1::2]).double() * 2.0 ** -12)
    room = 1.25 * p.double() * (4 * U + 2 * h + 6 * 2.0 ** -23) + 4 * U * want.abs()
    half = torch.finfo(T[x]).eps / 2
    tiny = torch.finfo(T[x]).smallest_normal * half
    bad = (y.double() - want).abs() > half * (want.abs() + room) + room + tiny
    assert not bad.any(), (int(bad.sum()), (y.double() - want).abs().max().item())
