"""GPU: the experts' layer of 8-bit weights with scales far from 1.

Tokens and activations go into its products with a power of two taken out, which is put back together with the
scales; neither may leave fp32's range on the way where the result does not."""
import pytest
import torch

import hyper_connection_residual_mixes_gb300 as hcg
from hyper_connection_residual_mixes_gb300 import _lib
from hyper_connection_residual_mixes_gb300 import build as hc_build
from tests import test_gpu_fp8_mm as mm
from tests.test_gpu_fp8_scales import _gen, _near

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hc_build.build()
    _lib.load()


@pytest.mark.parametrize("x", ["bf16", "fp16"])
@pytest.mark.parametrize("tokens", [1, 9, 40])
def test_experts(x, tokens):
    """The experts' layer: scales of G, U and D far from 1 whose products bring the activation and the
    output back.  With x = v 2^e, v from 1 to 2 and codes of one sign, all sums are of one sign, so that
    the relative errors of sums of n terms, (n + 40) 2^-23 of them as in the operator's own tests, go through:
    silu's slope times g / silu(g) is at most 1 + |g| for g > 0."""
    e = -100 if x == "bf16" else 0
    d, inner, k = 272, 144, 2
    g = _gen(tokens)
    rows = ((1 + torch.rand((tokens, d), generator=g, device="cuda")) * 2.0 ** e).to(T[x])
    code = lambda *s: (128 + 64 * torch.rand(s, generator=g, device="cuda")).to(torch.float8_e4m3fn).view(torch.uint8)
    up, down = code(3, 2, inner, d), code(3, d, inner)
    bi, bd = mm._blocks(inner), mm._blocks(d)
    us, ds = torch.empty((3, 2, bi, bd), device="cuda"), torch.empty((3, bd, bi), device="cuda")
    us[:, 0] = _near((3, bi, bd), -e - 17, "fp32", g)             # g of about 2
    us[:, 1] = _near((3, bi, bd), -132 if e == 0 else -34, "fp32", g)  # u of about 2^-116
    ds[:] = _near((3, bd, bi), 101, "fp32", g)                    # y of about 1
    ids = torch.stack([torch.randperm(3, generator=g, device="cuda")[:k] for _ in range(tokens)]).int()
    p = 0.5 + torch.rand((tokens, k), generator=g, device="cuda")
    y = hcg.hc_moe_tokens(rows, up, down, ids, p, up_scales=us, down_scales=ds)
    xd, want, room = rows.double(), torch.zeros((tokens, d), dtype=torch.float64, device="cuda"), torch.zeros((tokens, d), dtype=torch.float64, device="cuda")
    for i in range(3):
        t, j = (ids == i).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        G, V, D = mm._matrix(up[i, 0], us[i, 0]), mm._matrix(up[i, 1], us[i, 1]), mm._matrix(down[i], ds[i])
        gate, u = xd[t] @ G.t(), xd[t] @ V.t()
        a = p[t, j].double()[:, None] * gate / (1 + torch.exp(-gate)) * u
        off = ((d + 40) * 2.0 ** -23 * (2 + gate) + 8 * 2.0 ** -24 + 2.0 ** -22) * a
        want.index_add_(0, t, a @ D.t())
        room.index_add_(0, t, (off + (k * inner + 40) * 2.0 ** -23 * a) @ D.t())
    assert y.isfinite().all() and (want > 2.0 ** -8).all() and (want < 2.0 ** 12).all()
    half = torch.finfo(T[x]).eps / 2
    bad = (y.double() - want).abs() > half * (want + room) + room
    assert not bad.any(), (int(bad.sum()), ((y.double() - want).abs() / want).max().item())
    # rows of D that are 0 give 0, also of activations of 2^40 and 2^60 with scales of 2^100
    down[:, ::2], ds[:] = 0, 2.0 ** 100
    us[:, 1] = us[:, 0] * (2.0 ** 60 if e == 0 else 2.0 ** 40)
    y = hcg.hc_moe_tokens(rows, up, down, ids, p, up_scales=us, down_scales=ds)
    assert (y[:, ::2] == 0).all() and (y[:, 1::2] == float("inf")).all()
