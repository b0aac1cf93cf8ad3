"""GPU: the operators of sublayers in 8 bits together, as decoding and training use them.

Decoding: a chain launch collapses the streams, hc_rms_norm norms its h in bf16 and in
8 bits, a projection takes the codes, the experts' layer the bf16 rows, the sum of
both goes back into the streams; the next norm adds a residual.  Training: norm, cast,
product and their backward, the weights' gradient from hc_grouped_mm_weights, and one
AdamW step.  Every stage is held to its formula in 64 bits on the inputs it had, with
the bounds of the operators' own tests; captured into a graph the steps give the eager
ones' bits, also on two streams at once."""
import pytest
import torch

import hyper_connection_residual_mixes_gb300 as hcg
from hyper_connection_residual_mixes_gb300 import _lib, inputs
from hyper_connection_residual_mixes_gb300 import build as hc_build
from tests import test_gpu_fp8_mm as mm
from tests import test_gpu_moe_tokens as moe
from tests import test_gpu_rms_norm as norm

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
D, E, INNER, K = 1024, 8, 256, 2
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hc_build.build()
    _lib.load()


class Decode:
    """A side of a block whose sublayer is a projection beside experts, for n tokens."""

    def __init__(self, n, seed=0):
        g = torch.Generator(device=DEV).manual_seed(20 + seed)
        r = lambda *s: torch.randn(s, generator=g, device=DEV)
        self.x, self.pre_mix = inputs.streams(g, n, 4, D, device=DEV), inputs.pre_mix(g, n, device=DEV)
        self.hc_fn, self.hc_scale, self.hc_base, self.norm_w = inputs.side_params(g, d=D, device=DEV).astuple()
        self.w, self.w_scales = hcg.hc_fp8_cast_weights(r(D, D).mul_(D ** -0.5))
        self.up, self.up_scales = hcg.hc_fp8_cast_weights(r(E, 2, INNER, D).mul_(D ** -0.5).bfloat16())
        self.down, self.down_scales = hcg.hc_fp8_cast_weights(r(E, D, INNER).mul_(INNER ** -0.5).bfloat16())
        self.gate, self.next_w = r(E, D).mul_(D ** -0.5), 0.5 + r(D).abs()

    def step(self):
        o = {"h": torch.empty(self.x.shape[0], D, dtype=torch.bfloat16, device=DEV)}
        state = hcg.hc_chain_begin(self.x, self.pre_mix, self.hc_fn, self.hc_scale, self.hc_base, h_pre_out=o["h"])
        o["h_norm"] = hcg.hc_chain_norm(o["h"], state, self.norm_w)
        o.update({"n_" + k: v for k, v in hcg.hc_rms_norm(o["h"], self.norm_w, norm_eps=1e-20, out="both", return_rstd=True).items()})
        o["p"] = hcg.hc_fp8_mm(o["n_codes"], o["n_scales"], self.w, self.w_scales)
        o["logits"] = o["n_y"].float() @ self.gate.t()
        o["e"], o["ids"], o["weights"] = hcg.hc_moe_tokens(o["n_y"], self.up, self.down, logits=o["logits"], top_k=K, score="sigmoid",
                                                           up_scales=self.up_scales, down_scales=self.down_scales)
        o["y"] = hcg.hc_chain_side(self.x, o["p"] + o["e"], state, self.norm_w)[1]
        o.update({"m_" + k: v for k, v in hcg.hc_rms_norm(o["e"], self.next_w, o["p"], out="fp8", return_rstd=True).items()})
        return o


@pytest.mark.parametrize("n", [1, 7, 16, 40])
def test_decode_stages(n):
    s = Decode(n)
    o = s.step()
    # the norm of the chain's h is the chain's own, but for the last place (its statistic comes
    # from sums in another order)
    ulp = torch.finfo(torch.bfloat16).eps
    assert ((o["n_y"].float() - o["h_norm"].float()).abs() <= ulp * o["h_norm"].float().abs()).all()
    f = o["h"].double()
    rstd = 1 / torch.sqrt(f.square().mean(1, keepdim=True) + 1e-20)
    y = f * rstd * s.norm_w.double()
    assert ((o["n_rstd"].double() - rstd[:, 0]).abs() <= 64 * U * rstd[:, 0]).all()
    norm._check_codes(y, o["n_codes"], o["n_scales"], 100 * U)
    mm._check(o["p"], o["n_codes"], o["n_scales"], s.w, s.w_scales, False)
    ids, weights = moe._choose_ref(o["logits"].cpu(), K, "sigmoid", True, 1.0)
    assert torch.equal(o["ids"].cpu(), ids) and ((o["weights"].cpu().double() - weights).abs() <= 112 * U * weights).all()
    w = {"up": s.up, "down": s.down, "up_scales": s.up_scales, "down_scales": s.down_scales}
    moe._check(o["e"], o["n_y"], w, o["ids"], o["weights"])
    v, rstd, y = norm._ref(o["e"], s.next_w, o["p"], 1e-6)
    assert torch.equal(o["m_r"], v) and set(o) >= {"m_codes", "m_scales", "m_rstd"} and "m_y" not in o
    norm._check_codes(y, o["m_codes"], o["m_scales"], 100 * U)


@pytest.mark.parametrize("n", [1, 16, 40])
def test_decode_graph(n):
    """The whole step captured once and replayed on other tokens, bit for bit."""
    s, other = Decode(n), Decode(n, seed=1)
    s.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = s.step()
    for source in (s.x.clone(), other.x):
        s.x.copy_(source)
        graph.replay()
        for name, t in s.step().items():
            assert torch.equal(out[name], t), name
    assert _lib.raw("hc_consume_device_error", None) == 0


def test_decode_two_streams():
    """Two steps at once on two streams (all but the chain's launches, which want the SMs to
    themselves) give what they give alone."""
    pair = [Decode(16, seed=k) for k in (2, 3)]
    want = [p.step() for p in pair]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pair]
    got = [[], []]
    for _ in range(5):
        for k, (p, s, o) in enumerate(zip(pair, streams, want)):
            with torch.cuda.stream(s):
                n = hcg.hc_rms_norm(o["h"], p.norm_w, norm_eps=1e-20, out="both")
                y = hcg.hc_fp8_mm(n["codes"], n["scales"], p.w, p.w_scales)
                e = hcg.hc_moe_tokens(n["y"], p.up, p.down, logits=o["logits"], top_k=K, score="sigmoid", up_scales=p.up_scales,
                                      down_scales=p.down_scales)[0]
                got[k].append((n["y"], n["codes"], y, e))
    torch.cuda.synchronize()
    for k in (0, 1):
        for y, codes, p, e in got[k]:
            assert torch.equal(y, want[k]["n_y"]) and torch.equal(codes, want[k]["n_codes"])
            assert torch.equal(p, want[k]["p"]) and torch.equal(e, want[k]["e"])


class Train:
    """norm with residual -> cast -> y = h w^T, the loss sum(c y) + sum(past r), and a step of w and norm_w."""

    def __init__(self, n, d, N):
        g = torch.Generator(device=DEV).manual_seed(n)
        r = lambda *s: torch.randn(s, generator=g, device=DEV)
        self.x, self.res, self.c, self.past = r(n, d).bfloat16(), r(n, d).bfloat16(), r(n, N).bfloat16(), r(n, d)
        self.norm_w, self.w = 0.5 + r(d).abs(), r(N, d) * d ** -0.5
        self.grads = [torch.zeros_like(self.norm_w), torch.zeros_like(self.w)]
        m, v = zip(*[hcg.adamw_state(t) for t in (self.norm_w, self.w)])
        self.plan = hcg.adamw_plan([self.norm_w, self.w], self.grads, m, v)
        self.offsets = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        self.t = torch.zeros((1,), dtype=torch.int64, device=DEV)

    def step(self):
        o = dict(zip(("w", "w_scales"), hcg.hc_fp8_cast_weights(self.w)))
        o.update(hcg.hc_rms_norm(self.x, self.norm_w, self.res, out="both", return_rstd=True))
        o["p"] = hcg.hc_fp8_mm(o["codes"], o["scales"], o["w"], o["w_scales"], out_dtype=torch.float32)
        o["c"], o["c_scales"] = hcg.hc_fp8_cast(self.c)
        o["g_h"] = hcg.hc_fp8_mm(o["c"], o["c_scales"], o["w"], o["w_scales"], transposed=True, out_dtype=torch.float32)
        o["g_w"] = hcg.hc_grouped_mm_weights(self.c, o["y"], self.offsets, out_dtype=torch.float32)
        back = hcg.hc_rms_norm_backward(o["g_h"], o["r"], self.norm_w, o["rstd"], g_r=self.past)
        o["g_x"], o["g_norm_w"] = back["g_x"], back["g_norm_w"]
        o["norm_w"] = self.norm_w.clone()
        self.grads[0].copy_(o["g_norm_w"]), self.grads[1].copy_(o["g_w"][0])
        self.t.add_(1)
        hcg.hc_adamw_step(self.plan, lr=1e-3, step=self.t)
        o["after"] = self.w.clone()
        return o


@pytest.mark.parametrize("n,d,N", [(3, 272, 144), (300, 1024, 528), (2100, 1040, 1296)])
def test_training_stages(n, d, N):
    s = Train(n, d, N)
    before = s.w.clone()
    o = s.step()
    mm._check(o["p"], o["codes"], o["scales"], o["w"], o["w_scales"], False)
    mm._check(o["g_h"], o["c"], o["c_scales"], o["w"], o["w_scales"], True)
    norm._check_backward(o["g_h"], o["r"], o["norm_w"], o["rstd"], s.past, o)
    want, size = s.c.double().t() @ o["y"].double(), s.c.double().abs().t() @ o["y"].double().abs()
    assert ((o["g_w"][0].double() - want).abs() <= (n + 16) * 2.0 ** -23 * size).all()
    assert not torch.equal(before, o["after"]) and o["after"].isfinite().all()


def test_training_gradient_through_the_cast():
    """The gradient of x through norm, cast and product, the casts passing it through: against
    central differences of the 64-bit loss with w as the codes have it.  What the gradient's own
    cast takes from it: each value of c is off by at most 2^-4 of itself."""
    s = Train(6, 256, 144)
    o = s.step()
    w = mm._matrix(o["w"], o["w_scales"])
    c = mm._rows(o["c"], o["c_scales"])
    assert ((c - s.c.double()).abs() <= 2.0 ** -4 * s.c.double().abs() + 2.0 ** -10 * c.abs().amax()).all()

    def loss(r):
        h = r / torch.sqrt(r.square().mean(1, keepdim=True) + 1e-6) * o["norm_w"].double()
        return ((h @ w.t()) * c).sum() + (r * s.past.double()).sum()
    r, dr, h = o["r"].double(), torch.randn((6, 256), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).double(), 1e-4
    num = (loss(r + h * dr) - loss(r - h * dr)) / (2 * h)
    assert abs(num - (o["g_x"].double() * dr).sum()) <= 1e-5 * (o["g_x"].double() * dr).abs().sum()


def test_training_graph():
    """The step captured beside an eager one's tensors, three times replayed, gives three eager steps."""
    eager, s = Train(300, 1024, 528), Train(300, 1024, 528)
    s.step(), eager.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = s.step()
    for _ in range(3):
        graph.replay()
        o = eager.step()
    for name, t in o.items():
        assert torch.equal(out[name], t), name
    assert torch.equal(s.w, eager.w) and torch.equal(s.norm_w, eager.norm_w)


def test_first_call_in_a_capture():
    """The first call of a process, and each kernel's, may be the captured one: nothing that a
    capture forbids is done then."""
    import os
    import subprocess
    import sys
    code = """
import torch, hyper_connection_residual_mixes_gb300 as hcg
x = torch.randn(2000, 1024, device="cuda").bfloat16(); w = torch.ones(1024, device="cuda")
q = torch.full((1024, 1024), 0x38, dtype=torch.uint8, device="cuda"); s = torch.full((8, 8), 127, dtype=torch.uint8, device="cuda")
up = torch.zeros(4, 2, 64, 1024, device="cuda").bfloat16(); down = torch.zeros(4, 1024, 64, device="cuda").bfloat16()
lg = torch.randn(3, 4, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    n = hcg.hc_rms_norm(x, w, x, out="both", return_rstd=True)
    b = hcg.hc_rms_norm_backward(x, n["r"], w, n["rstd"])
    y = hcg.hc_fp8_mm(n["codes"], n["scales"], q, s)
    z = hcg.hc_fp8_mm(n["codes"][:4], n["scales"][:4], q, s)
    t = hcg.hc_fp8_mm(*hcg.hc_fp8_cast(y), q, s, transposed=True)
    c = hcg.hc_fp8_cast_weights(x)
    m = hcg.hc_moe_tokens(x[:3], up, down, logits=lg, top_k=2)
g.replay()
torch.cuda.synchronize()
assert torch.equal(z, hcg.hc_fp8_mm(n["codes"][:4], n["scales"][:4], q, s)) and torch.equal(y, hcg.hc_fp8_mm(n["codes"], n["scales"], q, s))
print("fine")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]
