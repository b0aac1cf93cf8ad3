"""GPU: the sublayer operators together, as a training step uses them.

One side of a block whose sublayer is a layer norm in front of two grouped
products: the chain's launch collapses the streams, hc_layer_norm norms them,
the rows go to their experts and back, the last chain launch writes the
streams; then the side's backward, both products' and the norm's, and one
AdamW step over everything that learns.  Every stage is held to its formula in
64 bits on the inputs it had, with the bounds of the operators' own tests; and
the whole step, captured into one graph, gives the eager step's bits."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
import hyper_connection_residual_mixes_gb300 as hcg
from hyper_connection_residual_mixes_gb300 import _lib, inputs
from hyper_connection_residual_mixes_gb300 import build as hc_build

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
N, D, F, E = 150, 1024, 264, 5
U = 2.0 ** -24
ADAM = dict(lr=1e-3, betas=(0.9, 0.95), weight_decay=0.1)


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hc_build.build()
    _lib.load()


class Side:
    """The step's tensors; `step` runs it once and returns what its stages gave."""

    def __init__(self, mxfp8):
        g = torch.Generator(device=DEV).manual_seed(11)
        r = lambda *s: torch.randn(s, generator=g, device=DEV)
        self.x = inputs.streams(g, N, 4, D, device=DEV)
        self.pre_mix = inputs.pre_mix(g, N, device=DEV)
        p = inputs.side_params(g, d=D, device=DEV)
        self.hc_fn, self.hc_scale, self.hc_base, self.norm_w = p.astuple()
        self.ln_w, self.ln_b = 0.5 + torch.rand((D,), generator=g, device=DEV), 0.1 * r(D)
        self.up, self.down = r(E, F, D) / D ** 0.5, r(E, D, F) / F ** 0.5   # fp32, with their bf16 copies
        self.up16, self.down16 = self.up.bfloat16(), self.down.bfloat16()
        expert = torch.randint(0, E - 1, (N,), generator=g, device=DEV)       # the last expert gets no row
        self.order = expert.argsort(stable=True)
        self.back = self.order.argsort()
        self.offsets = torch.searchsorted(expert[self.order], torch.arange(E + 1, device=DEV)).int()
        self.c = r(N, 4, D)                                                   # the loss is sum(c y)
        self.learn = [self.hc_fn, self.hc_scale, self.hc_base, self.ln_w, self.ln_b, self.up, self.down]
        self.grads = [torch.zeros_like(t) for t in self.learn]
        states = [hcg.adamw_state(t, mxfp8=mxfp8) for t in self.learn]
        self.m, self.v = [s[0] for s in states], [s[1] for s in states]
        self.plan = hcg.adamw_plan(self.learn, self.grads, self.m, self.v, [None] * 5 + [self.up16, self.down16])
        self.t = torch.zeros((1,), dtype=torch.int64, device=DEV)

    def step(self):
        o = {}
        o["h"] = torch.empty((N, D), dtype=torch.bfloat16, device=DEV)
        state = hcg.hc_chain_begin(self.x, self.pre_mix, self.hc_fn, self.hc_scale, self.hc_base, h_pre_out=o["h"])
        o["hn"], o["mean"], o["rstd"] = hcg.hc_layer_norm(o["h"], self.ln_w, self.ln_b, return_stats=True)
        o["rows"] = o["hn"][self.order]
        o["a"] = hcg.hc_grouped_mm(o["rows"], self.up16, self.offsets)
        o["s"] = torch.relu(o["a"])
        o["f_rows"] = hcg.hc_grouped_mm(o["s"], self.down16, self.offsets)
        f = o["f_rows"][self.back]
        o["y"] = hcg.hc_chain_side(self.x, f, state, self.norm_w)[1]
        side = hcg.hc_block_step_backward(self.x, self.pre_mix, f, self.hc_fn, self.hc_scale, self.hc_base, self.norm_w,
                                          torch.zeros((N, D), device=DEV), self.c)
        o["g_f"] = side["g_f"][self.order].bfloat16()
        o["g_s"] = hcg.hc_grouped_mm(o["g_f"], self.down16, self.offsets, transposed=True)
        hcg.hc_grouped_mm_weights(o["g_f"], o["s"], self.offsets, g_w=self.grads[6])
        o["g_a"] = torch.where(o["a"] > 0, o["g_s"], torch.zeros_like(o["g_s"]))
        b = hcg.hc_grouped_mm_backward(o["g_a"], o["rows"], self.up16, self.offsets, g_w=self.grads[5])
        o["g_rows"] = b["g_x"]
        o["g_hn"] = b["g_x"][self.back].float()
        n = hcg.hc_layer_norm_backward(o["g_hn"], o["h"], self.ln_w, o["mean"], o["rstd"])
        o["g_h"] = n["g_x"]
        for t, v in zip(self.grads, (side["g_hc_fn"], side["g_hc_scale"], side["g_hc_base"], n["g_norm_w"], n["g_norm_b"])):
            t.copy_(v)
        self.t.add_(1)
        hcg.hc_adamw_step(self.plan, step=self.t, **ADAM)
        return o

    def state(self):
        flat = [t for s in self.m + self.v for t in (s if isinstance(s, tuple) else (s,))]
        return self.learn + flat + [self.up16, self.down16, self.t]


def _product(got, x, w, offsets):
    o = offsets.tolist()
    for e in range(E):
        xe, we = x[o[e]:o[e + 1]].double(), w[e].double().t()
        want, room = xe @ we, (x.shape[1] / 16 + 2) * 2.0 ** -22 * (xe.abs() @ we.abs())
        assert ((got[o[e]:o[e + 1]].double() - want).abs() <= room + 2.0 ** -8 * (want.abs() + room)).all()


def test_stages_of_a_step():
    s = Side(False)
    up, down = s.up16.clone(), s.down16.clone()
    before = [t.clone() for t in s.learn]
    o = s.step()
    h, w, b = o["h"].double(), before[3].double(), before[4].double()
    xh = (h - h.mean(1, keepdim=True)) / torch.sqrt(h.var(1, correction=0, keepdim=True) + 1e-5)
    scale = h.abs().mean(1, keepdim=True) * o["rstd"].double()[:, None]
    room = 1024 * U * (w.abs() * (xh.abs() + scale) + b.abs())
    want = xh * w + b
    assert ((o["hn"].double() - want).abs() <= room + 2.0 ** -8 * (want.abs() + room)).all()
    _product(o["a"], o["rows"], up, s.offsets)
    _product(o["f_rows"], o["s"], down, s.offsets)
    _product(o["g_s"], o["g_f"], down.transpose(1, 2), s.offsets)
    _product(o["g_rows"], o["g_a"], up.transpose(1, 2), s.offsets)
    ends = s.offsets.tolist()
    for grad, g, x in ((s.grads[6], o["g_f"], o["s"]), (s.grads[5], o["g_a"], o["rows"])):
        assert (grad[E - 1] == 0).all()
        for e in range(E - 1):
            ge, xe = g[ends[e]:ends[e + 1]].double(), x[ends[e]:ends[e + 1]].double()
            k = ge.shape[0]
            assert ((grad[e].double() - ge.t() @ xe).abs() <= ((k / 16 + 2) * 2.0 ** -22 + U) * (ge.abs().t() @ xe.abs())).all()
    # the first step moves every weight with a gradient by lr, after its decay
    for p0, p1, g in zip(before, s.learn, s.grads):
        q = p0.double() * (1 - ADAM["lr"] * ADAM["weight_decay"]) - p1.double()
        gd = g.double()
        # lr and step come from the device: corrections within a few units, p rounded a few times
        assert ((q - ADAM["lr"] * gd / (gd.abs() + 1e-8)).abs() <= 64 * U * ADAM["lr"] + 8 * U * p0.double().abs()).all()
    assert torch.equal(s.up16, s.up.bfloat16()) and torch.equal(s.down16, s.down.bfloat16())
    assert _lib.raw("hc_consume_device_error", None) == 0


@pytest.mark.parametrize("mxfp8", [False, True])
def test_step_as_a_graph(mxfp8):
    """Three steps of one captured graph against three eager steps, bit for bit."""
    eager, graphed = Side(mxfp8), Side(mxfp8)
    warm = Side(mxfp8)
    warm.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.step()
    for _ in range(3):
        eager.step()
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager.state(), graphed.state()):
        assert torch.equal(a, b)
    assert int(graphed.t) == 3 and _lib.raw("hc_consume_device_error", None) == 0


def test_steps_on_two_streams():
    """Two sides' steps on two streams at once give what they give one after the other."""
    one, two, ref = Side(False), Side(True), (Side(False), Side(True))
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for side, st in zip((one, two), s):
            with torch.cuda.stream(st):
                side.step()
    torch.cuda.synchronize()
    for side in ref:
        for _ in range(3):
            side.step()
    for got, want in zip((one, two), ref):
        for a, b in zip(got.state(), want.state()):
            assert torch.equal(a, b)


_FIRST_CALLS = """
import threading, torch
import hyper_connection_residual_mixes_gb300 as hcg
torch.cuda.init()
g = torch.Generator(device="cuda").manual_seed(1)
r = lambda *s: torch.randn(s, generator=g, device="cuda")
x, w, gy = r(700, 5120).bfloat16(), r(5120), r(700, 5120)
rows, weights = r(300, 512).bfloat16(), r(4, 256, 512).bfloat16()
off = torch.tensor([0, 90, 100, 250, 300], dtype=torch.int32, device="cuda")
results, errors, go = {}, [], threading.Barrier(8)
torch.cuda.synchronize()

def work(k):
    try:
        p, s = torch.ones(5000, device="cuda"), torch.cuda.Stream()
        m, v = hcg.adamw_state(p)
        plan = hcg.adamw_plan([p], [torch.full_like(p, 0.5)], [m], [v])
        torch.cuda.synchronize()
        go.wait()
        with torch.cuda.stream(s):
            y, mean, rstd = hcg.hc_layer_norm(x, w, return_stats=True)
            n = hcg.hc_layer_norm_backward(gy, x, w, mean, rstd)
            b = hcg.hc_grouped_mm_backward(hcg.hc_grouped_mm(rows, weights, off), rows, weights, off)
            hcg.hc_adamw_step(plan, 1e-3, 1)
        s.synchronize()
        results[k] = [y, mean, rstd, *n.values(), *b.values(), p, m, v]
    except BaseException as e:
        errors.append(e)

threads = [threading.Thread(target=work, args=(k,)) for k in range(8)]
[t.start() for t in threads]
[t.join() for t in threads]
assert not errors, errors
assert all(torch.equal(a, b) for k in range(1, 8) for a, b in zip(results[0], results[k]))
assert all(t.isfinite().all() for t in results[0])
print("same")
"""


def test_first_calls_from_several_host_threads():
    """In a process of its own: eight host threads make its first calls at once."""
    out = subprocess.run([sys.executable, "-c", _FIRST_CALLS], capture_output=True, text=True, timeout=300,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert out.returncode == 0 and out.stdout.split() == ["same"], out.stdout + out.stderr


def test_gradient_of_the_streams_through_the_sublayer():
    """The sublayer reads h = sum_s pre_mix[s] x[s]; the side's backward takes no gradient
    of it, so what the layer norm's backward gives is added to the streams' and
    pre_mix's: g_x[s] += pre_mix[s] g_h, g_pre_mix[s] += <g_h, x[s]>.

    Bounds: the side's own (1e-4 of a value and of the largest), carried on through
    |W|, and half a step of each rounding to bf16 (2^-8); the norm's backward is
    linear in its gradient, its own error 1024 u and its fp32 statistics' 8 times that."""
    n, d = 37, 1024
    case = inputs.tiny(seed=3, n=n, d=d)
    x, pm, params = case.x.to(DEV), case.pre_mix.to(DEV), case.params[0].to(DEV).astuple()
    g = torch.Generator(device=DEV).manual_seed(7)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)
    ln_w, ln_b, w, c = 0.5 + torch.rand((d,), generator=g, device=DEV), 0.1 * r(d), (r(3, d, d) / d ** 0.5).bfloat16(), r(n, 4, d)
    ends = [0, 10, 10, n]
    off = torch.tensor(ends, dtype=torch.int32, device=DEV)
    h = torch.empty((n, d), dtype=torch.bfloat16, device=DEV)
    hcg.hc_chain_begin(x, pm, *params[:3], h_pre_out=h)
    hn, mean, rstd = hcg.hc_layer_norm(h, ln_w, ln_b, return_stats=True)
    f = hcg.hc_grouped_mm(hn, w, off)
    side = hcg.hc_block_step_backward(x, pm, f, *params, torch.zeros((n, d), device=DEV), c)
    g_hn = hcg.hc_grouped_mm(side["g_f"].bfloat16(), w, off, transposed=True)
    g_h = hcg.hc_layer_norm_backward(g_hn.float(), h, ln_w, mean, rstd)["g_x"]
    g_x = side["g_x"] + pm[..., None] * g_h[..., None, :]
    g_pre_mix = side["g_pre_mix"] + (x.float() * g_h[..., None, :]).sum(-1)

    D = lambda t: t.double().cpu().numpy()
    X, P, W, LW, LB, C, Q = D(x), D(pm), D(w), D(ln_w), D(ln_b), D(c), [D(t) for t in params]
    experts = [(e, slice(ends[e], ends[e + 1])) for e in range(3)]
    mean_of = lambda t: t.mean(1, keepdims=True)

    def norm_backward(H, g_n, room):
        """g_h and its bound from the gradient of the norm's output and its bound."""
        rs = 1 / np.sqrt(mean_of((H - mean_of(H)) ** 2) + 1e-5)
        xh, wg, wr = (H - mean_of(H)) * rs, g_n * LW, room * np.abs(LW)
        linear = lambda t: rs * (t + mean_of(t) + np.abs(xh) * mean_of(t * np.abs(xh)))
        return rs * (wg - mean_of(wg) - xh * mean_of(wg * xh)), linear(wr) + 8 * 1024 * U * linear(np.abs(wg) + wr)

    ref = oracle.side_backward(X, P, D(f), *Q, np.zeros((n, d)), C, rounded=True)
    side_room = lambda t: 1e-4 * np.abs(t) + 1e-4 * np.abs(t).max()
    room_f = side_room(ref["g_f"])
    room_f = room_f + 2.0 ** -8 * (np.abs(ref["g_f"]) + room_f)
    g_n, room_n = np.zeros((n, d)), np.zeros((n, d))
    for e, rows in experts:
        g_n[rows] = ref["g_f"][rows] @ W[e]
        room_n[rows] = room_f[rows] @ np.abs(W[e]) + (d / 16 + 2) * 2.0 ** -22 * ((np.abs(ref["g_f"]) + room_f)[rows] @ np.abs(W[e]))
    room_n = room_n + 2.0 ** -8 * (np.abs(g_n) + room_n)
    want_h, room_h = norm_backward(D(h), g_n, room_n)
    assert (np.abs(D(g_h) - want_h) <= room_h).all()
    want_x, room_x = ref["g_x"] + P[..., None] * want_h[:, None], side_room(ref["g_x"]) + np.abs(P)[..., None] * room_h[:, None]
    room_x = room_x + 4 * U * (np.abs(ref["g_x"]) + np.abs(P[..., None] * want_h[:, None]))
    assert (np.abs(D(g_x) - want_x) <= room_x).all()
    assert (np.abs(D(side["g_x"]) - want_x) > room_x).mean() > 0.5          # (the sublayer's part is no detail)
    want_p = ref["g_pre_mix"] + (X * want_h[:, None]).sum(-1)
    room_p = side_room(ref["g_pre_mix"]) + (np.abs(X) * room_h[:, None]).sum(-1) + d * U * (np.abs(X) * np.abs(want_h)[:, None]).sum(-1)
    assert (np.abs(D(g_pre_mix) - want_p) <= room_p).all()

    # the same chain without roundings against differences of the 64-bit loss, two steps joined
    def forward(X, P):
        H = (P[..., None] * X).sum(1)
        N = (H - mean_of(H)) / np.sqrt(mean_of((H - mean_of(H)) ** 2) + 1e-5) * LW + LB
        return H, np.concatenate([N[rows] @ W[e].T for e, rows in experts])

    loss = lambda X, P: (C * oracle.side_f64(X, P, forward(X, P)[1], *Q, rounded=False)["y"]).sum()
    H, F = forward(X, P)
    exact = oracle.side_backward(X, P, F, *Q, np.zeros((n, d)), C, rounded=False)
    e_h, _ = norm_backward(H, np.concatenate([exact["g_f"][rows] @ W[e] for e, rows in experts]), np.zeros((n, d)))
    e_x, e_p = exact["g_x"] + P[..., None] * e_h[:, None], exact["g_pre_mix"] + (X * e_h[:, None]).sum(-1)
    rng = np.random.default_rng(5)
    vx, vp = rng.standard_normal(X.shape), rng.standard_normal(P.shape)
    slope = lambda s: (loss(X + s * vx, P + s * vp) - loss(X - s * vx, P - s * vp)) / (2 * s)
    limit = (4 * slope(5e-5) - slope(1e-4)) / 3
    size = np.abs(e_x * vx).sum() + np.abs(e_p * vp).sum()
    assert abs((e_x * vx).sum() + (e_p * vp).sum() - limit) <= 1e-6 * size
    assert abs((exact["g_x"] * vx).sum() + (exact["g_pre_mix"] * vp).sum() - limit) > 1e-4 * size


def test_readme_example():
    """The README's training step runs on a side's tensors and moves every parameter."""
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as t:
        code = t.read().split("```python\n")[1].split("```")[0]
    s = Side(False)
    o = s.step()
    names = dict(torch=torch, x=s.x, pre_mix=s.pre_mix, f=o["f_rows"][s.back], hc_fn=s.hc_fn, hc_scale=s.hc_scale, hc_base=s.hc_base,
                 norm_w=s.norm_w, ln_w=s.ln_w, ln_b=s.ln_b, up=s.up16, h=o["h"], order=s.order, back=s.back, offsets=s.offsets,
                 g_a=o["g_a"], g_y=s.c, t=2)
    before = [v.clone() for v in (s.up16, s.ln_w, s.ln_b, s.hc_fn, s.hc_scale, s.hc_base)]
    exec(code, names)
    assert torch.equal(names["h_n"], hcg.hc_layer_norm(o["h"], before[1], before[2]))
    assert names["g_x"].shape == s.x.shape and names["g_pre_mix"].shape == s.pre_mix.shape
    for old, new in zip(before, names["params"]):
        assert new.isfinite().all() and not torch.equal(old, new)


_FIRST_CAPTURE = """
import torch
import hyper_connection_residual_mixes_gb300 as hcg
g = torch.Generator(device="cuda").manual_seed(2)
r = lambda *s: torch.randn(s, generator=g, device="cuda")
xs, w = [r(700, 5120).bfloat16(), r(9, 320), r(3, 9000).half()], r(9000)
rows, weights, off = r(300, 512).bfloat16(), r(4, 256, 512).bfloat16(), torch.tensor([0, 90, 100, 250, 300], dtype=torch.int32, device="cuda")
one, long = r(3, 8192).bfloat16(), r(2, 64, 8192).bfloat16()
few, many = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda"), torch.tensor([0, 9000], dtype=torch.int32, device="cuda")
a, b = r(9000, 64).bfloat16(), r(9000, 72).bfloat16()
params = [[torch.ones(5000, device="cuda"), torch.ones(70, 9, device="cuda")] for _ in range(2)]
states = [[hcg.adamw_state(p, mxfp8=k == 1) for k, p in enumerate(ps)] for ps in params]
plans = [hcg.adamw_plan(ps, [torch.full_like(p, 0.25) for p in ps], [s[0] for s in st], [s[1] for s in st]) for ps, st in zip(params, states)]

def work(k):
    out = []
    for x in xs:
        d = x.shape[1]
        y, mean, rstd = hcg.hc_layer_norm(x, w[:d].contiguous(), return_stats=True)
        out += [y, mean, rstd, *hcg.hc_layer_norm_backward(y, x, w[:d].contiguous(), mean, rstd).values()]
    out.append(hcg.hc_grouped_mm(rows, weights, off))
    out += hcg.hc_grouped_mm_backward(out[-1], rows, weights, off).values()
    out += [hcg.hc_grouped_mm(one, long, few), hcg.hc_grouped_mm_weights(a, b, many)]
    hcg.hc_adamw_step(plans[k], 1e-3, 1)
    return out

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = work(0)
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(p, q) for p, q in zip(captured, work(1)))
assert all(torch.equal(p, q) for p, q in zip(*params))
print("same")
"""


def test_first_calls_inside_a_capture():
    """In a process of its own: no kernel has run, or been loaded, before it is captured."""
    out = subprocess.run([sys.executable, "-c", _FIRST_CAPTURE], capture_output=True, text=True, timeout=300,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert out.returncode == 0 and out.stdout.split() == ["same"], out.stdout + out.stderr
