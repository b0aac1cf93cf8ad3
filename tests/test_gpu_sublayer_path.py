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

import pytest
import torch

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
