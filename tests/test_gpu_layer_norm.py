"""GPU: layer norm, forward and backward, against its formulas in 64 bits.

Bounds.  u = 2^-24.  A sum of the kernels adds at most 160 terms one after
the other in a lane and then some 15 partial sums, so it is off by at most
256 u times the sum of its terms' sizes.  With S = rstd mean|x| that makes
|d mean| rstd <= 256 u S, the relative error of rstd <= 300 u (the sum of
squares, its root and reciprocal), and
    |d y| <= (half a step of y's type) |y| + 1024 u (|w| (|xh| + S) + |b|),
    |d g_x| <= (half a step) |g_x| + 1024 u rstd (|wg| + mean|wg| + |xh| mean|wg xh|),
the constant with room for the few roundings per value.  Parameter gradients
add at most ceil(n / 128) + 128 terms one after the other: that many u times
the sum of the terms' sizes."""
import pytest
import torch

import hyper_connection_residual_mixes_gb300 as hcg
from hyper_connection_residual_mixes_gb300 import _lib
from hyper_connection_residual_mixes_gb300 import build as hc_build

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
T = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hc_build.build()
    _lib.load()


def _half(t):
    return torch.finfo(t).eps / 2


def _tiny(t):  # half the step of the type's smallest numbers
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def _inputs(n, d, x, w, g="fp32", pitch=0, seed=0, lead=0):
    gen = torch.Generator(device="cuda").manual_seed(1000 * seed + n + d)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    v = r(n, d) * (0.2 + 2 * torch.rand((n, 1), generator=gen, device="cuda")) + r(n, 1)
    buf = torch.full((n, d + pitch + lead), 7.0, dtype=T[x], device="cuda")
    buf[:, lead:lead + d] = v
    return (buf[:, lead:lead + d], (0.5 + torch.rand((d,), generator=gen, device="cuda")).to(T[w]),
            (0.3 * r(d)).to(T[w]), r(n, d).to(T[g]))


def _ref(x, w, b, eps):
    x, w = x.double(), w.double()
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + eps)
    xh = (x - mean) * rstd
    y = xh * w + (b.double() if b is not None else 0.0)
    room = 1024 * U * (w.abs() * (xh.abs() + rstd * x.abs().mean(1, keepdim=True)) + (b.double().abs() if b is not None else 0.0))
    return y, mean[:, 0], rstd[:, 0], room


def _check_forward(x, w, b, eps=1e-5):
    y, mean, rstd = hcg.hc_layer_norm(x, w, b, norm_eps=eps, return_stats=True)
    ry, rm, rr, room = _ref(x, w, b, eps)
    assert y.dtype == x.dtype and y.shape == x.shape
    assert ((y.double() - ry).abs() <= _half(x.dtype) * (ry.abs() + room) + _tiny(x.dtype) + room).all()
    assert ((mean.double() - rm).abs() <= 256 * U * x.double().abs().mean(1)).all()
    # the computed mean is off too: (mean + e)^2 adds e^2 to the variance
    e = 256 * U * x.double().abs().mean(1) * rr
    assert ((rstd.double() - rr).abs() <= (300 * U + e * e) * rr).all()
    return y, mean, rstd


CASES = [(1, 1), (1, 7), (3, 31), (5, 64), (2, 129), (7, 256), (4, 264), (33, 640), (3, 1000), (2, 1031), (17, 2048),
         (16, 5120), (2, 5121), (5, 8192), (2, 8200), (3, 16383), (2, 16384)]


@pytest.mark.parametrize("n,d", CASES)
@pytest.mark.parametrize("x,w", [("bf16", "fp32"), ("bf16", "bf16"), ("fp16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
def test_forward(n, d, x, w):
    x, w, b, _ = _inputs(n, d, x, w)
    _check_forward(x, w, b)
    _check_forward(x, w, None)


@pytest.mark.parametrize("d", [24, 256, 1024, 2048, 2056, 4096, 5120, 6144])
@pytest.mark.parametrize("x", ["bf16", "fp32"])
def test_forward_many_rows(d, x):
    x, w, b, _ = _inputs(1999, d, x, "fp32", seed=1)
    _check_forward(x, w, b)


@pytest.mark.parametrize("d,pitch,lead", [(512, 8, 0), (512, 1, 0), (512, 7, 1), (100, 4, 4), (5120, 3 * 5120, 0), (1030, 2, 2)])
@pytest.mark.parametrize("x,g", [("bf16", "fp32"), ("fp32", "fp32"), ("fp16", "fp16")])
def test_strided_rows(d, pitch, lead, x, g):
    """Rows of a wider buffer, aligned and not; the buffer around them stays as it is."""
    x, w, b, g_y = _inputs(37, d, x, "fp32", g, pitch, lead=lead)
    y, mean, rstd = _check_forward(x, w, b)
    out = torch.full((37, d + pitch + lead), 3.0, dtype=x.dtype, device="cuda")
    view = out[:, lead:lead + d]
    assert hcg.hc_layer_norm(x, w, b, y=view) is view
    assert torch.equal(view, y) or ((view.double() - y.double()).abs() <= 2 * torch.finfo(x.dtype).eps * (1 + y.double().abs())).all()
    assert (out[:, :lead] == 3).all() and (out[:, lead + d:] == 3).all()
    ref = _check_backward(x, w, g_y, mean, rstd)
    out = torch.full((37, d + pitch + lead), 3.0, dtype=g_y.dtype, device="cuda")
    view = out[:, lead:lead + d]
    got = hcg.hc_layer_norm_backward(g_y, x, w, mean, rstd, g_x=view)
    assert got["g_x"] is view and (out[:, :lead] == 3).all() and (out[:, lead + d:] == 3).all()
    _check_backward(x, w, g_y, mean, rstd, got)
    assert ref is not None


def test_one_stream_of_the_residual():
    """The streams of x [n, 4, d] as rows, all of them and one of them."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    s = torch.randn((9, 4, 320), generator=gen, device="cuda").to(torch.bfloat16)
    w, b = torch.rand((320,), device="cuda"), torch.rand((320,), device="cuda")
    every = hcg.hc_layer_norm(s, w, b)
    assert every.shape == s.shape
    for k in range(4):
        assert torch.equal(hcg.hc_layer_norm(s[:, k], w, b), every[:, k])
    assert torch.equal(hcg.hc_layer_norm(s[0, 0], w, b), every[0, 0])
    wide = s[0, 0].expand(5, 320)   # a broadcast row
    assert torch.equal(hcg.hc_layer_norm(wide, w, b), every[0, 0].expand(5, 320))


def _check_backward(x, w, g_y, mean, rstd, got=None, bias=True):
    if got is None:
        got = hcg.hc_layer_norm_backward(g_y, x, w, mean, rstd, bias=bias)
    n = x.shape[0]
    g, r = g_y.double(), rstd.double()[:, None]
    xh = (x.double() - mean.double()[:, None]) * r
    wg = g * w.double()
    m1, m2 = wg.mean(1, keepdim=True), (wg * xh).mean(1, keepdim=True)
    g_x = r * (wg - m1 - xh * m2)
    room = 1024 * U * r * (wg.abs() + wg.abs().mean(1, keepdim=True) + xh.abs() * (wg * xh).abs().mean(1, keepdim=True))
    t = g_y.dtype
    assert got["g_x"].dtype == t and got["g_x"].shape == x.shape
    assert ((got["g_x"].double() - g_x).abs() <= _half(t) * (g_x.abs() + room) + _tiny(t) + room).all()
    terms = -(-n // 128) + 128
    assert ((got["g_norm_w"].double() - (g * xh).sum(0)).abs() <= terms * U * (g * xh).abs().sum(0)).all()
    assert ("g_norm_b" in got) == bias
    if bias:
        assert ((got["g_norm_b"].double() - g.sum(0)).abs() <= terms * U * g.abs().sum(0)).all()
    return got


@pytest.mark.parametrize("n,d", CASES + [(1, 5120), (300, 128), (1300, 40), (700, 1024), (1000, 5120), (400, 2176),
                                         (305, 6152), (350, 8192)])
@pytest.mark.parametrize("x,g,w", [("bf16", "fp32", "fp32"), ("bf16", "bf16", "bf16"), ("fp16", "fp16", "fp32"),
                                   ("fp16", "fp32", "fp16"), ("fp32", "fp32", "fp32")])
def test_backward(n, d, x, g, w):
    x, w, b, g_y = _inputs(n, d, x, w, g, seed=2)
    _, mean, rstd = hcg.hc_layer_norm(x, w, b, return_stats=True)
    got = _check_backward(x, w, g_y, mean, rstd)
    again = _check_backward(x, w, g_y, mean, rstd, bias=False)
    assert torch.equal(got["g_x"], again["g_x"]) and torch.equal(got["g_norm_w"], again["g_norm_w"])


@pytest.mark.parametrize("x,g", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
def test_rows_of_one_column_have_no_gradient(x, g):
    """d = 1: x is its own mean, so y does not depend on it."""
    v, w, b, gr = _inputs(777, 1, x, "fp32", g, seed=6)
    y, mean, rstd = hcg.hc_layer_norm(v, w, b, return_stats=True)
    assert torch.equal(y, b.to(y.dtype).expand(777, 1)) and torch.equal(mean, v[:, 0].float())
    got = hcg.hc_layer_norm_backward(gr, v, w, mean, rstd)
    assert (got["g_x"] == 0).all() and (got["g_norm_w"] == 0).all()


@pytest.mark.parametrize("n,d,pitch,lead", [
    (2500, 1025, 0, 0), (2500, 1026, 0, 0), (2600, 1028, 0, 4), (1800, 1435, 0, 3), (1800, 1438, 2, 2), (900, 2999, 1, 0),
    (700, 5119, 1, 0), (700, 5119, 0, 1), (600, 5118, 0, 0), (600, 5121, 0, 0), (500, 6143, 8, 5), (400, 7001, 0, 7),
    (320, 8191, 0, 0), (320, 8190, 4, 2), (300, 9003, 0, 1), (260, 12286, 0, 2), (170, 16383, 0, 0), (19000, 131, 0, 1),
    (9800, 257, 0, 0), (9700, 258, 2, 0), (5000, 514, 0, 6), (2450, 1023, 0, 1), (6000, 520, 0, 0), (5, 1031, 0, 3), (1, 2049, 0, 5)])
@pytest.mark.parametrize("x,g", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
def test_rows_anywhere(n, d, pitch, lead, x, g):
    """Many rows that start and end inside 16-byte blocks, with NaN in all that is
    around them (before the first and behind the last row too)."""
    v, w, b, gr = _inputs(n, d, x, "fp32", g, seed=5)

    def among_nan(t):
        step = d + pitch
        buf = torch.full((lead + n * step + 16,), float("nan"), dtype=t.dtype, device="cuda")
        rows = buf[lead:lead + n * step].view(n, step)[:, :d]
        rows.copy_(t)
        return rows

    v, gr = among_nan(v), among_nan(gr)
    _, mean, rstd = _check_forward(v, w, b)
    y = among_nan(torch.zeros((n, d), dtype=v.dtype, device="cuda"))
    hcg.hc_layer_norm(v, w, b, y=y)
    assert torch.isfinite(y).all()
    if pitch:
        assert torch.isnan(y.as_strided((n - 1, pitch), (d + pitch, 1), y.storage_offset() + d)).all()
    g_x = among_nan(torch.zeros((n, d), dtype=gr.dtype, device="cuda"))
    got = hcg.hc_layer_norm_backward(gr, v, w, mean, rstd, g_x=g_x)
    _check_backward(v, w, gr, mean, rstd, got)
    if pitch:
        assert torch.isnan(g_x.as_strided((n - 1, pitch), (d + pitch, 1), g_x.storage_offset() + d)).all()


@pytest.mark.parametrize("x", ["bf16", "fp32"])
def test_overlapping_rows_anywhere(x):
    """Rows that are one another's neighbours by a single value, and one row for all."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    buf = torch.randn((3 + 2000 + 1301,), generator=gen, device="cuda").to(T[x])
    w, b = torch.rand((1301,), generator=gen, device="cuda"), torch.rand((1301,), generator=gen, device="cuda")
    for step in (0, 1):
        rows = buf.as_strided((2000, 1301), (step, 1), 3)
        _, mean, rstd = _check_forward(rows, w, b)
        _check_backward(rows, w, torch.randn((2000, 1301), generator=gen, device="cuda"), mean, rstd)


def test_gradients_against_differences():
    """Central differences of the kernel's own forward, in 32 bits, along random
    directions: they may be off by the forward's error over the step, and by
    the third derivative's part, for which the 64-bit forward's differences stand."""
    n, d, h = 6, 48, 2.0 ** -5
    x, w, b, g_y = _inputs(n, d, "fp32", "fp32", seed=5)
    _, mean, rstd = hcg.hc_layer_norm(x, w, b, return_stats=True)
    got = hcg.hc_layer_norm_backward(g_y, x, w, mean, rstd)
    gen = torch.Generator(device="cuda").manual_seed(8)
    for which, key in (("x", "g_x"), ("w", "g_norm_w"), ("b", "g_norm_b")):
        v = torch.randn({"x": (n, d), "w": (d,), "b": (d,)}[which], generator=gen, device="cuda")
        args = lambda s: {k: t + s * h * v if k == which else t for k, t in (("x", x), ("w", w), ("b", b))}
        loss, exact, room = [], [], 0.0
        for s in (1, -1):
            a = args(s)
            y, ry = hcg.hc_layer_norm(a["x"], a["w"], a["b"]).double(), _ref(a["x"], a["w"], a["b"], 1e-5)
            loss.append((g_y.double() * y).sum())
            exact.append((g_y.double() * ry[0]).sum())
            room += float((g_y.double().abs() * (ry[3] + U * ry[0].abs())).sum())
        kernel, formula = (loss[0] - loss[1]) / (2 * h), (exact[0] - exact[1]) / (2 * h)
        assert abs(float(kernel - formula)) <= room / (2 * h)
        # the 64-bit difference against the gradient: h^2 terms, from two steps
        a2 = {k: t.double() for k, t in (("x", x), ("w", w), ("b", b))}
        diff = lambda e: sum(s * float((g_y.double() * _ref(*[a2[k] + (s * e * v.double() if k == which else 0) for k in "xwb"], 1e-5)[0]).sum()) for s in (1, -1)) / (2 * e)
        d1, d2 = diff(h / 16), diff(h / 32)
        limit = d2 + (d2 - d1) / 3
        slope = float((got[key].double() * v.double()).sum())
        size = float((got[key].double().abs() * v.double().abs()).sum())
        assert abs(slope - limit) <= 1024 * U * 8 * size + 1e-6 * size


def test_rows_of_one_value_and_offsets():
    """Constant rows (variance 0), large offsets, a width of one."""
    w, b = torch.rand((256,), device="cuda"), torch.rand((256,), device="cuda")
    x = torch.full((3, 256), 5.0, device="cuda")
    assert torch.equal(hcg.hc_layer_norm(x, w, b), b.expand(3, 256))
    x = 4096.0 + torch.randn((64, 256), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    _check_forward(x, w, b)
    one = torch.tensor([[3.0], [-2.0]], device="cuda")
    assert torch.equal(hcg.hc_layer_norm(one, w[:1], b[:1]), b[:1].expand(2, 1))


@pytest.mark.parametrize("n,d", [(700, 1024), (1000, 5120), (650, 1304)])
def test_infinite_and_nan_rows_among_many(n, d):
    """The same where rows stream through a block one after the other."""
    x, w, b, g_y = _inputs(n, d, "bf16", "fp32", seed=10)
    clean = hcg.hc_layer_norm(x, w, b)
    x = x.clone()
    x[3, 5], x[n - 2, d - 1], x[400] = float("inf"), float("nan"), float("-inf")
    y, mean, rstd = hcg.hc_layer_norm(x, w, b, return_stats=True)
    rows = torch.ones((n,), dtype=torch.bool, device="cuda")
    rows[[3, n - 2, 400]] = False
    assert torch.equal(y[rows], clean[rows]) and y[~rows].isnan().all()
    got = hcg.hc_layer_norm_backward(g_y, x, w, mean, rstd)
    assert got["g_x"][rows].isfinite().all() and got["g_x"][n - 2].isnan().all()


def test_infinite_and_nan_rows_stay_in_their_row():
    x, w, b, g_y = _inputs(12, 1024, "bf16", "fp32", seed=9)
    clean = hcg.hc_layer_norm(x, w, b)
    x = x.clone()
    x[3, 5], x[7, 1000] = float("inf"), float("nan")
    y, mean, rstd = hcg.hc_layer_norm(x, w, b, return_stats=True)
    rows = [r for r in range(12) if r not in (3, 7)]
    assert torch.equal(y[rows], clean[rows]) and y[3].isnan().all() and y[7].isnan().all()
    got = hcg.hc_layer_norm_backward(g_y, x, w, mean, rstd)
    assert got["g_x"][rows].isfinite().all() and got["g_x"][7].isnan().all()


def test_empty():
    w = torch.ones((64,), device="cuda")
    x = torch.empty((0, 64), device="cuda")
    y, mean, rstd = hcg.hc_layer_norm(x, w, return_stats=True)
    assert y.shape == (0, 64) and mean.shape == (0,)
    got = hcg.hc_layer_norm_backward(x, x, w, mean, rstd)
    assert (got["g_norm_w"] == 0).all() and (got["g_norm_b"] == 0).all()


def test_other_stream_and_graph():
    """On a stream of its own, and captured: replays on new inputs give the eager bits."""
    x, w, b, g_y = _inputs(700, 1024, "bf16", "fp32", seed=11)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, mean, rstd = hcg.hc_layer_norm(x, w, b, return_stats=True, stream=s)
    got = hcg.hc_layer_norm_backward(g_y, x, w, mean, rstd, stream=s)
    s.synchronize()
    ref = hcg.hc_layer_norm(x, w, b)
    assert torch.equal(y, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cy, cm, cr = hcg.hc_layer_norm(x, w, b, return_stats=True)
        cg = hcg.hc_layer_norm_backward(g_y, x, w, cm, cr)
    for seed in (12, 13):
        x2, _, _, g2 = _inputs(700, 1024, "bf16", "fp32", seed=seed)
        x.copy_(x2), g_y.copy_(g2)
        graph.replay()
        torch.cuda.synchronize()
        y, mean, rstd = hcg.hc_layer_norm(x, w, b, return_stats=True)
        want = hcg.hc_layer_norm_backward(g_y, x, w, mean, rstd)
        assert torch.equal(cy, y) and all(torch.equal(cg[k], want[k]) for k in want)
    assert got["g_x"].shape == x.shape


def test_offsets_beyond_32_bits():
    """Rows whose elements lie past 2^31 in the buffer."""
    d, stride = 64, 1 << 28
    buf = torch.empty((10 * stride,), dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((10, d), (stride, 1))
    x.copy_(torch.randn((10, d), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda"))
    w = torch.rand((d,), device="cuda")
    assert torch.equal(hcg.hc_layer_norm(x, w), hcg.hc_layer_norm(x.contiguous(), w))


@pytest.mark.parametrize("n,d,pitch,lead", [(2500, 1025, 0, 1), (1800, 1438, 2, 2), (700, 5119, 1, 3), (500, 6143, 8, 5), (320, 8190, 4, 2),
                                            (170, 16383, 0, 7), (19000, 131, 0, 1), (9800, 258, 2, 0), (5, 1031, 0, 3), (3, 77, 5, 2),
                                            (1, 2049, 0, 5), (40, 512, 8, 8)])
@pytest.mark.parametrize("x,g", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
def test_outputs_lie_in_their_rows(n, d, pitch, lead, x, g):
    """Outputs in rows of a wider buffer: every value in its place, every NaN around
    them (before the first row, between rows, behind the last) still there."""
    v, w, b, gr = _inputs(n, d, x, "fp32", g, seed=7)
    _, mean, rstd = _check_forward(v, w, b)

    def among_nan(dtype):
        buf = torch.full((lead + n * (d + pitch) + 16,), float("nan"), dtype=dtype, device="cuda")
        rows = buf[lead:lead + n * (d + pitch)].view(n, d + pitch)[:, :d]
        outside = torch.ones_like(buf, dtype=torch.bool)
        outside[lead:lead + n * (d + pitch)].view(n, d + pitch)[:, :d] = False
        return buf, rows, outside

    buf, y, outside = among_nan(v.dtype)
    hcg.hc_layer_norm(v, w, b, y=y)
    want, _, _, room = _ref(v, w, b, 1e-5)
    assert ((y.double() - want).abs() <= _half(v.dtype) * (want.abs() + room) + _tiny(v.dtype) + room).all()
    assert buf[outside].isnan().all()
    buf, g_x, outside = among_nan(gr.dtype)
    _check_backward(v, w, gr, mean, rstd, hcg.hc_layer_norm_backward(gr, v, w, mean, rstd, g_x=g_x))
    assert buf[outside].isnan().all()
