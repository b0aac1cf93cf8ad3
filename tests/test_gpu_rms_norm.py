"""GPU: RMS norm with the residual, its backward and the casts to 8 bits, against
their formulas in 64 bits.

Bounds.  u = 2^-24.  A lane adds at most 64 squares one after the other, then some
10 partial sums: the sum of squares is off by at most 80 u of itself, its mean, root
and reciprocal by some units more: rstd by 64 u, y in fp32 by 70 u, which leaves
    |d y| <= (half a step of y's type) |y| + 100 u |y|.
A code stands for a value within half a step (2^-4 of it, at least 2^-10 scales) of
y; its scale is the smallest power of two at or above amax / 448 of amax, itself
100 u off.  In the backward, with the same sums,
    |d g_x| <= (half a step) |g_x| + 128 u (|g_r| + rstd (|wg| + |xh| mean|wg xh|)),
parameter gradients add at most ceil(n / 304) + 64 terms one after the other: that
many u, and some for each term, times the sum of the terms' sizes."""
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


def _rand(seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(s, generator=gen, device="cuda")


def _in(v, t, lead=0, pitch=0):
    """v in rows of a wider buffer."""
    n, d = v.shape
    buf = torch.full((n, lead + d + pitch), 7.0, dtype=t, device="cuda")
    buf[:, lead:lead + d] = v
    return buf[:, lead:lead + d]


def _two(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _spread(scales, d):
    return scales.repeat_interleave(128, -1)[..., :d]


def _check_codes(y, codes, scales, off):
    """codes and scales of y, known to `off` of itself."""
    n, d = y.shape
    assert codes.dtype == scales.dtype == torch.uint8 and codes.shape == y.shape and scales.shape == (n, -(-d // 128))
    pad = torch.nn.functional.pad(y, (0, -d % 128)).view(n, -1, 128)
    amax, s = pad.abs().amax(2), _two(scales.long() - 127)
    assert (scales >= 1).all() and (amax * (1 - off) <= 448 * s).all()
    assert ((amax * (1 + off) > 224 * s) | (scales == 1)).all()
    s = _spread(s, d)
    v = codes.view(torch.float8_e4m3fn).double() * s
    assert ((v - y).abs() <= 2.0 ** -4 * torch.maximum(y.abs(), s * 2.0 ** -6) + off * y.abs()).all()


def _ref(x, w, res, eps):
    v = x
    if res is not None:
        v = (x.float() + res.float()).to(x.dtype)
    f = v.double()
    rstd = 1 / torch.sqrt(f.square().mean(1, keepdim=True) + eps)
    return v, rstd[:, 0], f * rstd * w.double()


def _check_forward(x, w, res, eps=1e-6, **given):
    v, rstd, y = _ref(x, w, res, eps)
    got = hcg.hc_rms_norm(x, w, res, norm_eps=eps, out="both", return_rstd=True, **given)
    assert set(got) == {"y", "codes", "scales", "rstd"} | ({"r"} if res is not None else set())
    if res is not None:
        assert got["r"].dtype == x.dtype and torch.equal(got["r"], v)
    assert ((got["rstd"].double() - rstd).abs() <= 64 * U * rstd).all()
    assert got["y"].dtype == x.dtype
    assert ((got["y"].double() - y).abs() <= (_half(x.dtype) + 100 * U) * y.abs() + _tiny(x.dtype)).all()
    _check_codes(y, got["codes"], got["scales"], 100 * U)
    return got


CASES = [(1, 1), (1, 7), (3, 31), (5, 64), (2, 128), (2, 129), (7, 256), (4, 264), (33, 640), (3, 1000), (2, 1031), (17, 2048),
         (16, 5120), (2, 5121), (5, 8192), (2, 8200), (3, 16383), (2, 16384)]


@pytest.mark.parametrize("n,d", CASES)
@pytest.mark.parametrize("x,w", [("bf16", "fp32"), ("bf16", "bf16"), ("fp16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
def test_forward(n, d, x, w):
    r = _rand(n + d)
    xv, wv = (3 * r(n, d)).to(T[x]), (0.5 + r(d).abs()).to(T[w])
    res = r(n, d).to(T[x])
    both = _check_forward(xv, wv, res)
    _check_forward(xv, wv, None)
    # the outputs by themselves are the same
    y = hcg.hc_rms_norm(xv, wv, res)
    assert set(y) == {"r", "y"} and torch.equal(y["y"], both["y"]) and torch.equal(y["r"], both["r"])
    q = hcg.hc_rms_norm(xv, wv, res, out="fp8")
    assert set(q) == {"r", "codes", "scales"} and torch.equal(q["codes"], both["codes"]) and torch.equal(q["scales"], both["scales"])


@pytest.mark.parametrize("d", [24, 256, 1024, 2048, 2056, 4096, 5120, 6144])
@pytest.mark.parametrize("x", ["bf16", "fp32"])
def test_forward_many_rows(d, x):
    r = _rand(d)
    _check_forward(r(1999, d).to(T[x]), r(d), r(1999, d).to(T[x]))


@pytest.mark.parametrize("n,d", [(400, 8192), (320, 12288), (310, 16384)])
@pytest.mark.parametrize("x", ["bf16", "fp32"])
def test_many_wide_rows(n, d, x):
    """Rows of which few, or one, fit into an SM's memory at a time."""
    r = _rand(d)
    xv, w, res = r(n, d).to(T[x]), r(d), r(n, d).to(T[x])
    got = _check_forward(xv, w, res)
    _check_forward(xv, w, None)
    gy, gr = r(n, d), r(n, d)
    _check_backward(gy, xv, w, got["rstd"], gr, hcg.hc_rms_norm_backward(gy, xv, w, got["rstd"], g_r=gr))


def test_offsets_past_32_bits():
    """The last of 840,000 rows of 5,120, more than 2^32 values."""
    n, d = 840000, 5120
    x, w = torch.empty((n, d), dtype=torch.bfloat16, device="cuda"), _rand(1)(d)
    x[:64], x[-64:] = _rand(2)(64, d), _rand(3)(64, d)
    x[64:-64] = 1
    got = hcg.hc_rms_norm(x, w, out="both", return_rstd=True)
    _, rstd, y = _ref(x[-64:], w, None, 1e-6)
    assert ((got["y"][-64:].double() - y).abs() <= (_half(x.dtype) + 100 * U) * y.abs() + _tiny(x.dtype)).all()
    _check_codes(y, got["codes"][-64:], got["scales"][-64:], 100 * U)
    codes, scales = hcg.hc_fp8_cast(got["y"], codes=got["codes"], scales=got["scales"])
    again = hcg.hc_fp8_cast(got["y"][-64:].clone())
    assert torch.equal(codes[-64:], again[0]) and torch.equal(scales[-64:], again[1])
    back = hcg.hc_rms_norm_backward(x, x, w, got["rstd"], g_x=got["y"])     # (g_x over y, which nothing reads)
    gy = x[-64:]
    alone = hcg.hc_rms_norm_backward(gy.contiguous(), gy.contiguous(), w, got["rstd"][-64:].contiguous())
    _check_backward(gy, gy, w, got["rstd"][-64:], None, {"g_x": back["g_x"][-64:], "g_norm_w": alone["g_norm_w"]})


@pytest.mark.parametrize("d,pitch,lead", [(512, 8, 0), (512, 1, 0), (512, 7, 1), (100, 4, 4), (5120, 5120, 0), (1030, 2, 2)])
@pytest.mark.parametrize("x,g", [("bf16", "fp32"), ("fp32", "fp32"), ("fp16", "fp16")])
def test_strided_rows(d, pitch, lead, x, g):
    """Rows of wider buffers, aligned and not; the buffers around them stay as they are."""
    r, t = _rand(d), T[x]
    xv, res, w = _in(r(37, d), t, lead, pitch), _in(r(37, d), t, lead, pitch), r(d)
    out = [_in(torch.zeros((37, d), device="cuda"), q, lead, pitch) for q in (t, t, torch.uint8)]
    whole = [o._base for o in out]
    scales = torch.empty((37, -(-d // 128)), dtype=torch.uint8, device="cuda")
    got = _check_forward(xv, w, res, r=out[0], y=out[1], codes=out[2], scales=scales)
    assert got["r"] is out[0] and got["y"] is out[1] and got["codes"] is out[2] and got["scales"] is scales
    for b in whole:
        assert (b[:, :lead] == 7).all() and (b[:, lead + d:] == 7).all()
    gy, gr = _in(r(37, d), T[g], lead, pitch), _in(r(37, d), T[g], lead, pitch)
    gx = _in(torch.zeros((37, d), device="cuda"), T[g], lead, pitch)
    back = hcg.hc_rms_norm_backward(gy, got["r"], w, got["rstd"], g_r=gr, g_x=gx)
    assert back["g_x"] is gx and (gx._base[:, :lead] == 7).all() and (gx._base[:, lead + d:] == 7).all()
    _check_backward(gy, got["r"], w, got["rstd"], gr, back)


@pytest.mark.parametrize("n,d", [(3, 40), (300, 1024), (700, 5120), (5, 1031)])
def test_in_place(n, d):
    """r written over the residual, over x, and over both where they are one."""
    r = _rand(n * d)
    x, res, w = r(n, d).bfloat16(), r(n, d).bfloat16(), r(d)
    want = hcg.hc_rms_norm(x, w, res, out="both")
    for target in (0, 1):
        a, b = x.clone(), res.clone()
        got = hcg.hc_rms_norm(a, w, b, out="both", r=(a, b)[target])
        assert got["r"] is (a, b)[target]
        for k in want:
            assert torch.equal(want[k], got[k]), k
    a = x.clone()
    got = hcg.hc_rms_norm(a, w, a, r=a)
    assert torch.equal(a, x + x)
    g, gr = r(n, d), r(n, d)
    rstd = torch.rand((n,), device="cuda")
    want = hcg.hc_rms_norm_backward(g, x, w, rstd, g_r=gr)
    got = hcg.hc_rms_norm_backward(g, x, w, rstd, g_r=gr, g_x=gr)
    assert torch.equal(want["g_x"], gr) and torch.equal(want["g_norm_w"], got["g_norm_w"])


def test_broadcast_rows():
    """One row for all: x and the residual with stride 0; the sum of gradients is the caller's."""
    r = _rand(5)
    x, res, w = r(1, 320).expand(9, 320), r(9, 320), r(320)
    _check_forward(x, w, res)
    _check_forward(res, w, x)
    three = hcg.hc_rms_norm(r(2, 3, 320), w, out="fp8")
    assert three["codes"].shape == (2, 3, 320) and three["scales"].shape == (2, 3, 3)


def _check_backward(g, v, w, rstd, gr, got):
    f, rs, gd = v.double(), rstd.double()[:, None], g.double()
    n, d = f.shape
    xh, wg = f * rs, gd * w.double()
    past = gr.double() if gr is not None else torch.zeros_like(f)
    want = past + rs * (wg - xh * (wg * xh).mean(1, keepdim=True))
    room = 128 * U * (past.abs() + rs * (wg.abs() + xh.abs() * (wg * xh).abs().mean(1, keepdim=True)))
    assert got["g_x"].dtype == g.dtype
    assert ((got["g_x"].double() - want).abs() <= _half(g.dtype) * (want.abs() + room) + room + _tiny(g.dtype)).all()
    room = (-(-n // 304) + 72) * U * (gd * xh).abs().sum(0)
    assert ((got["g_norm_w"].double() - (gd * xh).sum(0)).abs() <= room).all()


@pytest.mark.parametrize("n,d", CASES + [(1999, 40), (1999, 512), (701, 5120), (650, 2056), (611, 1031), (40, 16384)])
@pytest.mark.parametrize("x,g", [("bf16", "fp32"), ("bf16", "bf16"), ("fp16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
def test_backward(n, d, x, g):
    r = _rand(n + 3 * d)
    v, w, gy, gr = r(n, d).to(T[x]), r(d).to(T[x]), r(n, d).to(T[g]), r(n, d).to(T[g])
    rstd = (v.double().square().mean(1) + 1e-6).rsqrt().float()
    for past in (gr, None):
        got = hcg.hc_rms_norm_backward(gy, v, w, rstd, g_r=past)
        _check_backward(gy, v, w, rstd, past, got)
        again = hcg.hc_rms_norm_backward(gy, v, w, rstd, g_r=past)
        assert torch.equal(got["g_x"], again["g_x"]) and torch.equal(got["g_norm_w"], again["g_norm_w"])


def test_backward_against_differences():
    """The gradient along a direction against central differences of the formula in 64
    bits: of a step h = 1e-4 these are off by some h^2 = 1e-8 of the third derivative."""
    r = _rand(11)
    x, res, w, g, gr = (r(6, 200) for _ in range(5))
    w = w[0].contiguous()
    got = hcg.hc_rms_norm(x, w, res, norm_eps=1e-3, return_rstd=True)
    back = hcg.hc_rms_norm_backward(g, got["r"], w, got["rstd"], g_r=gr)

    def loss(v, w):
        y = v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-3) * w
        return (y * g.double()).sum() + (v * gr.double()).sum()
    v, dv, dw, h = got["r"].double(), r(6, 200).double(), r(200).double(), 1e-4
    num = (loss(v + h * dv, w.double()) - loss(v - h * dv, w.double())) / (2 * h)
    assert abs(num - (back["g_x"].double() * dv).sum()) <= 1e-6 * (back["g_x"].double() * dv).abs().sum()
    num = (loss(v, w.double() + h * dw) - loss(v, w.double() - h * dw)) / (2 * h)
    assert abs(num - (back["g_norm_w"].double() * dw).sum()) <= 1e-6 * (back["g_norm_w"].double() * dw).abs().sum()


def test_no_rows():
    w = torch.ones((64,), device="cuda")
    got = hcg.hc_rms_norm(torch.empty((0, 64), device="cuda"), w, out="both")
    assert got["y"].shape == got["codes"].shape == (0, 64) and got["scales"].shape == (0, 1)
    back = hcg.hc_rms_norm_backward(torch.empty((0, 64), device="cuda"), torch.empty((0, 64), device="cuda"), w, torch.empty((0,), device="cuda"))
    assert back["g_x"].shape == (0, 64) and (back["g_norm_w"] == 0).all()
    assert hcg.hc_fp8_cast(torch.empty((0, 64), device="cuda"))[0].shape == (0, 64)


# ------------------------------------------------------------------ casts
def _cast_ref(v):
    """Codes and scale bytes of groups v [..., m] of finite values, from the rule."""
    mant, expo = torch.frexp(v.abs().amax(-1))
    e = torch.where(mant == 0, -126, expo - 9 + (mant > 0.875).int()).clamp(min=-126)
    q = v.double() / _two(e)[..., None]
    return q.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _groups(x):
    d = x.shape[-1]
    return torch.nn.functional.pad(x, (0, -d % 128)).unflatten(-1, (-1, 128))


def _values(n, d, t, seed):
    """Rows over the whole range of sizes, groups of zeros, of subnormals, at the borders of a scale."""
    r = _rand(seed)
    top = 20 if t == torch.float32 else 12
    x = r(n, d) * torch.exp2(r(n, 1) * top / 3).clamp(2.0 ** -top, 2.0 ** top)
    x[0] = 0
    if n > 1:
        x[1] *= 2.0 ** -20 if t == torch.float16 else 2.0 ** -130
    if n > 2:
        x[2] = 0.01 * r(d)
        x[2, 0] = 448.0
    if n > 3:
        x[3] = r(d)
        x[3, -1] = -450.0
    return x.to(t)


@pytest.mark.parametrize("n,d", [(1, 1), (4, 5), (3, 128), (5, 130), (7, 1031), (9, 1024), (64, 5120), (1000, 136), (2, 40000)])
@pytest.mark.parametrize("t", ["fp32", "bf16", "fp16"])
def test_cast(n, d, t):
    x = _values(n, d, T[t], n + d)
    codes, scales = hcg.hc_fp8_cast(x)
    q, s = _cast_ref(_groups(x.float()))
    assert torch.equal(scales, s) and torch.equal(codes, q.flatten(-2)[..., :d])
    # rows that start anywhere, codes in a wider buffer
    out = _in(torch.zeros((n, d), device="cuda"), torch.uint8, 3, 2)
    got = hcg.hc_fp8_cast(_in(x, T[t], 1, 2), codes=out, scales=torch.empty_like(scales))
    assert torch.equal(got[0], codes) and torch.equal(got[1], scales)
    assert (out._base[:, :3] == 7).all() and (out._base[:, 3 + d:] == 7).all()


@pytest.mark.parametrize("shape", [(1, 1), (128, 128), (130, 260), (3, 64, 200), (2, 2, 384, 136), (5, 1031)])
@pytest.mark.parametrize("t", ["fp32", "bf16", "fp16"])
def test_cast_weights(shape, t):
    w = _values(shape[0], torch.Size(shape[1:]).numel(), T[t], sum(shape)).view(shape).contiguous()
    codes, scales = hcg.hc_fp8_cast_weights(w)
    N, K = shape[-2:]
    f = torch.nn.functional.pad(w.float(), (0, -K % 128, 0, -N % 128))
    f = f.unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128)).transpose(-3, -2)       # [.., nb, kb, 128, 128]
    q, s = _cast_ref(f.flatten(-2))
    q = q.unflatten(-1, (128, 128)).transpose(-3, -2).flatten(-4, -3).flatten(-2)[..., :N, :K]
    assert torch.equal(scales, s) and torch.equal(codes, q)


def test_not_finite():
    """A NaN stays one and leaves its group's scale to the others; an infinite value is
    one again when decoded; other groups and rows are not touched."""
    x = torch.ones((3, 300), device="cuda")
    x[0, 5], x[1, 140] = float("nan"), -float("inf")
    for t in (torch.float32, torch.bfloat16, torch.float16):
        codes, scales = hcg.hc_fp8_cast(x.to(t))
        v = codes.view(torch.float8_e4m3fn).float() * _spread(_two(scales.long() - 127), 300).float()
        assert v[0, 5].isnan() and v[1, 140] == -float("inf")
        ok = torch.ones_like(x, dtype=torch.bool)
        ok[0, 5] = False
        ok[1, 128:256] = False
        assert (v[ok] == 1).all()
    w = torch.ones((64,), device="cuda")
    big = torch.full((2, 64), 1e30, device="cuda")
    big[1] = 1
    got = hcg.hc_rms_norm(big, w, out="both", return_rstd=True)
    # a sum of squares that overflows: rstd is 0, and so is the row; the other row is its own
    assert got["rstd"][0] == 0 and (got["y"][0] == 0).all() and (got["codes"][0] == 0).all()
    assert ((got["y"][1] - 1).abs() < 1e-5).all()
    nan = torch.ones((2, 64), device="cuda")
    nan[0, 3] = float("nan")
    got = hcg.hc_rms_norm(nan, w, out="both")
    assert got["y"][0].isnan().all() and (got["codes"][0] & 0x7f == 0x7f).all() and ((got["y"][1] - 1).abs() < 1e-5).all()


def test_streams():
    """Calls on a stream of their own."""
    r = _rand(8)
    x, res, w = r(500, 1024).bfloat16(), r(500, 1024).bfloat16(), r(1024)
    want = hcg.hc_rms_norm(x, w, res, out="both", return_rstd=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = hcg.hc_rms_norm(x, w, res, out="both", return_rstd=True, stream=side)
    back = hcg.hc_rms_norm_backward(x.float(), got["r"], w, got["rstd"], stream=side)
    codes, scales = hcg.hc_fp8_cast(got["y"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for k in want:
        assert torch.equal(want[k], got[k]), k
    assert torch.equal(back["g_x"], hcg.hc_rms_norm_backward(x.float(), want["r"], w, want["rstd"])["g_x"])
    assert torch.equal(codes, hcg.hc_fp8_cast(want["y"])[0])
