"""GPU: scales from all over their range, fp32 and UE8M0, in the products of 8-bit numbers.

The two scales of a block are multiplied first, and their product is an fp32 number: one that is
subnormal keeps fewer bits, from 2^128 on it is infinite.  So the reference takes this product
rounded to fp32, and everything else in 64 bits:
    y = sum over blocks of fp32(sx sw) sum.
Bounds: those of the operator's own tests with these products; sums of subnormal terms are off by
at most 2^-149 for each of the blocks and slices added."""
import pytest
import torch

import hyper_connection_residual_mixes_gb300 as hcg
from hyper_connection_residual_mixes_gb300 import _lib
from hyper_connection_residual_mixes_gb300 import build as hc_build
from tests import test_gpu_fp8_mm as mm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hc_build.build()
    _lib.load()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _near(shape, e, kind, g):
    """Scales of 2^e: UE8M0, or fp32 up to twice that."""
    if kind == "ue8m0":
        return torch.full(shape, e + 127, dtype=torch.uint8, device="cuda")
    return torch.ldexp(1 + torch.rand(shape, generator=g, device="cuda"), torch.tensor(e, device="cuda"))


def _check(y, x, sx, w, sw, transposed):
    """fp32 outputs; transposed as hc_fp8_mm's."""
    a, b = (t.view(torch.float8_e4m3fn).double() for t in (x, w))
    b, s = (b, sw) if transposed else (b.t(), sw.t())           # [L, C], [blocks of L, blocks of C]
    want = torch.zeros(y.shape, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for i in range(mm._blocks(x.shape[1])):
        k = slice(128 * i, min(128 * i + 128, x.shape[1]))
        # (both factors in 64 bits, their product exactly, rounded once)
        p = (mm._value(sx[:, i:i + 1]) * mm._value(s[i:i + 1]).repeat_interleave(128, 1)[:, :y.shape[1]]).float().double()
        want += p * (a[:, k] @ b[k])
        size += p.abs() * (a[:, k].abs() @ b[k].abs())
    blocks = mm._blocks(x.shape[1])
    room = (132 * 2.0 ** -23 + (blocks + 5) * U) * size + (blocks + 1) * 2.0 ** -149
    bad = (y.double() - want).abs() > room
    assert y.dtype == torch.float32 and not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


# few rows, tiles of 128 and 256 columns, a contraction that is cut
SIZES = [(1, 144, 272), (12, 528, 1040), (40, 272, 400), (300, 528, 1040), (2304, 2064, 144), (64, 640, 4112)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("xe,xk,we,wk", [(-126, "ue8m0", -13, "fp32"), (-13, "fp32", -126, "ue8m0"), (-70, "fp32", -76, "fp32"),
                                         (-127, "ue8m0", -20, "ue8m0"), (-127, "ue8m0", -30, "ue8m0"), (-100, "fp32", 90, "fp32"),
                                         (110, "ue8m0", -120, "fp32")])
def test_far_from_one(M, N, K, transposed, xe, xk, we, wk):
    """Products of scales that are subnormal, 0, or of a large and a small one."""
    g = _gen(M + N)
    L = N if transposed else K
    code = lambda *s: (256 + 192 * torch.rand(s, generator=g, device="cuda")).to(torch.float8_e4m3fn).view(torch.uint8)
    x, w = code(M, L), code(N, K)
    sx, sw = _near((M, mm._blocks(L)), xe, xk, g), _near((mm._blocks(N), mm._blocks(K)), we, wk, g)
    y = hcg.hc_fp8_mm(x, sx, w, sw, transposed=transposed, out_dtype=torch.float32)
    assert (y > 0).all() == (xe + we >= -149) and y.isfinite().all()
    _check(y, x, sx, w, sw, transposed)
    # such blocks beside ordinary ones, of which nothing is lost
    sx2, sw2 = mm._value(sx).float(), _near(sw.shape, -20, "fp32", g)
    sx2[:, 1::2] = 1.5
    y = hcg.hc_fp8_mm(x, sx2, w, sw2, transposed=transposed, out_dtype=torch.float32)
    _check(y, x, sx2, w, sw2, transposed)


@pytest.mark.parametrize("M", [3, 40, 300])
@pytest.mark.parametrize("transposed", [False, True])
def test_past_the_largest(M, transposed):
    """A product of scales past 2^128 is infinite, with the sum's sign; 2^127 is not."""
    w = torch.full((272, 400), 0x38, dtype=torch.uint8, device="cuda")              # 1
    L = 272 if transposed else 400
    x = torch.zeros((M, L), dtype=torch.uint8, device="cuda")
    x[:, 5] = 0x38
    x[1] ^= 0x80
    sx = torch.full((M, mm._blocks(L)), 127, dtype=torch.uint8, device="cuda")
    sx[:, 0] = 127 + 100
    for e, want in ((27, 2.0 ** 127), (28, float("inf"))):
        sw = torch.full((3, 4), 127 + e, dtype=torch.uint8, device="cuda")
        y = hcg.hc_fp8_mm(x, sx, w, sw, transposed=transposed, out_dtype=torch.float32)
        assert (y[1] == -want).all() and (y[0] == want).all() and (y[2:] == want).all()


@pytest.mark.parametrize("M", [9, 40, 300])
def test_empty_groups(M):
    """Rows of which all or some groups are empty, as the cast makes them: scale 2^-126 and codes 0."""
    g = _gen(M)
    v = torch.randn((M, 400), generator=g, device="cuda")
    v[0], v[2, 128:256], v[M - 1, :128] = 0, 0, 0
    x, sx = hcg.hc_fp8_cast(v)
    assert (sx[0] == 1).all() and sx[2, 1] == 1
    w, sw = mm._codes((272, 400), g), mm._scales((3, 4), "fp32", g)
    y = hcg.hc_fp8_mm(x, sx, w, sw, out_dtype=torch.float32)
    assert (y[0] == 0).all()
    mm._check(y, x, sx, w, sw, False)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_zero_and_the_ends(M):
    g = _gen(M)
    x, w = mm._codes((M, 400), g), mm._codes((272, 400), g)
    sx, sw = mm._scales((M, 4), "fp32", g), mm._scales((3, 4), "fp32", g)
    sx[0], sx[1, 1], sw[1, 2] = 0.0, 0.0, 0.0
    y = hcg.hc_fp8_mm(x, sx, w, sw, out_dtype=torch.float32)
    assert (y[0] == 0).all()
    _check(y, x, sx, w, sw, False)
    sx[:], sw[:] = torch.finfo(torch.float32).max, 2.0 ** -149
    _check(hcg.hc_fp8_mm(x, sx, w, sw, out_dtype=torch.float32), x, sx, w, sw, False)
