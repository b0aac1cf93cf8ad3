"""GPU: products of 8-bit numbers with scales for blocks of 128 against 64 bits.

Bounds.  Products of two codes are exact.  A block's 128 of them are added by the
tensor cores, which may cut off the last bit: at most 132 steps of 2^-23 of the sum of
their sizes; the scaled blocks are added in fp32: a half step each.  With S the
sum of all terms' sizes and B the number of blocks
    |d y| <= (half a step of y's type) |y| + (132 * 2^-23 + (B + 4) * 2^-24) S.
(A contraction that is cut adds the blocks of a slice, then the slices: no more than B
roundings.)"""
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
    yield
    assert _lib.raw("hc_consume_device_error", None) == 0


def _blocks(n):
    return -(-n // 128)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _codes(shape, g):
    """All codes but the NaNs, most of them of middling size."""
    c = (torch.randn(shape, generator=g, device="cuda") * 20).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    any_ = torch.randint(0, 127, shape, generator=g, device="cuda", dtype=torch.uint8)
    return torch.where(torch.rand(shape, generator=g, device="cuda") < 0.05, any_, c)


def _scales(shape, kind, g):
    if kind == "fp32":
        return 0.01 * torch.exp(torch.randn(shape, generator=g, device="cuda"))
    return torch.randint(115, 124, shape, generator=g, device="cuda", dtype=torch.uint8)


def _value(s):
    return s.double() if s.dtype == torch.float32 else ((s.long() + 896) << 52).view(torch.float64)


def _rows(x, sx):
    return x.view(torch.float8_e4m3fn).double() * _value(sx).repeat_interleave(128, 1)[:, :x.shape[1]]


def _matrix(w, sw):
    s = _value(sw).repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)[:, :w.shape[1]]
    return w.view(torch.float8_e4m3fn).double() * s


def _inputs(M, N, K, transposed, xs, ws, seed=0, pitch=0):
    g = _gen(seed + M + 3 * N + 7 * K)
    L = N if transposed else K
    x = torch.zeros((M, L + pitch), dtype=torch.uint8, device="cuda")
    x[:, :L] = _codes((M, L), g)
    return (x[:, :L], _scales((M, _blocks(L)), xs, g), _codes((N, K), g), _scales((_blocks(N), _blocks(K)), ws, g))


def _check(y, x, sx, w, sw, transposed):
    a, b = _rows(x.contiguous(), sx), _matrix(w, sw)
    b = b if transposed else b.t()
    want, size = a @ b, a.abs() @ b.abs()
    assert y.shape == want.shape
    room = (132 * 2.0 ** -23 + (_blocks(x.shape[1]) + 4) * U) * size
    half = torch.finfo(y.dtype).eps / 2
    tiny = torch.finfo(y.dtype).smallest_normal * half
    bad = (y.double() - want).abs() > half * (want.abs() + room) + room + tiny
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


SIZES = [(1, 16, 16), (1, 512, 1024), (2, 32, 160), (3, 48, 144), (5, 2048, 128), (8, 4096, 336), (16, 256, 2048), (17, 144, 272),
         (33, 1040, 720), (64, 528, 1040), (65, 528, 1040), (127, 128, 128), (129, 400, 656), (300, 528, 1056), (777, 1040, 720),
         (2000, 1504, 656), (2049, 1552, 1040), (256, 12288, 144), (12, 16384, 5120)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("xs,ws", [("ue8m0", "ue8m0"), ("fp32", "fp32"), ("ue8m0", "fp32")])
def test_product(M, N, K, transposed, xs, ws):
    i = _inputs(M, N, K, transposed, xs, ws)
    y = hcg.hc_fp8_mm(*i, transposed=transposed, out_dtype=torch.float32)
    _check(y, *i, transposed)
    assert torch.equal(y, hcg.hc_fp8_mm(*i, transposed=transposed, out_dtype=torch.float32))
    for t in (torch.bfloat16, torch.float16):
        assert torch.equal(hcg.hc_fp8_mm(*i, transposed=transposed, out_dtype=t), y.to(t))
    assert hcg.hc_fp8_mm(*i, transposed=transposed).dtype == torch.bfloat16


@pytest.mark.parametrize("M", list(range(1, 36)) + [47, 48, 49, 63, 96, 128, 130, 255, 257])
@pytest.mark.parametrize("transposed", [False, True])
def test_every_count_of_rows(M, transposed):
    i = _inputs(M, 320, 448, transposed, "ue8m0", "fp32")
    _check(hcg.hc_fp8_mm(*i, transposed=transposed), *i, transposed)


@pytest.mark.parametrize("M,N,K", [(3, 256, 384), (40, 272, 400), (700, 528, 1040), (2304, 1296, 144)])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("pitch,lead", [(16, 8), (48, 1), (0, 0)])
def test_strided_rows(M, N, K, transposed, pitch, lead):
    """Rows of wider buffers; the output's buffer around them stays as it is."""
    i = _inputs(M, N, K, transposed, "fp32", "ue8m0", pitch=pitch)
    C = K if transposed else N
    for t in (torch.bfloat16, torch.float32):
        buf = torch.full((M, C + lead + 3), 9.0, dtype=t, device="cuda")
        out = buf[:, lead:lead + C]
        assert hcg.hc_fp8_mm(*i, transposed=transposed, y=out) is out
        _check(out, *i, transposed)
        assert (buf[:, :lead] == 9).all() and (buf[:, lead + C:] == 9).all()


CUT = [(17, 1040, 5120), (64, 640, 4112), (129, 272, 8192), (130, 16, 16384), (300, 1296, 2576), (257, 2064, 4096)]


@pytest.mark.parametrize("M,N,K", CUT)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("t", sorted(T))
def test_cut_contraction(M, N, K, transposed, t):
    """Few tiles and a long contraction, which is cut into slices: a workspace of the very
    size, what lies behind it and around the output untouched, the same bits each time."""
    if transposed:
        N, K = K, N
    need = _lib.load().hc_fp8_mm_workspace_bytes(transposed, M, N, K)
    C = K if transposed else N
    assert need >= 2 * M * C * 4 and need % (M * C * 4) == 0
    i = _inputs(M, N, K, transposed, "fp32", "ue8m0", pitch=16)
    room = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    first = None
    for lead in (8, 1):
        buf = torch.full((M, C + 16), 9.0, dtype=T[t], device="cuda")
        y = hcg.hc_fp8_mm(*i, transposed=transposed, y=buf[:, lead:lead + C], workspace=room[:need])
        _check(y, *i, transposed)
        assert (buf[:, :lead] == 9).all() and (buf[:, lead + C:] == 9).all() and (room[need:] == 255).all()
        assert first is None or torch.equal(first, y)
        first = y.clone()
        room[:need] = 255
    assert torch.equal(first, hcg.hc_fp8_mm(*i, transposed=transposed, out_dtype=T[t]))
    with pytest.raises(RuntimeError):
        hcg.hc_fp8_mm(*i, transposed=transposed, workspace=room[:need - 1])


def test_cut_contractions_share_a_workspace():
    """Graphs of products of one workspace, replayed in turn on one stream; NaN codes."""
    a, b = _inputs(64, 640, 4112, False, "ue8m0", "fp32"), _inputs(33, 272, 8192, False, "fp32", "fp32", seed=5)
    want = [hcg.hc_fp8_mm(*i) for i in (a, b)]
    room = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.empty_like(w) for w in want], []
    for i, o in zip((a, b), outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            hcg.hc_fp8_mm(*i, y=o, workspace=room)
    for _ in range(20):
        for o, g in zip(outs, graphs):
            o.fill_(7)
            g.replay()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    x, sx, w, sw = a
    y = hcg.hc_fp8_mm(_put(x, (2, 4100), 0x7f), sx, w, sw)
    assert y[2].isnan().all() and torch.equal(y[:2], want[0][:2]) and torch.equal(y[3:], want[0][3:])


@pytest.mark.parametrize("M", [3, 16, 40])
@pytest.mark.parametrize("transposed", [False, True])
def test_offsets_past_32_bits(M, transposed):
    """The last columns of products with a matrix of 65,552 x 65,536 codes."""
    N, K = 65552, 65536
    g = _gen(M)
    w = torch.randint(0, 120, (N, K), generator=g, dtype=torch.uint8, device="cuda")
    C, L = (K, N) if transposed else (N, K)
    x, sx = _codes((M, L), g), _scales((M, _blocks(L)), "ue8m0", g)
    sw = _scales((_blocks(N), _blocks(K)), "fp32", g)
    y = hcg.hc_fp8_mm(x, sx, w, sw, transposed=transposed)
    assert y.shape == (M, C)
    for c in (0, C // 256 * 128, (C - 1) // 128 * 128):
        part = w[:, c:c + 128] if transposed else w[c:c + 128]
        s = sw[:, c // 128:c // 128 + 1] if transposed else sw[c // 128:c // 128 + 1]
        _check(y[:, c:c + 128], x, sx, part.contiguous(), s.contiguous(), transposed)


def test_nan_codes_and_scales():
    """A NaN among the codes or scales spoils what it goes into, nothing else."""
    for M in (4, 300):
        x, sx, w, sw = _inputs(M, 272, 400, False, "ue8m0", "ue8m0")
        clean = hcg.hc_fp8_mm(x, sx, w, sw)
        for code in (0x7f, 0xff):
            y = hcg.hc_fp8_mm(_put(x, (2, 130), code), sx, w, sw)
            assert y[2].isnan().all() and torch.equal(y[:2], clean[:2]) and torch.equal(y[3:], clean[3:])
            y = hcg.hc_fp8_mm(x, sx, _put(w, (200, 399), code), sw)
            assert y[:, 200].isnan().all() and torch.equal(y[:, :200], clean[:, :200]) and torch.equal(y[:, 201:], clean[:, 201:])
        y = hcg.hc_fp8_mm(x, _put(sx, (1, 2), 255), w, sw)
        assert y[1].isnan().all() and torch.equal(y[2:], clean[2:])
        y = hcg.hc_fp8_mm(x, sx, w, _put(sw, (1, 3), 255))
        assert y[:, 128:256].isnan().all() and torch.equal(y[:, :128], clean[:, :128]) and torch.equal(y[:, 256:], clean[:, 256:])
        y = hcg.hc_fp8_mm(x, _put(sx, (1, 2), 0), w, sw, out_dtype=torch.float32)     # 2^-127, subnormal
        _check(y, x, _put(sx, (1, 2), 0), w, sw, False)


def _put(t, at, v):
    t = t.clone()
    t[at] = v
    return t


def test_no_rows():
    x, sx, w, sw = _inputs(4, 32, 64, False, "fp32", "fp32")
    assert hcg.hc_fp8_mm(x[:0], sx[:0], w, sw).shape == (0, 32)


def test_binding_shapes():
    x, sx, w, sw = _inputs(4, 32, 160, False, "fp32", "fp32")
    with pytest.raises(ValueError, match="x has shape"):
        hcg.hc_fp8_mm(x, sx, w, sw, transposed=True)
    with pytest.raises(ValueError, match="x_scales has shape"):
        hcg.hc_fp8_mm(x, sx[:, :1], w, sw)
    with pytest.raises(ValueError, match="w_scales has shape"):
        hcg.hc_fp8_mm(x, sx, w, sw.t().contiguous())
    with pytest.raises(TypeError, match="out_dtype"):
        hcg.hc_fp8_mm(x, sx, w, sw, out_dtype=torch.float64)
    with pytest.raises(TypeError, match="x_scales must be"):
        hcg.hc_fp8_mm(x, sx.half(), w, sw)


def test_gradient_against_differences():
    """x -> y = x w^T of exact numbers: the transposed product of the output's gradient is
    the gradient along any direction.  Codes of whole numbers up to 8 and scales of 1,
    so that all sums are exact."""
    g = _gen(5)
    whole = lambda *s: torch.randint(-8, 9, s, generator=g, device="cuda").float()
    one = lambda *s: torch.full(s, 127, dtype=torch.uint8, device="cuda")
    code = lambda v: v.to(torch.float8_e4m3fn).view(torch.uint8)
    x, dx, w, gy = whole(20, 256), whole(20, 256), whole(144, 256), whole(20, 144)
    loss = lambda v: (hcg.hc_fp8_mm(code(v), one(20, 2), code(w), one(2, 2), out_dtype=torch.float32).double() * gy.double()).sum()
    gx = hcg.hc_fp8_mm(code(gy), one(20, 2), code(w), one(2, 2), transposed=True, out_dtype=torch.float32)
    # (codes of 0 to 16 are exact for whole numbers, so is the difference of a step of 1)
    assert loss(x + dx) - loss(x) == (gx.double() * dx.double()).sum()


@pytest.mark.parametrize("M", [4, 100, 2500])
def test_streams_and_graph(M):
    """On a stream of its own, and captured and replayed on new inputs."""
    x, sx, w, sw = _inputs(M, 1296, 656, False, "ue8m0", "ue8m0")
    want = hcg.hc_fp8_mm(x, sx, w, sw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = hcg.hc_fp8_mm(x, sx, w, sw, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
    x2 = _inputs(M, 1296, 656, False, "ue8m0", "ue8m0", seed=3)
    static = [t.clone() for t in (x, sx)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = hcg.hc_fp8_mm(*static, w, sw)
    graph.replay()
    assert torch.equal(out, want)
    for s, t in zip(static, x2):
        s.copy_(t)
    graph.replay()
    assert torch.equal(out, hcg.hc_fp8_mm(x2[0], x2[1], w, sw))
