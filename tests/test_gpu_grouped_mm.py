"""GPU: the experts' products and their gradients against 64 bits.

Bounds.  Products of 16-bit values are exact in fp32.  The tensor cores add 16
of them to the accumulator at a time and may cut the sum off at the last bit
of its largest term: each of the K / 16 additions is off by at most 2^-22 of
the sum of the terms' sizes S = sum |x w|.  So |d y| <= (K / 16 + 2) 2^-22 S
before the one rounding, half a step of the output's type."""
import pytest
import torch

import hyper_connection_residual_mixes_gb300 as hcg
from hyper_connection_residual_mixes_gb300 import _lib
from hyper_connection_residual_mixes_gb300 import build as hc_build

pytestmark = pytest.mark.gpu

T = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hc_build.build()
    _lib.load()


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert _lib.raw("hc_consume_device_error", None) == 0


def _offsets(counts, lead=0):
    o = [lead]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device="cuda")


def _inputs(counts, N, K, t, kn=False, lead=0, rest=0, seed=0, pitch=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + 31 * N + K)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").to(T[t])
    n, E = lead + sum(counts) + rest, len(counts)
    x, g = r(n, K + pitch)[:, :K], r(n, N + pitch)[:, :N]
    return x, r(E, K, N) if kn else r(E, N, K), g, _offsets(counts, lead)


def _close(got, want, size, terms):
    half = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * half
    room = (terms / 16 + 2) * 2.0 ** -22 * size
    assert ((got.double() - want).abs() <= room + half * (want.abs() + room) + tiny).all()


def _check(x, w, off, kn, y, rows=None):
    """y of every expert's rows; returns a mask of the rows of no expert."""
    o, free = off.tolist(), torch.ones((x.shape[0],), dtype=torch.bool, device="cuda")
    for e in range(w.shape[0]):
        a, b = o[e], o[e + 1]
        free[a:b] = False
        if b > a:
            xe, we = x[a:b].double(), w[e].double() if kn else w[e].double().t()
            _close(y[a:b], xe @ we, xe.abs() @ we.abs(), x.shape[1])
    return free


def _check_weights(g, x, off, kn, g_w):
    o = off.tolist()
    for e in range(len(o) - 1):
        ge, xe = g[o[e]:o[e + 1]].double(), x[o[e]:o[e + 1]].double()
        a, b = (xe, ge) if kn else (ge, xe)
        if o[e + 1] == o[e]:
            assert (g_w[e] == 0).all()
        else:
            _close(g_w[e], a.t() @ b, a.abs().t() @ b.abs(), o[e + 1] - o[e])


COUNTS = {"one_row": [1], "token": [1, 0, 1, 1, 0, 0, 2, 1], "few": [3, 0, 17, 31, 32, 33, 1], "one_expert": [257],
          "ragged": [100, 0, 255, 256, 257, 0, 1, 300, 64], "tail16": [16, 15, 48, 63, 65, 127, 129], "empty": [0, 0, 0]}


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("N,K", [(8, 8), (128, 64), (136, 200), (264, 72), (512, 1024), (1000, 520)])
@pytest.mark.parametrize("t,kn", [("bf16", False), ("fp16", True)])
def test_product_and_gradients(counts, N, K, t, kn):
    x, w, g, off = _inputs(COUNTS[counts], N, K, t, kn, rest=3)
    y = hcg.hc_grouped_mm(x, w, off, transposed=kn)
    free = _check(x, w, off, kn, y)
    assert (y[free] == 0).all()
    got = hcg.hc_grouped_mm_backward(g, x, w, off, transposed=kn)
    free = _check(g, w, off, not kn, got["g_x"])
    assert (got["g_x"][free] == 0).all() and got["g_w"].shape == w.shape
    _check_weights(g, x, off, kn, got["g_w"])


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("kn", [False, True])
def test_fp32_outputs(t, kn):
    x, w, g, off = _inputs([70, 0, 130, 5], 200, 328, t, kn, seed=1)
    y = hcg.hc_grouped_mm(x, w, off, transposed=kn, out_dtype=torch.float32)
    assert y.dtype == torch.float32
    _check(x, w, off, kn, y)
    g_w = hcg.hc_grouped_mm_weights(g, x, off, transposed=kn, out_dtype=torch.float32)
    assert g_w.dtype == torch.float32
    _check_weights(g, x, off, kn, g_w)
    assert torch.equal(g_w.to(T[t]), hcg.hc_grouped_mm_weights(g, x, off, transposed=kn))


def test_many_experts_and_long_contractions():
    gen = torch.Generator(device="cuda").manual_seed(4)
    counts = torch.randint(0, 9, (1024,), generator=gen, device="cuda").tolist()
    x, w, g, off = _inputs(counts, 16, 24, "bf16")
    y = hcg.hc_grouped_mm(x, w, off)
    _check(x, w, off, False, y)
    _check_weights(g, x, off, False, hcg.hc_grouped_mm_weights(g, x, off))
    x, w, g, off = _inputs([5, 700, 2000], 320, 5120, "bf16")
    _check(x, w, off, False, hcg.hc_grouped_mm(x, w, off))
    got = hcg.hc_grouped_mm_backward(g, x, w, off)
    _check(g, w, off, True, got["g_x"])
    _check_weights(g, x, off, False, got["g_w"])


@pytest.mark.parametrize("counts,N,K", [([5000], 16, 216), ([4097], 264, 1032), ([1, 0, 20000, 77, 130], 520, 72),
                                        ([2100, 2300, 2200], 2048, 256), ([0, 9000, 600], 8, 8), ([40000], 512, 328)])
@pytest.mark.parametrize("t,kn", [("bf16", False), ("fp16", True)])
def test_gradients_of_few_and_long_experts(counts, N, K, t, kn):
    """Rows summed in slices: some of them empty, some ending inside a block; NaN in
    the rows of no expert; outputs at odd places; every repeat gives the same bits."""
    assert _lib.load().hc_grouped_mm_weights_workspace_bytes(sum(counts) + 3, len(counts), N, K) > 0
    x, _, g, off = _inputs(counts, N, K, t, kn, rest=3, seed=11)
    x[sum(counts):], g[sum(counts):] = float("nan"), float("inf")
    got = hcg.hc_grouped_mm_weights(g, x, off, transposed=kn)
    _check_weights(g, x, off, kn, got)
    f32 = hcg.hc_grouped_mm_weights(g, x, off, transposed=kn, out_dtype=torch.float32)
    _check_weights(g, x, off, kn, f32)
    assert torch.equal(f32.to(T[t]), got)
    for out in (T[t], torch.float32):
        flat = torch.full((got.numel() + 2,), 5.0, dtype=out, device="cuda")
        odd = flat[1:-1].view(got.shape)
        hcg.hc_grouped_mm_weights(g, x, off, transposed=kn, g_w=odd)
        assert torch.equal(odd, got if out is T[t] else f32) and flat[0] == 5 and flat[-1] == 5
    for _ in range(10):
        assert torch.equal(hcg.hc_grouped_mm_weights(g, x, off, transposed=kn), got)


@pytest.mark.parametrize("counts,N,K", [([1], 8, 8200), ([3], 3776, 5936), ([2, 0, 5, 40, 1], 264, 9000), ([700], 136, 16384),
                                        ([0, 300, 1], 8, 5568), ([20, 1, 33], 1032, 4160)])
@pytest.mark.parametrize("t,kn", [("bf16", False), ("fp16", True)])
def test_products_of_few_tiles_and_long_sums(counts, N, K, t, kn):
    """Contractions in slices, the last of them shorter or empty; rows of no expert
    before and behind stay, or become zeros; strided and oddly placed outputs."""
    x, w, _, off = _inputs(counts, N, K, t, kn, rest=3, seed=14)
    assert _lib.load().hc_grouped_mm_workspace_bytes(x.shape[0], len(counts), N, K) > 0
    off = off.clone()
    off[0] = min(1, counts[0])   # a first row of no expert, where there is one to take
    x[sum(counts):] = float("nan")
    y = hcg.hc_grouped_mm(x, w, off, transposed=kn)
    free = _check(x, w, off, kn, y)
    assert (y[free] == 0).all()
    f32 = hcg.hc_grouped_mm(x, w, off, transposed=kn, out_dtype=torch.float32)
    _check(x, w, off, kn, f32)
    assert torch.equal(f32.to(T[t]), y)
    for out in (T[t], torch.float32):
        for pitch, lead in ((0, 1), (5, 3), (8, 0)):
            flat = torch.full((lead + x.shape[0] * (N + pitch) + 1,), 5.0, dtype=out, device="cuda")
            rows = flat[lead:-1].view(x.shape[0], N + pitch)
            hcg.hc_grouped_mm(x, w, off, transposed=kn, y=rows[:, :N])
            want = (y if out is T[t] else f32).clone()
            want[free] = 5.0
            assert torch.equal(rows[:, :N], want) and (rows[:, N:] == 5).all() and (flat[:lead] == 5).all() and flat[-1] == 5
    for _ in range(10):
        assert torch.equal(hcg.hc_grouped_mm(x, w, off, transposed=kn), y)


def test_bad_offsets_with_slices():
    x, w, _, off = _inputs([4, 4, 4], 64, 8192, "bf16", seed=15)
    _lib.raw("hc_consume_device_error", None)
    bad = torch.tensor([0, 40, 8, 12], dtype=torch.int32, device="cuda")
    y = torch.full((12, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    hcg.hc_grouped_mm(x, w, bad, y=y)
    assert _lib.raw("hc_consume_device_error", None) == 1 and _lib.raw("hc_consume_device_error", None) == 0
    assert (y[:8] == 3).all() and torch.equal(y[8:], hcg.hc_grouped_mm(x, w, off)[8:])


def test_slices_on_two_streams_and_in_a_graph():
    """Calls with workspaces of their own at once; a captured call reads new offsets."""
    x, _, g, off = _inputs([3000, 2500], 264, 136, "bf16", seed=12)
    x2, _, g2, off2 = _inputs([2500, 3000], 264, 136, "bf16", seed=13)
    want, want2 = hcg.hc_grouped_mm_weights(g, x, off), hcg.hc_grouped_mm_weights(g2, x2, off2)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(a):
            got = hcg.hc_grouped_mm_weights(g, x, off)
        with torch.cuda.stream(b):
            got2 = hcg.hc_grouped_mm_weights(g2, x2, off2)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(got2, want2)
    size = _lib.load().hc_grouped_mm_weights_workspace_bytes(5500, 2, 264, 136)
    ws, out = torch.empty((size,), dtype=torch.uint8, device="cuda"), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hcg.hc_grouped_mm_weights(g, x, off, g_w=out, workspace=ws)
        hcg.hc_grouped_mm_weights(g, x, off, g_w=out, workspace=ws)
    off.copy_(off2)
    graph.replay()
    torch.cuda.synchronize()
    _check_weights(g, x, off2, False, out)
    with pytest.raises(_lib.HcError):
        hcg.hc_grouped_mm_weights(g, x, off, workspace=ws[:-16])


@pytest.mark.parametrize("kn", [False, True])
def test_narrow_and_wide_tiles_in_turn(kn):
    """Experts of a few rows between experts of many: tiles of different widths
    follow one another through the same stages.  Every repeat gives the same bits."""
    counts = [5, 700, 3, 260, 9, 600, 1, 40, 500]
    x, w, g, off = _inputs(counts, 1536, 320, "bf16", kn, seed=9)
    y, got = hcg.hc_grouped_mm(x, w, off, transposed=kn), hcg.hc_grouped_mm_backward(g, x, w, off, transposed=kn)
    _check(x, w, off, kn, y)
    _check(g, w, off, not kn, got["g_x"])
    _check_weights(g, x, off, kn, got["g_w"])
    for _ in range(20):
        assert torch.equal(hcg.hc_grouped_mm(x, w, off, transposed=kn), y)
        again = hcg.hc_grouped_mm_backward(g, x, w, off, transposed=kn)
        assert torch.equal(again["g_x"], got["g_x"]) and torch.equal(again["g_w"], got["g_w"])


@pytest.mark.parametrize("pitch", [8, 56])
def test_strides_and_rows_of_no_expert(pitch):
    """Inputs cut out of wider rows; rows before the first and behind the last
    expert's, and the columns around y, stay as they were."""
    counts, N, K = [20, 0, 75, 3], 72, 104
    x, w, g, off = _inputs(counts, N, K, "bf16", lead=5, rest=9, pitch=pitch)
    buf = torch.full((x.shape[0], N + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    y = buf[:, 1:1 + N]
    assert hcg.hc_grouped_mm(x, w, off, y=y) is y
    free = _check(x, w, off, False, y)
    assert free.sum() == 14 and (buf[free] == 7).all() and (buf[:, 0] == 7).all() and (buf[:, 1 + N:] == 7).all()
    assert torch.equal(hcg.hc_grouped_mm(x, w, off)[~free], y[~free])
    _check_weights(g, x, off, False, hcg.hc_grouped_mm_weights(g, x, off))


def test_other_experts_values_do_not_leak():
    """NaN and infinities in the neighbours' rows, behind the last row and in the
    neighbours' weights stay out of an expert's results."""
    counts, N, K = [30, 41, 77], 136, 72
    x, w, g, off = _inputs(counts, N, K, "bf16", rest=20)
    y, g_w = hcg.hc_grouped_mm(x, w, off), hcg.hc_grouped_mm_weights(g, x, off)
    x2, g2, w2 = x.clone(), g.clone(), w.clone()
    x2[:30], x2[71:], g2[:30], g2[71:] = float("nan"), float("inf"), float("inf"), float("nan")
    w2[0], w2[2] = float("nan"), float("inf")
    assert torch.equal(hcg.hc_grouped_mm(x2, w2, off)[30:71], y[30:71])
    assert torch.equal(hcg.hc_grouped_mm_weights(g2, x2, off)[1], g_w[1])


def test_gradients_against_differences():
    """The product is linear in x and in w: its difference along a direction is
    the product with the direction, whose sum with g_y is the gradient's with
    the direction, up to both sides' own bounds."""
    counts, N, K = [13, 0, 40], 48, 56
    x, w, g, off = _inputs(counts, N, K, "bf16", seed=2)
    got = hcg.hc_grouped_mm_backward(g, x, w, off)
    vx, vw, _, _ = _inputs(counts, N, K, "bf16", seed=3)
    gd = g.double()
    for v, y, size, grad in ((vx, hcg.hc_grouped_mm(vx, w, off, out_dtype=torch.float32), hcg.hc_grouped_mm(vx.abs(), w.abs(), off), got["g_x"]),
                             (vw, hcg.hc_grouped_mm(x, vw, off, out_dtype=torch.float32), hcg.hc_grouped_mm(x.abs(), vw.abs(), off), got["g_w"])):
        room = float((gd.abs() * size.double()).sum()) * (N / 16 + K / 16 + 4) * 2.0 ** -22
        room += float((grad.double().abs() * v.double().abs()).sum()) * 2.0 ** -8
        assert abs(float((gd * y.double()).sum() - (grad.double() * v.double()).sum())) <= room


def test_bad_offsets_are_reported():
    x, w, g, _ = _inputs([50, 50], 64, 64, "bf16")
    for bad in ([0, 60, 101], [0, -5, 100], [-1, 50, 100], [0, 70, 60], [1 << 30, 1 << 30, 1 << 30]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        y = torch.full((100, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        hcg.hc_grouped_mm(x, w, off, y=y)
        assert _lib.raw("hc_consume_device_error", None) == 1, bad
        hcg.hc_grouped_mm_weights(g, x, off)
        assert _lib.raw("hc_consume_device_error", None) == 1, bad
    y = hcg.hc_grouped_mm(x, w, _offsets([50, 50]))
    _check(x, w, _offsets([50, 50]), False, y)


def test_no_rows():
    x, w, g, off = _inputs([0, 0], 64, 32, "bf16")
    assert hcg.hc_grouped_mm(x, w, off).shape == (0, 64)
    got = hcg.hc_grouped_mm_backward(g, x, w, off)
    assert got["g_x"].shape == (0, 32) and (got["g_w"] == 0).all() and got["g_w"].shape == w.shape


def test_other_stream_and_graph():
    """Captured once; replays follow new rows and new offsets."""
    N, K = 264, 200
    x, w, g, off = _inputs([40, 300, 0, 10], N, K, "bf16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = hcg.hc_grouped_mm(x, w, off, stream=s)
    s.synchronize()
    assert torch.equal(y, hcg.hc_grouped_mm(x, w, off))
    hcg.hc_grouped_mm_backward(g, x, w, off)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cy = hcg.hc_grouped_mm(x, w, off)
        cg = hcg.hc_grouped_mm_backward(g, x, w, off)
    for counts in ([40, 300, 0, 10], [0, 0, 350, 0], [100, 1, 1, 17]):
        x2, _, g2, _ = _inputs([350], N, K, "bf16", seed=sum(counts) + counts[0])
        x.copy_(x2), g.copy_(g2), off.copy_(_offsets(counts))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cy, hcg.hc_grouped_mm(x, w, off))
        want = hcg.hc_grouped_mm_backward(g, x, w, off)
        assert all(torch.equal(cg[k], want[k]) for k in want)


def test_two_streams_at_once():
    """Two calls in flight on two streams keep to themselves."""
    a, b = _inputs([700, 300], 512, 1024, "bf16", seed=5), _inputs([10, 900, 90], 1024, 512, "bf16", seed=6)
    want = [hcg.hc_grouped_mm(c[0], c[1], c[3]) for c in (a, b)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[hcg.hc_grouped_mm(c[0], c[1], c[3], stream=st) for c, st in zip((a, b), s)] for _ in range(10)]
    torch.cuda.synchronize()
    for pair in got:
        assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])


def test_offsets_beyond_32_bits():
    """Outputs past 2^31 elements."""
    n, N, K = 300_000, 8192, 8
    x, w, g, off = _inputs([n - 1, 1], N, K, "bf16")
    y = hcg.hc_grouped_mm(x, w, off)
    for a, e in ((n - 3, 0), (n - 1, 1), (262_143, 0), (262_144, 0)):
        b = a + 1
        xe, we = x[a:b].double(), w[e].double().t()
        _close(y[a:b], xe @ we, xe.abs() @ we.abs(), K)


@pytest.mark.parametrize("K,N", [(64, 72), (8192, 64)])
@pytest.mark.parametrize("bad,taken", [([0, 60, 20, 100, 100], {0}), ([0, 50, 100, 0, 100], {0, 1}), ([90, 10, 40, 30, 100], {1}),
                                       ([0, 120, 30, 80, 60], {2}), ([0, 100] * 8 + [0, 100], {0}), ([0, 1, 0, 2, 0, 3, 2, 5], {0, 6})])
def test_ranges_that_share_rows(K, N, bad, taken):
    """A range that begins before an earlier one's end counts as empty: every row has
    one expert, also where others' ranges are out of order (K = 8,192: in slices)."""
    x, w, _, _ = _inputs([100] + [0] * (len(bad) - 2), N, K, "bf16", seed=17)
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    _lib.raw("hc_consume_device_error", None)
    y = torch.full((100, N), 3.0, dtype=torch.bfloat16, device="cuda")
    hcg.hc_grouped_mm(x, w, off, y=y)
    assert _lib.raw("hc_consume_device_error", None) == 1
    free = torch.ones((100,), dtype=torch.bool, device="cuda")
    for e in taken:
        a, b = bad[e], bad[e + 1]
        free[a:b] = False
        xe, we = x[a:b].double(), w[e].double().t()
        _close(y[a:b], xe @ we, xe.abs() @ we.abs(), K)
    assert (y[free] == 3).all()


@pytest.mark.parametrize("scale", [1, 90])
def test_gradients_of_ranges_that_share_rows(scale):
    """The weights' gradient likewise, with 9,000 rows in slices."""
    n = 100 * scale
    x, _, g, _ = _inputs([n, 0, 0], 72, 64, "bf16", seed=18)
    assert (_lib.load().hc_grouped_mm_weights_workspace_bytes(n, 3, 72, 64) > 0) == (scale > 1)
    bad = [b * scale for b in (0, 60, 20, 100)]
    _lib.raw("hc_consume_device_error", None)
    got = hcg.hc_grouped_mm_weights(g, x, torch.tensor(bad, dtype=torch.int32, device="cuda"))
    assert _lib.raw("hc_consume_device_error", None) == 1
    _check_weights(g, x, torch.tensor([0, 60 * scale, 60 * scale, 60 * scale], device="cuda"), False, got)


@pytest.mark.parametrize("K,N", [(64, 72), (8192, 64)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad,taken", [([0, 60, 101], {0}), ([0, -5, 100], set()), ([0, 70, 60], {0}), ([5, 30, 130, 60, 90], {0, 3}),
                                       ([-1, 20, 100], {1}), ([100, 0, 0, 0], set())])
def test_rows_of_refused_ranges_are_zeros(K, N, out, bad, taken):
    """In a y made by the call; in one that is given they stay.  With K = 8,192 the
    contraction is summed in slices."""
    x, w, _, _ = _inputs([100] + [0] * (len(bad) - 2), N, K, "bf16", seed=16)
    sliced = _lib.load().hc_grouped_mm_workspace_bytes(100, len(bad) - 1, N, K) > 0
    assert sliced == (K == 8192)
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    _lib.raw("hc_consume_device_error", None)
    for _ in range(3):
        torch.full((100, N), 7.0, dtype=out, device="cuda")   # what the next allocation of this size holds
        y = hcg.hc_grouped_mm(x, w, off, out_dtype=out)
        given = torch.full((100, N), 3.0, dtype=out, device="cuda")
        hcg.hc_grouped_mm(x, w, off, y=given)
        assert _lib.raw("hc_consume_device_error", None) == 1
        free = torch.ones((100,), dtype=torch.bool, device="cuda")
        for e in taken:
            a, b = bad[e], bad[e + 1]
            free[a:b] = False
            xe, we = x[a:b].double(), w[e].double().t()
            _close(y[a:b], xe @ we, xe.abs() @ we.abs(), K)
        assert (y[free] == 0).all() and (given[free] == 3).all() and torch.equal(given[~free], y[~free])
