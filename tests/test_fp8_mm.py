"""Products of 8-bit numbers on the host: refusals of the C entry point (before any
CUDA call; the pointers are not allocations) and of the binding."""
import pytest
import torch

import hyper_connection_residual_mixes_gb300 as hcg
from hyper_connection_residual_mixes_gb300 import _lib
from hyper_connection_residual_mixes_gb300 import build as hc_build

F32, BF16, F16, UE8M0 = 0, 1, 2, 3
A, STEP = 0x1000000, 0x10000000


@pytest.fixture(scope="module", autouse=True)
def _built():
    hc_build.build()


def _mm(**kw):
    a = dict(x=A, xs=64, sx=A + STEP, xt=UE8M0, w=A + 2 * STEP, sw=A + 3 * STEP, wt=F32, transposed=0, M=100, N=32, K=64,
             y=A + 4 * STEP, ys=32, yt=BF16, ws=A + 5 * STEP, ws_bytes=1 << 24, stream=None)
    a.update(kw)
    return _lib.raw("hc_fp8_mm", *a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(M=-1), 1), (dict(N=0), 1), (dict(K=-16), 1), (dict(xt=BF16), 1), (dict(wt=4), 1), (dict(yt=UE8M0), 1), (dict(yt=-1), 1),
    (dict(N=24), 2), (dict(K=72, xs=80), 2), (dict(M=1 << 31), 2), (dict(M=(1 << 31) - 1), 2), (dict(xs=72), 2), (dict(xs=1 << 38), 2),
    (dict(N=(1 << 31) - 16, ys=1 << 31), 2), (dict(N=1 << 30, K=1 << 30, xs=1 << 30, ys=1 << 30), 2),
    (dict(xs=48), 1), (dict(ys=31), 1), (dict(transposed=1), 1), (dict(transposed=1, xs=32), 1),
    (dict(x=None), 1), (dict(sx=None), 1), (dict(w=None), 1), (dict(sw=None), 1), (dict(y=None), 1),
    (dict(x=A + 8), 3), (dict(w=A + 2 * STEP + 4), 3), (dict(sw=A + 3 * STEP + 2), 3), (dict(xt=F32, sx=A + STEP + 1), 3),
    (dict(y=A + 4 * STEP + 1), 3), (dict(yt=F32, y=A + 4 * STEP + 2), 3),
    (dict(y=A + 64), 4), (dict(y=A + STEP), 4), (dict(y=A + 2 * STEP + 64), 4), (dict(y=A + 3 * STEP), 4),
    (dict(M=0), 0), (dict(M=0, x=None, y=None), 0),
])
def test_refusals(kw, expect):
    assert _mm(**kw) == expect


def test_workspace_bytes():
    f = _lib.load().hc_fp8_mm_workspace_bytes
    assert f(0, 0, 64, 64) == 0 and f(0, -1, 64, 64) == 0 and f(0, 4, 60, 64) == 0 and f(1, 4, 64, 0) == 0
    for t in (0, 1):
        for M in (1, 40, 1000, 100000):
            for N, K in ((16, 16), (272, 1040), (2048, 5120)):
                assert f(t, M, N, K) >= 0
    assert f(0, 100, 32, 64) == 0 and f(0, 16, 272, 8192) == 0    # one block; few rows
    # sums by slice, 2 to 32 of them, of the output's size; none where the tiles fill the SMs
    for t, N, K in ((0, 272, 8192), (1, 8192, 272), (0, 16, 65536), (0, 5120, 5120)):
        for M in (17, 130):
            n, rest = divmod(f(t, M, N, K), M * (K if t else N) * 4)
            assert rest == 0 and 2 <= n <= 32, (t, M, N, K, n)
        assert f(t, 100000, N, K) == 0
    for M in (17, 130, 1000, 5000, (1 << 31) - 4097):
        for N, K in ((16, 16), (144, 5120), (4096, 65536), (65536, 4096)):
            assert f(0, M, N, K) <= 152 * 128 * 256 * 4
            assert f(1, M, K, N) == f(0, M, N, K) or M <= 16


def test_workspace_refusals():
    need = _lib.load().hc_fp8_mm_workspace_bytes(0, 100, 32, 4096)
    cut = dict(K=4096, xs=4096)
    assert need > 0
    assert _mm(**cut, ws=None) == 1 and _mm(**cut, ws_bytes=need - 1) == 1
    assert _mm(**cut, ws=A + 5 * STEP + 8) == 3
    assert _mm(**cut, ws=A) == 4 and _mm(**cut, ws=A + 4 * STEP) == 4


def test_binding_refusals():
    x, w = torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((32, 64), dtype=torch.uint8)
    s = torch.zeros((4, 1), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        hcg.hc_fp8_mm(x, s, w, s)
    with pytest.raises(TypeError, match="uint8"):
        hcg.hc_fp8_mm(x.float(), s, w, s)
