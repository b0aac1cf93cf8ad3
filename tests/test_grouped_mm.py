"""The experts' products on the host: refusals of the C entry points (before any
CUDA call; the pointers are not allocations) and of the binding."""
import pytest
import torch

import hyper_connection_residual_mixes_gb300 as hcg
from hyper_connection_residual_mixes_gb300 import _lib
from hyper_connection_residual_mixes_gb300 import build as hc_build

F32, BF16, F16 = 0, 1, 2
A, STEP = 0x1000000, 0x10000000


@pytest.fixture(scope="module", autouse=True)
def _built():
    hc_build.build()


def _mm(**kw):
    a = dict(x=A, xs=64, w=A + STEP, transposed=0, offsets=A + 2 * STEP, n=16, experts=4, N=32, K=64, type=BF16,
             y=A + 3 * STEP, ys=32, yt=BF16, zero=0, ws=None, ws_bytes=0, stream=None)
    a.update(kw)
    return _lib.raw("hc_grouped_mm", *a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(n=-1), 1), (dict(experts=0), 1), (dict(N=0), 1), (dict(K=-8), 1), (dict(type=5), 1), (dict(yt=-1), 1),
    (dict(type=F32, yt=F32), 2), (dict(type=F16), 2), (dict(experts=1025), 2), (dict(N=33, ys=40), 2), (dict(K=63), 2),
    (dict(n=1 << 31), 2), (dict(n=(1 << 31) - 1), 2), (dict(xs=68), 2), (dict(xs=1 << 38), 2), (dict(N=1 << 30, K=1 << 30, xs=1 << 30, ys=1 << 30), 2),
    (dict(n=1, experts=1, N=(1 << 31) - 8, K=8, xs=8, ys=(1 << 31) - 8), 2),
    (dict(n=1, experts=1, N=8, K=(1 << 31) - 8, xs=(1 << 31) - 8, ys=8), 2),
    (dict(xs=56), 1), (dict(ys=31), 1), (dict(x=None), 1), (dict(w=None), 1), (dict(offsets=None), 1), (dict(y=None), 1),
    (dict(x=A + 8), 3), (dict(w=A + STEP + 2), 3), (dict(offsets=A + 2 * STEP + 2), 3), (dict(y=A + 3 * STEP + 1), 3),
    (dict(yt=F32, y=A + 3 * STEP + 2), 3),
    (dict(y=A + 64), 4), (dict(y=A + STEP + 100), 4), (dict(y=A + 2 * STEP + 16), 4),
    (dict(n=0), 0), (dict(n=0, x=None, y=None), 0),
    # a contraction of 8,192 in slices, which need room
    (dict(K=8192, xs=8192), 1), (dict(K=8192, xs=8192, ws=A + 4 * STEP, ws_bytes=16 * 32 * 4), 1),
    (dict(K=8192, xs=8192, ws=A + 4 * STEP + 8, ws_bytes=1 << 24), 3),
    (dict(K=8192, xs=8192, ws=A + 64, ws_bytes=1 << 24), 4),
    (dict(K=8192, xs=8192, ws=A + 3 * STEP + 512, ws_bytes=1 << 24), 4),
])
def test_product_refusals(kw, expect):
    assert _mm(**kw) == expect


def _weights(**kw):
    a = dict(g=A, gs=32, x=A + STEP, xs=64, offsets=A + 2 * STEP, n=16, experts=4, N=32, K=64, type=F16, gw=A + 3 * STEP,
             transposed=0, gt=F32, ws=None, ws_bytes=0, stream=None)
    a.update(kw)
    return _lib.raw("hc_grouped_mm_weights", *a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(n=-1), 1), (dict(experts=-3), 1), (dict(gt=9), 1), (dict(gt=BF16), 2), (dict(type=F32), 2), (dict(N=36, gs=40), 2),
    (dict(n=1, experts=1, N=(1 << 31) - 8, K=8, gs=(1 << 31) - 8, xs=8), 2),
    (dict(gs=24), 1), (dict(gs=36), 2), (dict(xs=65), 2), (dict(g=None), 1), (dict(gw=None), 1), (dict(offsets=None), 1),
    (dict(g=A + 2), 3), (dict(x=A + STEP + 8), 3), (dict(gw=A + 3 * STEP + 2), 3),
    (dict(gw=A + 32), 4), (dict(gw=A + 2 * STEP), 4),
    # one expert of 8,192 rows: 32 x 64 sums in slices, which need room
    (dict(n=8192, experts=1), 1), (dict(n=8192, experts=1, ws=A + 4 * STEP, ws_bytes=32 * 64 * 8 - 1), 1),
    (dict(n=8192, experts=1, ws=A + 4 * STEP + 8, ws_bytes=1 << 24), 3),
    (dict(n=8192, experts=1, ws=A + 64, ws_bytes=1 << 24), 4),
    (dict(n=8192, experts=1, ws=A + 3 * STEP + 4096, ws_bytes=1 << 24), 4),
])
def test_weights_refusals(kw, expect):
    assert _weights(**kw) == expect


def test_workspace_bytes():
    f = _lib.load().hc_grouped_mm_weights_workspace_bytes
    assert f(100, 4, 512, 1024) == 0 and f(0, 1, 64, 64) == 0 and f(-1, 1, 64, 64) == 0 and f(1 << 20, 1, 60, 64) == 0
    assert f(1 << 20, 64, 2048, 5120) == 0   # tiles enough
    assert f(2047, 1, 256, 256) == 0 and f(2048, 1, 256, 256) == 4 * 256 * 256 * 4
    assert f(1 << 20, 1, 256, 512) == 38 * 256 * 512 * 4
    for n in (1, 1000, 5000, 100000):
        for experts in (1, 3, 20, 1024):
            for N, K in ((8, 8), (264, 1032), (2048, 5120)):
                slices = f(n, experts, N, K) / (experts * N * K * 4)
                assert slices == int(slices) and slices != 1
                assert slices * experts * -(-N // 256) * -(-K // 256) <= 76


def test_product_workspace_bytes():
    f = _lib.load().hc_grouped_mm_workspace_bytes
    assert f(100, 4, 512, 1024) == 0 and f(0, 1, 64, 8192) == 0 and f(-1, 1, 64, 8192) == 0 and f(4, 1, 60, 8192) == 0
    assert f(1, 1, 512, 4088) == 0 and f(1, 1, 512, 4096) == 8 * 512 * 4
    assert f(768, 64, 5120, 8192) == 0   # tiles enough
    for n in (1, 40, 1000, 100000):
        for experts in (1, 3, 20, 1024):
            for N, K in ((8, 8192), (264, 1 << 20), (2048, 5120), (5120, 16384)):
                slices = f(n, experts, N, K) / (n * N * 4)
                assert slices == int(slices) and slices != 1 and slices * experts <= 1024 and slices <= 152


def test_binding_refusals():
    x, w, off = torch.zeros(4, 64).bfloat16(), torch.zeros(2, 32, 64).bfloat16(), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        hcg.hc_grouped_mm(x, w, off)
    with pytest.raises(ValueError, match="CUDA"):
        hcg.hc_grouped_mm_weights(x[:, :32], x, off)
    with pytest.raises(ValueError, match="experts"):
        hcg.hc_grouped_mm_weights(x, x, off[:1])
