"""RMS norm and the casts to 8 bits on the host: the C entry points' refusals (made
before any CUDA call; the pointers are not allocations) and the binding's."""
import pytest
import torch

import hyper_connection_residual_mixes_gb300 as hcg
from hyper_connection_residual_mixes_gb300 import _lib
from hyper_connection_residual_mixes_gb300 import build as hc_build

F32, BF16, F16, UE8M0 = 0, 1, 2, 3
A, STEP = 0x1000000, 0x1000000


@pytest.fixture(scope="module", autouse=True)
def _built():
    hc_build.build()


def _fwd(**kw):
    a = dict(x=A, xs=64, res=A + STEP, res_s=64, t=BF16, w=A + 2 * STEP, wt=F32, n=16, d=64, eps=1e-6, r=A + 3 * STEP, rs=64,
             y=A + 4 * STEP, ys=64, codes=A + 5 * STEP, cs=64, scales=A + 6 * STEP, rstd=A + 7 * STEP, stream=None)
    a.update(kw)
    return _lib.raw("hc_rms_norm", *a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(n=-1), 1), (dict(d=0), 1), (dict(d=16385), 2), (dict(n=1 << 31), 2), (dict(t=UE8M0), 1), (dict(t=-1), 1),
    (dict(wt=F16), 2), (dict(wt=UE8M0), 1), (dict(t=F32, wt=BF16), 2),
    (dict(eps=-1.0), 1), (dict(eps=float("inf")), 1), (dict(xs=-1), 1), (dict(res_s=-64), 1), (dict(rs=63), 1), (dict(ys=63), 1),
    (dict(cs=63), 1), (dict(xs=1 << 62), 1),
    (dict(x=None), 1), (dict(w=None), 1), (dict(r=None), 1), (dict(res=None), 1), (dict(codes=None), 1), (dict(scales=None), 1),
    (dict(y=None, codes=None, scales=None), 1),
    (dict(x=A + 1), 3), (dict(res=A + STEP + 1), 3), (dict(w=A + 2 * STEP + 2), 3), (dict(r=A + 3 * STEP + 1), 3),
    (dict(y=A + 4 * STEP + 1), 3), (dict(rstd=A + 7 * STEP + 2), 3),
    (dict(y=A), 4), (dict(y=A + STEP), 4), (dict(y=A + 3 * STEP), 4), (dict(codes=A + 4 * STEP), 4), (dict(scales=A + 5 * STEP), 4),
    (dict(rstd=A + 2 * STEP), 4), (dict(r=A + 64), 4), (dict(r=A + 2 * STEP), 4), (dict(r=A + STEP + 128), 4),
    (dict(r=A, rs=128), 4), (dict(r=A + STEP, rs=72), 4),
    (dict(r=A, x=A, res=A + 64), 4),                 # r is x, but meets the residual's other rows
    (dict(n=0), 0), (dict(n=0, x=None, y=None), 0),
])
def test_forward_refusals(kw, expect):
    assert _fwd(**kw) == expect


def _bwd(**kw):
    a = dict(g=A, gs=64, gr=A + STEP, grs=64, gt=F32, r=A + 2 * STEP, rs=64, t=BF16, w=A + 3 * STEP, wt=F32, rstd=A + 4 * STEP,
             n=16, d=64, gx=A + 5 * STEP, gxs=64, gw=A + 6 * STEP, ws=A + 7 * STEP, ws_bytes=STEP, stream=None)
    a.update(kw)
    return _lib.raw("hc_rms_norm_backward", *a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(n=-1), 1), (dict(d=0), 1), (dict(d=16385), 2), (dict(gt=7), 1), (dict(gt=F16), 2), (dict(t=F32, gt=BF16), 2),
    (dict(gs=-1), 1), (dict(grs=-1), 1), (dict(gxs=60), 1), (dict(gw=None), 1), (dict(rstd=None), 1), (dict(gx=None), 1),
    (dict(ws=None), 1), (dict(ws_bytes=16 * 64 * 4 - 1), 1), (dict(ws=A + 7 * STEP + 8), 3), (dict(g=A + 2), 3), (dict(gr=A + STEP + 2), 3),
    (dict(gx=A), 4), (dict(gx=A + 2 * STEP), 4), (dict(gx=A + STEP + 256), 4), (dict(gx=A + STEP, gxs=65), 4),
    (dict(gw=A + STEP), 4), (dict(ws=A + 5 * STEP), 4), (dict(ws=A + STEP), 4),
])
def test_backward_refusals(kw, expect):
    assert _bwd(**kw) == expect


def test_backward_workspace_size():
    f = _lib.load().hc_rms_norm_backward_workspace_bytes
    assert f(0, 64) == 0 and f(-1, 64) == 0 and f(4, 0) == 0 and f(4, 20000) == 0
    assert f(16, 64) == 16 * 64 * 4                      # one row of partial sums per row at the most
    assert f(1 << 20, 5120) == f(1 << 30, 5120)          # and no more than the blocks of a launch


def _cast(**kw):
    a = dict(x=A, xs=64, t=BF16, n=16, d=64, codes=A + STEP, cs=64, scales=A + 2 * STEP, stream=None)
    a.update(kw)
    return _lib.raw("hc_fp8_cast", *a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(n=-1), 1), (dict(d=0), 1), (dict(t=UE8M0), 1), (dict(n=1 << 31), 2), (dict(n=1 << 24, d=1 << 20, xs=1 << 20, cs=1 << 20), 2),
    (dict(xs=-1), 1), (dict(cs=63), 1), (dict(x=None), 1), (dict(codes=None), 1), (dict(scales=None), 1), (dict(x=A + 1), 3),
    (dict(codes=A), 4), (dict(scales=A + 8), 4), (dict(scales=A + STEP + 64), 4), (dict(n=0), 0),
])
def test_cast_refusals(kw, expect):
    assert _cast(**kw) == expect


def _cast_w(**kw):
    a = dict(w=A, t=F16, count=2, N=64, K=96, codes=A + STEP, scales=A + 2 * STEP, stream=None)
    a.update(kw)
    return _lib.raw("hc_fp8_cast_weights", *a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(count=-1), 1), (dict(N=0), 1), (dict(K=-1), 1), (dict(t=3), 1), (dict(count=1 << 31), 2), (dict(N=1 << 30, K=1 << 30), 2),
    (dict(w=None), 1), (dict(codes=None), 1), (dict(scales=None), 1), (dict(w=A + 1), 3), (dict(codes=A), 4), (dict(scales=A), 4),
    (dict(scales=A + STEP + 64), 4), (dict(count=0), 0),
])
def test_cast_weights_refusals(kw, expect):
    assert _cast_w(**kw) == expect


def test_binding_refusals():
    x, w = torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(ValueError, match="CUDA"):
        hcg.hc_rms_norm(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        hcg.hc_rms_norm_backward(x, x, w, torch.zeros(4))
    with pytest.raises(TypeError, match="x must be"):
        hcg.hc_rms_norm(x.double(), w)
    with pytest.raises(ValueError, match="evenly spaced"):
        hcg.hc_rms_norm(torch.zeros(4, 3, 6, 64)[:, :2, :4], w)
    with pytest.raises(ValueError, match="CUDA"):
        hcg.hc_fp8_cast(x)
    with pytest.raises(TypeError, match="x must be"):
        hcg.hc_fp8_cast(x.int())
    with pytest.raises(ValueError, match="CUDA"):
        hcg.hc_fp8_cast_weights(x)
    with pytest.raises(ValueError, match="N, K"):
        hcg.hc_fp8_cast_weights(w)
