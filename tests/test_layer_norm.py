"""Layer norm on the host: the C entry points' refusals (made before any CUDA
call; the pointers are not allocations) and the binding's."""
import pytest
import torch

import hyper_connection_residual_mixes_gb300 as hcg
from hyper_connection_residual_mixes_gb300 import _lib
from hyper_connection_residual_mixes_gb300 import build as hc_build

F32, BF16, F16 = 0, 1, 2
A = 0x1000000
STEP = 0x1000000


@pytest.fixture(scope="module", autouse=True)
def _built():
    hc_build.build()


def _fwd(**kw):
    a = dict(x=A, xs=64, xt=BF16, w=A + STEP, b=A + 2 * STEP, wt=F32, n=16, d=64, eps=1e-5, y=A + 3 * STEP, ys=64,
             mean=A + 4 * STEP, rstd=A + 5 * STEP, stream=None)
    a.update(kw)
    return _lib.raw("hc_layer_norm", *a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(n=-1), 1), (dict(d=0), 1), (dict(d=-5), 1), (dict(d=16385), 2), (dict(xt=3), 1), (dict(wt=-1), 1),
    (dict(n=1 << 31), 2),
    (dict(wt=F16), 2), (dict(xt=F32, wt=BF16), 2),   # norm_w: fp32 or x's type
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(xs=-1), 1), (dict(ys=63), 1), (dict(xs=1 << 62), 1),
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1),
    (dict(x=A + 1), 3), (dict(w=A + STEP + 2), 3), (dict(mean=A + 4 * STEP + 2), 3), (dict(y=A + 3 * STEP + 1), 3),
    (dict(y=A + 64), 4),                             # y overlaps x
    (dict(y=A, ys=64), 4),                           # in place is refused
    (dict(mean=A + 3 * STEP + 4), 4), (dict(rstd=A + STEP), 4),
    (dict(n=0), 0), (dict(n=0, x=None, y=None), 0),
])
def test_forward_refusals(kw, expect):
    assert _fwd(**kw) == expect


def _bwd(**kw):
    a = dict(g=A, gs=64, gt=F32, x=A + STEP, xs=64, xt=BF16, w=A + 2 * STEP, wt=F32, mean=A + 3 * STEP,
             rstd=A + 4 * STEP, n=16, d=64, gx=A + 5 * STEP, gxs=64, g_w=A + 6 * STEP, g_b=A + 7 * STEP,
             ws=A + 8 * STEP, ws_bytes=STEP, stream=None)
    a.update(kw)
    return _lib.raw("hc_layer_norm_backward", *a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(n=-1), 1), (dict(d=0), 1), (dict(d=16385), 2), (dict(gt=7), 1), (dict(gt=F16), 2),
    (dict(xt=F32, gt=BF16), 2), (dict(xt=F16, wt=BF16), 2),
    (dict(gxs=60), 1), (dict(gs=-64), 1), (dict(g_w=None), 1), (dict(mean=None), 1), (dict(gx=None), 1),
    (dict(ws=None), 1), (dict(ws_bytes=8191), 1), (dict(ws=A + 8 * STEP + 8), 3), (dict(g=A + 2), 3),
    (dict(g_b=A + 7 * STEP + 1), 3),
    (dict(gx=A, gxs=64), 4), (dict(gx=A + STEP + 32), 4), (dict(g_w=A + 7 * STEP), 4), (dict(ws=A + 5 * STEP), 4),
])
def test_backward_refusals(kw, expect):
    assert _bwd(**kw) == expect


def test_backward_workspace_size():
    f = _lib.load().hc_layer_norm_backward_workspace_bytes
    assert f(0, 64) == 0 and f(-1, 64) == 0 and f(4, 0) == 0 and f(4, 20000) == 0
    assert f(16, 64) == 16 * 2 * 64 * 4                  # one row of partial sums per row at the most
    assert f(1 << 20, 5120) == f(1 << 30, 5120)          # and no more than the blocks of a launch


def test_binding_refusals():
    x, w = torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(ValueError, match="CUDA"):
        hcg.hc_layer_norm(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        hcg.hc_layer_norm_backward(x, x, w, torch.zeros(4), torch.zeros(4))
    with pytest.raises(TypeError, match="x must be"):
        hcg.hc_layer_norm(x.double(), w)
    with pytest.raises(ValueError, match="dense along"):
        hcg.hc_layer_norm(torch.zeros(64, 4).t(), w)
    with pytest.raises(ValueError, match="evenly spaced"):
        hcg.hc_layer_norm(torch.zeros(4, 3, 6, 64)[:, :2, :4], w)
