"""The experts' layer for a few tokens on the host: refusals of the C entry point (before
any CUDA call; the pointers are not allocations) and of the binding."""
import pytest
import torch

import hyper_connection_residual_mixes_gb300 as hcg
from hyper_connection_residual_mixes_gb300 import _lib
from hyper_connection_residual_mixes_gb300 import build as hc_build

F32, BF16, F16, UE8M0, E4M3 = 0, 1, 2, 3, 4
A, STEP = 0x1000000, 0x10000000


@pytest.fixture(scope="module", autouse=True)
def _built():
    hc_build.build()


def _moe(**kw):
    a = dict(x=A, xs=64, t=BF16, T=4, d=64, experts=8, inner=32, top=2, logits=A + STEP, score=0, norm=1, scale=1.0,
             ids=A + 2 * STEP, p=A + 3 * STEP, up=A + 4 * STEP, down=A + 5 * STEP, wt=E4M3, us=A + 6 * STEP, ds=A + 7 * STEP,
             st=UE8M0, y=A + 8 * STEP, ys=64, ws=A + 9 * STEP, ws_bytes=1 << 20, stream=None)
    a.update(kw)
    return _lib.raw("hc_moe_tokens", *a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), 1), (dict(d=0), 1), (dict(experts=0), 1), (dict(inner=-16), 1), (dict(top=0), 1), (dict(t=UE8M0), 1), (dict(wt=UE8M0), 1),
    (dict(wt=5), 1), (dict(st=BF16), 1), (dict(t=F32), 2), (dict(wt=F16, us=None, ds=None), 2), (dict(T=65), 2), (dict(top=17, experts=32), 2),
    (dict(experts=1025), 2), (dict(d=72, xs=72, ys=72), 2), (dict(inner=40), 2), (dict(d=65552, xs=65552, ys=65552), 2), (dict(xs=68), 2),
    (dict(top=9), 1), (dict(score=2), 1), (dict(scale=float("nan")), 1), (dict(ys=63), 1), (dict(xs=-8), 1),
    (dict(x=None), 1), (dict(up=None), 1), (dict(down=None), 1), (dict(y=None), 1), (dict(us=None), 1), (dict(ds=None), 1),
    (dict(wt=BF16), 1), (dict(logits=None, ids=None), 1), (dict(logits=None, p=None), 1), (dict(ws=None), 1),
    (dict(ws_bytes=4 * 2 * 32 * 4 - 1), 1),
    (dict(x=A + 8), 3), (dict(up=A + 4 * STEP + 8), 3), (dict(down=A + 5 * STEP + 2), 3), (dict(y=A + 8 * STEP + 1), 3),
    (dict(logits=A + STEP + 2), 3), (dict(ids=A + 2 * STEP + 1), 3), (dict(p=A + 3 * STEP + 2), 3), (dict(st=F32, us=A + 6 * STEP + 1), 3),
    (dict(ws=A + 9 * STEP + 4), 3),
    (dict(y=A), 4), (dict(y=A + 4 * STEP + 64), 4), (dict(y=A + 7 * STEP), 4), (dict(ws=A + 8 * STEP), 4), (dict(ids=A + 3 * STEP), 4),
    (dict(ids=A + STEP), 4), (dict(p=A + 8 * STEP), 4), (dict(logits=None, y=A + 2 * STEP), 4), (dict(logits=None, ws=A + 3 * STEP), 4),
    (dict(T=0), 0), (dict(T=0, x=None, y=None), 0),
])
def test_refusals(kw, expect):
    assert _moe(**kw) == expect


def test_workspace_bytes():
    f = _lib.load().hc_moe_tokens_workspace_bytes
    assert f(0, 2, 64) == 0 and f(65, 2, 64) == 0 and f(4, 0, 64) == 0 and f(4, 17, 64) == 0 and f(4, 2, 0) == 0
    assert f(4, 2, 64) == 4 * 2 * 64 * 4 and f(64, 16, 65536) == 64 * 16 * 65536 * 4


def test_binding_refusals():
    x, up, down = torch.zeros(4, 64).bfloat16(), torch.zeros(8, 2, 32, 64).bfloat16(), torch.zeros(8, 64, 32).bfloat16()
    with pytest.raises(ValueError, match="CUDA"):
        hcg.hc_moe_tokens(x, up, down, logits=torch.zeros(4, 8), top_k=2)
    with pytest.raises(TypeError, match="x must be"):
        hcg.hc_moe_tokens(x.float(), up, down, logits=torch.zeros(4, 8), top_k=2)
