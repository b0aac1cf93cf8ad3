"""GPU: weights of experts whose sigmoids are tiny.

sigmoid(v) = e^v / (1 + e^v) leaves the normal numbers of fp32 at v = -87; divided by the sum over the
chosen ones it is an ordinary number for any v.  Bounds, u = 2^-24: an exponential of an argument
that was rounded, by at most u times its size (104 at the most before the result is 0 in
fp32), and 2 units of the exponential's own, of up to 17 of them, and some divisions: 160 u of the
weight.  A weight that is not normalised is held in fp32: below its normal numbers to 2^-149."""
import pytest
import torch

import hyper_connection_residual_mixes_gb300 as hcg
from hyper_connection_residual_mixes_gb300 import _lib
from hyper_connection_residual_mixes_gb300 import build as hc_build
from tests import test_gpu_moe_tokens as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hc_build.build()
    _lib.load()


def _log_sigmoid(v):
    return torch.where(v < 0, v - torch.log1p(torch.exp(v)), -torch.log1p(torch.exp(-v)))


@pytest.mark.parametrize("E", [8, 300])
@pytest.mark.parametrize("normalise", [True, False])
def test_tiny_sigmoids(E, normalise):
    g = torch.Generator(device="cuda").manual_seed(E)
    k = 4
    logits = torch.full((12, E), -INF, device="cuda")
    for t, row in enumerate([[-100.0, -100.5, -101, -102], [-88.5, -88.9, -90, -103], [-1000.0, -1000.25, -1003, -1200],
                             [-3.4e38, -3.4e38, -3.4e38, -INF], [-90.0, -INF, -INF, -INF], [-80.0, -85, -95, -104],
                             [3.0, -20.0, -90.0, -100], [-19.5, -20.0, -20.5, -21.0], [-INF] * 4, [0.0, -88.0, -89.0, -3.4e38],
                             [-25.0, -25.0, -25.0, -25.0]]):
        logits[t, 1:5] = torch.tensor(row)
    logits[11] = -150 + torch.randn((E,), generator=g, device="cuda") * 3
    x = torch.randn((12, 64), generator=g, device="cuda").bfloat16()
    w = moe._weights(E, 64, 32, "bf16", "ue8m0", g)
    y, ids, p = moe._call(x, w, logits=logits, top_k=k, score="sigmoid", normalise=normalise, scale=1.5)
    for t in range(12):
        order = sorted((i for i, v in enumerate(logits[t].tolist()) if v > -INF), key=lambda i: (-logits[t, i].item(), i))[:k]
        assert ids[t].tolist() == order + [-1] * (k - len(order))
        v = _log_sigmoid(logits[t, order].double().cpu())
        want = torch.softmax(v, 0) if normalise else torch.exp(v)
        got = p[t, :len(order)].double().cpu() / 1.5
        assert ((got - want).abs() <= 160 * U * want + 2.0 ** -149).all(), (t, got, want)
        assert (p[t, len(order):] == 0).all()
        assert not normalise or not order or abs(got.sum().item() - 1) <= 160 * U
    moe._check(y, x, w, ids, p)
