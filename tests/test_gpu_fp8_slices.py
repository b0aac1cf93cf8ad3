"""GPU: products of rows that are cut out of the middle of a wider buffer, with rows in front and behind.

Bounds: those of the operator's own tests; the same bits as of a copy of the rows."""
import pytest
import torch

import hyper_connection_residual_mixes_gb300 as hcg
from hyper_connection_residual_mixes_gb300 import _lib
from hyper_connection_residual_mixes_gb300 import build as hc_build
from tests import test_gpu_fp8_mm as mm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hc_build.build()
    _lib.load()


@pytest.mark.parametrize("M,N,K", [(1, 144, 272), (12, 528, 1040), (40, 272, 400), (100, 1296, 656), (300, 528, 1040), (2304, 1296, 144), (64, 640, 4112)])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("lead,behind", [(16, 0), (48, 64), (208, 16)])
def test_rows_inside_a_buffer(M, N, K, transposed, lead, behind):
    """All that is not part of x holds codes of NaN."""
    x, sx, w, sw = mm._inputs(M, N, K, transposed, "ue8m0", "fp32")
    L = N if transposed else K
    buf = torch.full((M + 7, lead + L + behind), 0x7f, dtype=torch.uint8, device="cuda")
    cut = buf[3:3 + M, lead:lead + L]
    cut.copy_(x)
    y = hcg.hc_fp8_mm(cut, sx, w, sw, transposed=transposed)
    mm._check(y, x, sx, w, sw, transposed)
    assert torch.equal(y, hcg.hc_fp8_mm(x.contiguous(), sx, w, sw, transposed=transposed))
