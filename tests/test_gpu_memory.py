"""GPU: an output that the device has no room for is refused as PyTorch's own allocations are."""
import pytest
import torch

import hyper_connection_residual_mixes_gb300 as hcg
from hyper_connection_residual_mixes_gb300 import _lib
from hyper_connection_residual_mixes_gb300 import build as hc_build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hc_build.build()
    _lib.load()


def test_no_room_for_the_output():
    """The process's own limit is set, so that the refusal is the allocator's and nothing is filled."""
    x, w = torch.ones((1, 1024), device="cuda").expand(1 << 20, 1024), torch.ones((1024,), device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()  # (what earlier calls left in the cache would be room)
    room = (torch.cuda.memory_reserved() + (64 << 20)) / torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction(room)
    try:
        for call in (lambda: hcg.hc_fp8_cast(x), lambda: hcg.hc_rms_norm(x, w), lambda: hcg.hc_layer_norm(x, w)):
            with pytest.raises(torch.cuda.OutOfMemoryError):
                call()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    codes, scales = hcg.hc_fp8_cast(x[:4])
    assert torch.equal(codes, codes[:1].expand(4, 1024)) and scales.shape == (4, 8)
