"""Errors of the binding of dobb_ops.h that only a GPU shows."""
import pytest
import torch

pytestmark = pytest.mark.gpu
dobb = pytest.importorskip("block_diagonal_eigenbasis_amd")
DEV = "cuda"


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def test_an_allocation_that_fails_is_torchs_error():
    """torch's limit for the process forced to nothing: what a call allocates is refused by the allocator."""
    x = torch.randn(4096, 4096, device=DEV)
    codes, scales = dobb.dobb_mx4_quantize(x)
    want = dobb.dobb_mx4_dequantize(codes, scales, 4096)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(0.0)
    try:
        with pytest.raises(torch.OutOfMemoryError, match="out of memory"):
            dobb.dobb_mx4_dequantize(codes, scales, 4096)        # 64 MB, more than is left over in any segment
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert torch.equal(dobb.dobb_mx4_dequantize(codes, scales, 4096), want)
