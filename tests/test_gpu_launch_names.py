"""The launch timer (dobb_profile_*) names what it times: the moments' kernels by the format of the captures."""
import pytest
import torch

pytestmark = pytest.mark.gpu
dobb = pytest.importorskip("block_diagonal_eigenbasis_amd")


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("nb", [48, 200])
def test_moments_in_splits(nb):
    x, A = torch.randn(4096, 2 * nb, device="cuda"), torch.zeros(2, nb, nb, device="cuda")
    codes, scales = dobb.dobb_mx4_quantize(x)
    op = dobb.dobb_fp8_quantize(x, rows=False, cols=True)[1]
    width = "narrow" if nb <= 128 else "wide"
    for fmt, run in (("mx4", lambda: dobb.dobb_accumulate_moment_mx4(codes, scales, A, nb, 4096)),
                     ("fp8", lambda: dobb.dobb_accumulate_moment_fp8(op, A, nb))):
        dobb.dobb_profile_reset()
        dobb.dobb_profile_enable(True)
        try:
            run()
        finally:
            dobb.dobb_profile_enable(False)
        names = dobb.dobb_profile_read()
        dobb.dobb_profile_reset()
        # (narrow blocks of so few tokens may be summed whole)
        assert f"moment_{fmt}_{width}" in names and set(names) <= {f"moment_{fmt}_{width}", f"moment_{fmt}_reduce"}
        assert width == "narrow" or len(names) == 2
