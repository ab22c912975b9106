"""FP8 moments of long captures whose small terms an fp32 sum does not see.

One token of ones and then tokens of 2^-14: sixteen products of 2^-28 are half of the last bit of a sum that holds the 1, and
are lost to it, whatever it rounds to.  A sum of at most 4096 tokens loses 4095 2^-28 < 2^-16; those of the other tokens are
exact.  So every entry, (1 + (N - 1) 2^-28)/N, may be (2^-16 + 4 u)/N off, u = 2^-24 for three additions and the result,
where one sum of all 16384 tokens would be 2^-14/N off.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
dobb = pytest.importorskip("block_diagonal_eigenbasis_amd")
DEV = "cuda"


@pytest.mark.parametrize("nb,B", [(32, 600), (100, 576), (128, 16), (129, 8), (192, 128), (400, 192), (400, 4), (1024, 20)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_small_terms_of_a_long_capture(nb, B, fmt):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N = 16384
    x = torch.full((N, nb * B), 2.0 ** -14, dtype=torch.bfloat16, device=DEV)
    x[0] = 1.0
    op = dobb.dobb_fp8_quantize(x, rows=False, cols=True, fmt=fmt)[1]
    A = dobb.dobb_accumulate_moment_fp8(op, torch.empty(B, nb, nb, device=DEV), nb)
    off = (A.double() * N - (1 + (N - 1) * 2.0 ** -28)).abs().max()
    assert float(off) <= 2.0 ** -16 + 4 * 2.0 ** -24
