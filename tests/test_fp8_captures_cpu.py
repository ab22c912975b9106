"""What a capture held in FP8 may hold, without a GPU: the sizes that the C call derives its reads from agree with the
tensors, and captures of one weight agree with each other before a step takes them.
"""
import pytest
import torch

import block_diagonal_eigenbasis_amd as dobb


def operand(T, n, K, fmt="e4m3"):
    return dobb.Fp8Operand(torch.zeros(T, 8, n, 16, dtype=torch.uint8), torch.zeros(T, (n + 3) // 4 * 4, dtype=torch.uint8), K, fmt)


@pytest.mark.parametrize("K", [74, 1, 128, 257, 100000, 0, -1])
def test_an_operand_of_other_tiles_than_its_codes_is_refused(K):
    """Two micro-batches of 37 tokens take a tile each: K = 74 would leave the second out, K = 100000 read past both."""
    with pytest.raises(ValueError, match="K must be"):
        dobb.Fp8Capture(operand(2, 6, K), (37, 37))
    with pytest.raises(ValueError):
        dobb.Fp8Capture(operand(2, 6, K))


@pytest.mark.parametrize("K", [129, 165, 256])
def test_an_operand_of_its_codes_tiles_is_taken(K):
    c = dobb.Fp8Capture(operand(2, 6, K), (37, 37))
    assert c.shape == (74, 6) and c.tiles == 2 == dobb.fp8_tiles(c.operand.K)
