"""How many tokens one fp32 sum of an FP8 moment holds, read off the workspace that a call asks for: blocks wider than
128 columns are split so that none holds more than 32 tiles (4096 tokens), whatever else the plan weighs."""
import pytest

import block_diagonal_eigenbasis_amd as dobb


@pytest.mark.parametrize("nb,blocks", [(129, 1), (192, 64), (400, 1), (400, 16), (400, 192), (400, 768), (512, 32), (1024, 8)])
@pytest.mark.parametrize("tiles", [33, 64, 65, 128, 129, 500, 1025])
def test_wide_blocks_are_split(nb, blocks, tiles):
    splits = -(-tiles // 32)
    assert dobb.dobb_moment_fp8_workspace_size([(1, nb * blocks, nb)], tiles) >= splits * blocks * nb * nb * 4


def test_blocks_of_few_tokens_may_be_whole():
    assert dobb.dobb_moment_fp8_workspace_size([(1, 400 * 192, 400)], 32) == 0
