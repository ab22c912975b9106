"""What a capture held in FP8 may hold, without a GPU: the sizes that the C call derives its reads from agree with the
tensors, and captures of one weight agree with each other before a step takes them.
"""
import copy
import types

import pytest
import torch

import block_diagonal_eigenbasis_amd as dobb
from block_diagonal_eigenbasis_amd import _layers


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


def test_the_operand_of_joined_captures_knows_its_tokens():
    """Parts of 100 and 77 tokens take a tile each: K is 128 + 77, the tokens are 177."""
    one = dobb.Fp8Capture(operand(1, 6, 100))
    assert one.operand.tokens == 100 and type(one.operand) is dobb.Fp8Operand
    op = dobb.Fp8Capture.cat([one, dobb.Fp8Capture(operand(1, 6, 77))]).operand
    assert op.K == 205 and op.tokens == 177 and isinstance(op, dobb.Fp8Operand) and len(op) == 4
    for other in (op._replace(fmt="e5m2"), copy.copy(op), dobb.Fp8Capture(op, (100, 77)).operand):
        assert other.K == 205 and other.tokens == 177
    assert dobb.Fp8Operand(*op).tokens == 205


def test_the_default_divisor_of_joined_captures_is_their_tokens(monkeypatch):
    seen = []
    monkeypatch.setattr(_layers, "_host", lambda: types.SimpleNamespace(moment_fp8=lambda ops, As, nbs, N, beta, ws: seen.append(N) or 0))
    A = torch.zeros(2, 3, 3)
    joined = dobb.Fp8Capture.cat([dobb.Fp8Capture(operand(1, 6, 100)), dobb.Fp8Capture(operand(1, 6, 77))])
    for op, N, want in ((joined.operand, None, 177), (joined.operand, 205, 205), (operand(2, 6, 205), None, 205),
                        (dobb.Fp8Capture(operand(2, 6, 256), (100, 77)).operand, None, 177)):
        assert dobb.dobb_accumulate_moment_fp8(op, A, 3, N) is A
        assert seen.pop() == want
