"""What a capture held in FP8 may hold, without a GPU: the sizes that the C call derives its reads from agree with the
tensors, and captures of one weight agree with each other before a step takes them.
"""
import copy
import gc
import types
import weakref

import pytest
import torch

import block_diagonal_eigenbasis_amd as dobb
from block_diagonal_eigenbasis_amd import _layers
from block_diagonal_eigenbasis_amd.optimizer import Dobb, DobbGroup, Mx4Capture


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


def _held(kind, N=50, n=6):
    if kind == "mx4":
        T = dobb.mx4_tiles(N)
        return Mx4Capture(torch.zeros(T, 4, n, 16, dtype=torch.uint8), torch.zeros(T, n, 4, dtype=torch.uint8), (N,))
    return torch.zeros(N, n) if kind == "native" else dobb.Fp8Capture(operand(dobb.fp8_tiles(N), n, N, kind))


@pytest.mark.parametrize("first,second", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e4m3", "mx4"), ("native", "e4m3"), ("mx4", "native")])
def test_captures_that_cannot_be_joined_are_refused_when_they_come(first, second):
    """.. and not by every step from then on."""
    p = torch.nn.Parameter(torch.zeros(8, 6))
    opt = Dobb([p], block_size=3, capture="all")
    opt.capture(p, _held(first))
    with pytest.raises(ValueError, match="held alike"):
        opt.capture(p, _held(second))
    opt.capture(p, _held(first, 7))
    assert [c.shape[0] for c in opt._captured[id(p)]] == [50, 7]


@pytest.mark.parametrize("policy", ["first", "all"])
@pytest.mark.parametrize("kind", ["native", "e4m3", "e5m2", "mx4"])
@pytest.mark.parametrize("basis", ["activation", "output_gradient"])
def test_a_capture_of_another_width_is_refused_when_it_comes(policy, kind, basis):
    p = torch.nn.Parameter(torch.zeros(9, 6))
    opt = Dobb([p], block_size=3, capture=policy, basis=basis)
    for n in (3, 6, 9):
        if n != (6 if basis == "activation" else 9):
            with pytest.raises(ValueError, match="capture 0"):
                opt.capture(p, _held(kind, n=n))
    assert not opt._captured
    opt.capture(p, _held(kind, n=6 if basis == "activation" else 9))
    assert len(opt._captured) == 1


def test_a_capture_of_another_type_is_refused_when_it_comes():
    p = torch.nn.Parameter(torch.zeros(8, 6))
    opt = Dobb([p], block_size=3)
    with pytest.raises(TypeError):
        opt.capture(p, torch.zeros(5, 6).half())
    assert not opt._captured
    with pytest.raises(ValueError):
        opt.capture(p, torch.zeros(5, 6, device="meta"))
    assert not opt._captured


def _shifted(t):
    """t at an address that is not a multiple of 4."""
    raw = torch.zeros(t.numel() + 16, dtype=torch.uint8)
    out = raw[(1 - raw.data_ptr()) % 4:][:t.numel()].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("kind", ["e4m3", "mx4"])
def test_a_capture_that_is_not_aligned_is_refused_before_anything_is_enqueued(kind):
    """The C call refuses it, but only after the calls for other weights."""
    c = _held(kind, 200)
    for part in ("codes", "scales"):
        if kind == "mx4":
            odd = Mx4Capture(*(_shifted(t) if k == part else t for k, t in (("codes", c.codes), ("scales", c.scales))), c.parts)
        else:
            odd = dobb.Fp8Capture(c.operand._replace(**{part: _shifted(getattr(c.operand, part))}))
        g = DobbGroup([torch.zeros(8, 6)], [3])
        with pytest.raises(ValueError, match="aligned"):
            g._plan([odd])
        g._plan([type(odd).cat([odd])])
        p = torch.nn.Parameter(torch.zeros(8, 6))
        opt = Dobb([p], block_size=3)
        opt.capture(p, odd)                                       # copied, not kept as it is
        (got,) = opt._captured[id(p)]
        assert got.aligned and not odd.aligned and got.parts == odd.parts and got.shape == odd.shape
        g._plan([got])


@pytest.mark.parametrize("kind", ["native", "e4m3", "mx4"])
def test_joined_captures_take_the_place_of_their_parts(monkeypatch, kind):
    """With capture="all" a refresh does not hold every weight's captures twice."""
    params = [torch.nn.Parameter(torch.zeros(8, 6)) for _ in range(3)]
    opt = Dobb(params, block_size=3, capture="all")
    parts = []
    for N in (50, 7, 130):
        for p in params:
            opt.capture(p, _held(kind, N))
            parts.append(weakref.ref(opt._captured[id(p)][-1]))
    assert all(r() is not None for r in parts)
    seen = []

    def refresh_step(xs, *args, **kw):
        gc.collect()
        seen.append([x.shape[0] for x in xs])
        assert all(r() is None for r in parts)
        if len(seen) == 1:
            raise RuntimeError("this step fails")
    monkeypatch.setattr(opt._group, "refresh_step", refresh_step)
    with pytest.raises(RuntimeError, match="this step fails"):
        opt.step()
    opt.step()                                                    # with what was joined
    assert seen == [[187] * 3] * 2 and not opt._captured
