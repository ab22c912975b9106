"""Which captures the torch.optim wrapper takes and how it hands them to the quantiser, without a GPU: the
quantiser is a stand-in that notes its input (a tensor whose rows have unit column stride and do not overlap).
"""
import pytest
import torch

import block_diagonal_eigenbasis_amd as dobb
from block_diagonal_eigenbasis_amd import _ops
from block_diagonal_eigenbasis_amd.optimizer import Dobb, Mx4Capture


def rows_are_taken(x):
    N, n = x.shape
    return N >= 1 and not x.is_neg() and (n == 1 or x.stride(1) == 1) and (N == 1 or x.stride(0) >= n)


@pytest.fixture
def seen(monkeypatch):
    got = []

    def quantize(x, codes=None, scales=None, stream=None):
        assert rows_are_taken(x), (x.shape, x.stride())
        got.append(x)
        T, n = dobb.mx4_tiles(x.shape[0]), x.shape[1]
        return torch.zeros(T, 4, n, 16, dtype=torch.uint8), torch.zeros(T, n, 4, dtype=torch.uint8)
    monkeypatch.setattr(_ops, "dobb_mx4_quantize", quantize)
    return got


def layouts():
    base = torch.randn(6, 40)
    return {
        "dense": base,
        "rows of a wider buffer": base[:, 3:20],
        "three axes": torch.randn(2, 5, 16),
        "transposed": base.T,
        "every second column": base[:, ::2],
        "one token, every second column": base[:1, ::2],
        "one row for all tokens": base[:1].expand(9, 40),
        "one entry for all": torch.ones(()).expand(9, 40),
        "one entry for all, three axes": torch.ones(()).expand(3, 3, 40),
        "overlapping rows": base.reshape(-1).as_strided((9, 40), (7, 1)),
        "one column of a wider buffer": base[:, 3:4],
        "one column, one entry": torch.ones(()).expand(9, 1),
        "negated view": torch.randn(6, 8, dtype=torch.complex64).conj().imag,
        "negated dense view": torch.view_as_real(torch.randn(6, 8, dtype=torch.complex64)).select(2, 1)._neg_view(),
    }


@pytest.mark.parametrize("name", layouts())
def test_every_layout_is_captured(seen, name):
    x = layouts()[name]
    n = x.shape[-1]
    for fmt in ("native", "mx4"):
        w = torch.nn.Parameter(torch.zeros(4, n))
        opt = Dobb([w], blocks=1, capture_format=fmt)
        opt.capture(w, x)
        (held,) = opt._captured[id(w)]
        want = x.reshape(-1, n)
        assert held.shape == tuple(want.shape)
        assert torch.equal(seen[0] if fmt == "mx4" else held, want)
    if rows_are_taken(want):                                     # no copy where the quantiser reads the rows as they are
        assert seen[0].data_ptr() == want.data_ptr() or name == "three axes"
    Mx4Capture.quantize(want)


@pytest.mark.parametrize("fmt", ["native", "mx4"])
@pytest.mark.parametrize("policy", ["first", "all"])
def test_micro_batches_without_tokens_are_passed_over(seen, fmt, policy):
    w = torch.nn.Parameter(torch.zeros(4, 16))
    opt = Dobb([w], blocks=1, capture_format=fmt, capture=policy)
    for k in (0, 3, 0, 5):
        opt.capture(w, torch.randn(2, k, 16))
    assert [c.shape[0] for c in opt._captured[id(w)]] == ([6, 10] if policy == "all" else [6])


@pytest.mark.parametrize("policy", ["first", "all"])
def test_a_refused_capture_leaves_nothing_behind(monkeypatch, policy):
    def refuse(*a, **k):
        raise TypeError("unsupported dtype")
    monkeypatch.setattr(_ops, "dobb_mx4_quantize", refuse)
    w = torch.nn.Parameter(torch.zeros(4, 16))
    opt = Dobb([w], blocks=1, capture_format="mx4", capture=policy)
    with pytest.raises(TypeError, match="unsupported dtype"):
        opt.capture(w, torch.randn(3, 16).half())
    assert not opt._captured
