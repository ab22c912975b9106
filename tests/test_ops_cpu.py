"""The C ABI of include/dobb_ops.h without a GPU: every declared entry point is exported, and bad
arguments are refused on the host before anything is enqueued.

Every call below is invalid in at least one argument, so the non-null "device pointers" are never
dereferenced.
"""
import ctypes
import os
import re

import pytest
import torch

import block_diagonal_eigenbasis_amd as dobb
from block_diagonal_eigenbasis_amd import _abi, _ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000
INVALID, SHAPE, DTYPE, WORKSPACE = -1, -2, -3, -4


def test_library_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "dobb_ops.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(dobb_\w+)\s*\(", text)))
    assert len(names) == 9
    L = _ops._lib()
    assert not [n for n in names if not hasattr(L, n)]


def _i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


def _int(*v):
    return (ctypes.c_int * len(v))(*v)


def _ptr(*v):
    return (ctypes.c_void_p * len(v))(*v)


def _norm(numel=(64, 10), G=(FAKE, FAKE + 0x1000), dt=(0, 1), total=0x80000, ws=0x90000, wsb=1 << 20, count=None):
    return _ops._lib().dobb_grad_norm_grouped(len(numel) if count is None else count, _i64(*numel), _ptr(*G), _int(*dt),
                                              None, total, ws, wsb, None)


def test_grad_norm_refusals():
    assert _norm(count=0) == INVALID
    assert _norm(total=None) == INVALID
    assert _norm(G=(FAKE, None)) == INVALID
    assert _norm(G=(FAKE, FAKE + 1)) == INVALID          # not aligned to its entries
    assert _norm(G=(FAKE + 2, FAKE)) == INVALID
    assert _norm(dt=(0, 2)) == DTYPE
    assert _norm(numel=(64, -1)) == SHAPE
    assert _norm(ws=None) == WORKSPACE
    assert _norm(ws=0x90010) == WORKSPACE
    assert _norm(wsb=8) == WORKSPACE
    size = _ops._lib().dobb_grad_norm_workspace_size
    assert size(2, _i64(64, 10), _int(0, 1)) >= 8 * 2
    assert size(1, _i64(0), _int(0)) > 0                 # the call still writes the total
    assert size(0, _i64(1), _int(0)) == 0 and size(1, _i64(-1), _int(0)) == 0 and size(1, _i64(1), _int(3)) == 0
    # the partial sums of a large list stay few: one per chunk, chunks grow with the list
    assert size(192, _i64(*[7680000] * 192), _int(*[1] * 192)) <= 8 * (8192 + 192) + 512


def _clip(numel=(64, 64), G=(FAKE, FAKE + 0x1000), dt=(0, 0), out=(FAKE, FAKE + 0x1000), odt=(0, 0), total=FAKE + 0x8000,
          max_norm=1.0):
    a = (len(numel), _i64(*numel), _ptr(*G), _int(*dt), _ptr(*out), _int(*odt))
    one = _ops._lib().dobb_clip_grads_grouped(*a, total, max_norm, None)
    # the call with the norm in front refuses the same, before its workspace is looked at
    assert one == _ops._lib().dobb_clip_grad_norm_grouped(*a, max_norm, None, total, None, 0, None)
    return one


def test_clip_refusals():
    nan, inf = float("nan"), float("inf")
    assert _clip(total=None) == INVALID
    assert _clip(max_norm=-1.0) == INVALID and _clip(max_norm=nan) == INVALID and _clip(max_norm=-inf) == INVALID
    assert _clip(odt=(0, 5)) == DTYPE and _clip(dt=(7, 0)) == DTYPE
    assert _clip(out=(FAKE, None)) == INVALID
    assert _clip(numel=(64, -2)) == SHAPE
    # one tensor twice in place, or one buffer for two outputs: it would be scaled twice
    assert _clip(G=(FAKE, FAKE), out=(FAKE, FAKE)) == INVALID
    assert _clip(out=(0x40000, 0x40000)) == INVALID
    assert _clip(out=(0x40000, 0x40000 + 255)) == INVALID
    assert _clip(out=(0x40000, 0x40000 + 252)) == INVALID            # 64 fp32 entries are 256 bytes
    # an output over another tensor, or shifted over its own, or in place with another type
    assert _clip(out=(FAKE + 0x1000, 0x40000)) == INVALID
    assert _clip(out=(FAKE + 4, FAKE + 0x1000)) == INVALID
    assert _clip(odt=(1, 0)) == INVALID
    # one long buffer around several shorter ones
    assert _clip(numel=(4096, 16), G=(0x20000, 0x10000), out=(0x40000, 0x40000 + 8192)) == INVALID
    # the total among what is written, or read, and the sums and the workspace over a gradient
    assert _clip(total=FAKE + 8) == INVALID
    lib, one = _ops._lib(), (1, _i64(64), _ptr(FAKE), _int(0))
    assert lib.dobb_grad_norm_grouped(*one, None, FAKE + 252, 0x40000, 1 << 20, None) == INVALID
    assert lib.dobb_grad_norm_grouped(*one, FAKE, 0x80000, 0x40000, 1 << 20, None) == INVALID
    assert lib.dobb_grad_norm_grouped(*one, 0x80000, 0x80000, 0x40000, 1 << 20, None) == INVALID
    assert lib.dobb_grad_norm_grouped(*one, None, 0x80000, FAKE, 1 << 20, None) == INVALID
    assert lib.dobb_clip_grad_norm_grouped(*one, _ptr(0x20000), _int(0), 1.0, None, 0x80000, 0x20000, 1 << 20, None) == INVALID
    # many separate allocations, in no order: the same answers
    import random
    at = [0x100000 + 0x1000 * i for i in range(400)]
    random.Random(1).shuffle(at)
    many = dict(numel=(64,) * 400, G=tuple(at), dt=(0,) * 400, odt=(0,) * 400)
    assert _clip(**many, out=tuple(a if i != 399 else at[17] for i, a in enumerate(at))) == INVALID
    a = (400, _i64(*many["numel"]), _ptr(*at), _int(*many["dt"]), _ptr(*at), _int(*many["odt"]))
    assert lib.dobb_clip_grad_norm_grouped(*a, 1.0, None, 0x40000, None, 0, None) == WORKSPACE      # this list is in order
    # the bad list of a call is refused with its workspace in order too
    bad = (2, _i64(64, 64), _ptr(FAKE, FAKE), _int(0, 0), _ptr(FAKE, FAKE), _int(0, 0))
    assert _ops._lib().dobb_clip_grad_norm_grouped(*bad, 1.0, None, FAKE, FAKE, 1 << 20, None) == INVALID
    good = (2, _i64(64, 64), _ptr(FAKE, FAKE + 256), _int(0, 0), _ptr(FAKE, FAKE + 256), _int(0, 0))
    assert _ops._lib().dobb_clip_grad_norm_grouped(*good, 1.0, None, 0x80000, None, 0, None) == WORKSPACE


def test_mx4_refusals():
    L = _ops._lib()

    def both(N=100, n=40, X=FAKE, dt=0, ld=40, codes=FAKE, scales=FAKE):
        a = L.dobb_mx4_quantize(N, n, X, dt, ld, codes, scales, None)
        b = L.dobb_mx4_dequantize(N, n, codes, scales, X, dt, ld, None)
        assert a == b
        return a
    assert both(X=None) == INVALID and both(codes=None) == INVALID and both(scales=None) == INVALID
    assert both(N=0) == INVALID and both(n=0) == SHAPE and both(ld=39) == SHAPE and both(n=(1 << 24) + 1, ld=1 << 26) == SHAPE
    assert both(dt=2) == DTYPE
    assert both(codes=FAKE + 8) == INVALID and both(scales=FAKE + 2) == INVALID and both(X=FAKE + 2) == INVALID
    assert both(N=1 << 39, n=1 << 20, ld=1 << 20) == SHAPE            # more tiles than a grid holds


def test_moment_mx4_refusals():
    L = _ops._lib()
    s = _abi.Shape(1, 768, 192)

    def call(s=s, codes=FAKE, scales=FAKE, tiles=64, N=8192, beta=0.5, A=FAKE, ws=None, wsb=0):
        return L.dobb_accumulate_moment_mx4(ctypes.byref(s), codes, scales, tiles, N, beta, A, ws, wsb, None)
    assert L.dobb_accumulate_moment_mx4(None, FAKE, FAKE, 8, 1024, 0.5, FAKE, None, 0, None) == INVALID
    assert call(codes=None) == INVALID and call(scales=None) == INVALID and call(A=None) == INVALID
    assert call(codes=FAKE + 8) == INVALID and call(scales=FAKE + 1) == INVALID and call(A=FAKE + 2) == INVALID
    assert call(tiles=0) == INVALID and call(N=0) == INVALID and call(N=8193) == INVALID
    assert call(beta=1.0) == INVALID and call(beta=-0.5) == INVALID and call(beta=float("nan")) == INVALID
    for n, nb in ((0, 1), (768, 0), (768, 100), (4096, 2048), (1 << 26, 64)):
        assert call(s=_abi.Shape(1, n, nb)) == SHAPE
    need = dobb.dobb_moment_mx4_workspace_size([(1, 768, 192)], 64)
    assert need > 0 and need % 256 == 0
    two = (_abi.Shape * 2)(_abi.Shape(1, 768, 192), _abi.Shape(1, 768, 192))
    grouped = L.dobb_accumulate_moment_mx4_grouped
    size_a, size_c = 768 * 192 * 4, 64 * 64 * 768
    C, S, A = 0x10000000, 0x20000000, 0x30000000
    assert grouped(2, two, _ptr(C, C), _ptr(S, S), 64, 8192, 0.5, _ptr(A, A), None, 0, None) == INVALID          # one moment twice
    assert grouped(2, two, _ptr(C, C), _ptr(S, S), 64, 8192, 0.5, _ptr(A, A + size_a - 4), None, 0, None) == INVALID
    assert grouped(2, two, _ptr(C, C), _ptr(S, S), 64, 8192, 0.5, _ptr(A, C + size_c - 4), None, 0, None) == INVALID
    assert grouped(2, two, _ptr(C, C), _ptr(S, S), 64, 8192, 0.5, _ptr(A, A + size_a), None, 0, None) == WORKSPACE  # a shared capture
    assert call(codes=C, scales=S, A=A) == WORKSPACE
    assert call(codes=C, scales=S, A=A, ws=FAKE, wsb=need - 1) == WORKSPACE and call(codes=C, scales=S, A=A, ws=FAKE + 64, wsb=need) == WORKSPACE
    size = dobb.dobb_moment_mx4_workspace_size
    assert size([(1, 768, 100)], 8) == 0 and size([(1, 768, 192)], 0) == 0
    # one tile has nothing to split; a long capture is split whatever the grid
    assert size([(1, 768, 192)], 1) == 0
    assert size([(1, 128 * 1024, 128)], 1024) > 0
    # the last launch of a group of many (one matrix here) is split where the full one before it is not
    assert size([(1, 1600, 100)] * 97, 128) >= size([(1, 1600, 100)], 128) > 0


def test_python_refusals_without_a_gpu():
    x = torch.zeros(4, 4)
    with pytest.raises(ValueError, match="empty"):
        dobb.dobb_grad_norm_grouped([])
    for call in (lambda: dobb.dobb_grad_norm_grouped([x]), lambda: dobb.dobb_clip_grad_norm_grouped([x], 1.0),
                 lambda: dobb.dobb_clip_grads_grouped([x], x, 1.0), lambda: dobb.dobb_mx4_quantize(x),
                 lambda: dobb.dobb_mx4_dequantize(x, x, 1)):
        with pytest.raises(TypeError, match="GPU tensor"):
            call()
    with pytest.raises(ValueError, match="same number"):
        dobb.dobb_accumulate_moment_mx4_grouped([], [], [], [], 1)
    assert [dobb.mx4_tiles(n) for n in (1, 128, 129, 16384)] == [1, 1, 2, 128]


def test_optimizer_options_are_checked():
    from block_diagonal_eigenbasis_amd.optimizer import Dobb, clip_grad_norm_
    w = torch.nn.Parameter(torch.zeros(4, 4))
    with pytest.raises(ValueError, match="capture_format"):
        Dobb([w], blocks=1, capture_format="fp4")
    for bad in (-1.0, float("nan")):
        with pytest.raises(ValueError, match="max_grad_norm"):
            Dobb([w], blocks=1, max_grad_norm=bad)
    assert float(clip_grad_norm_([w], 1.0)) == 0.0               # no gradient anywhere
    w.grad = torch.zeros(4, 4)
    with pytest.raises(TypeError, match="GPU tensor"):
        clip_grad_norm_(w, 1.0)


def test_captures_are_checked():
    from block_diagonal_eigenbasis_amd.optimizer import Mx4Capture
    codes, scales = torch.zeros(2, 4, 6, 16, dtype=torch.uint8), torch.zeros(2, 6, 4, dtype=torch.uint8)
    assert Mx4Capture(codes, scales, (128, 100)).shape == (228, 6)
    for c, s, parts, err in [
        (codes, scales, (256, 1), ValueError), (codes, scales, (0, 200), ValueError), (codes, scales, (), ValueError),
        (codes[:, :2], scales, (200,), ValueError), (codes[:, 0], scales, (200,), ValueError),
        (codes, scales[:1], (200,), ValueError), (codes, scales[:, :5], (200,), ValueError),
        (codes[:, :, ::2], scales[:, ::2].contiguous(), (200,), ValueError),       # strided
        (codes[:1].expand(2, 4, 6, 16), scales, (200,), ValueError),
        (codes, scales[:1].expand(2, 6, 4), (200,), ValueError),
        (codes.int(), scales, (200,), TypeError), (codes, scales.to(torch.int8), (200,), TypeError),
    ]:
        with pytest.raises(err):
            Mx4Capture(c, s, parts)


def test_overlapping_captures_and_workspaces_are_refused():
    """Everything that reaches the overlap check below breaks it, so nothing is enqueued."""
    L = _ops._lib()
    X, C, S, A = 0x10000000, 0x20000000, 0x30000000, 0x40000000
    N, n, ld = 300, 40, 50                                       # 3 tiles: 7680 bytes of codes, 480 of scales
    xb = ((N - 1) * ld + n) * 4
    for x, c, s in [(X, X, S), (X, X + (xb // 16) * 16, S), (X, X - 7680 + 16, S), (X, C, X), (X, C, X + xb - 4),
                    (X, C, C), (X, C, C + 7680 - 4), (X, C, C - 480 + 4)]:
        assert L.dobb_mx4_quantize(N, n, x, 0, ld, c, s, None) == INVALID, (x, c, s)
        assert L.dobb_mx4_dequantize(N, n, c, s, x, 0, ld, None) == INVALID, (x, c, s)
    sh = _abi.Shape(1, 768, 192)
    need = dobb.dobb_moment_mx4_workspace_size([(1, 768, 192)], 64)
    for ws in (C, S, A, C - need + 256, A - need + 256, C + 64 * 64 * 768 - 256, A + 768 * 192 * 4 - 256):
        assert L.dobb_accumulate_moment_mx4(ctypes.byref(sh), C, S, 64, 8192, 0.5, A, ws, need, None) == INVALID, ws


@pytest.mark.parametrize("n,offset", [(5, 0), (16000, 0), (16000, 2)])
def test_captures_are_joined_whatever_their_size_and_offset(n, offset):
    from block_diagonal_eigenbasis_amd.optimizer import Mx4Capture
    g = torch.Generator().manual_seed(n + offset)

    def held(*shape):
        k = torch.Size(shape).numel()
        return torch.randint(0, 256, (k + offset,), dtype=torch.uint8, generator=g)[offset:].view(shape)
    caps = [Mx4Capture(held(t, 4, n, 16), held(t, n, 4), parts) for t, parts in ((8, (1000,)), (2, (100, 7)), (7, (896,)))]
    got = Mx4Capture.cat(caps)
    assert got.parts == (1000, 100, 7, 896) and got.shape == (2003, n)
    assert got.codes.shape == (17, 4, n, 16) and got.codes.is_contiguous() and got.scales.is_contiguous()
    at = 0
    for c in caps:
        assert torch.equal(got.codes[at:at + c.tiles], c.codes) and torch.equal(got.scales[at:at + c.tiles], c.scales)
        at += c.tiles
