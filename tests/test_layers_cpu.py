"""The C ABI of include/dobb_layers.h and its binding without a GPU: every declared entry point is exported, bad
arguments are refused on the host before anything is enqueued, and captures are joined and kept as documented.

Every C call below is invalid in at least one argument, so the non-null "device pointers" are never
dereferenced.
"""
import ctypes
import os
import re

import pytest
import torch

import block_diagonal_eigenbasis_amd as dobb
from block_diagonal_eigenbasis_amd import _abi, _layers
from block_diagonal_eigenbasis_amd.optimizer import Dobb, DobbGroup, Mx4Capture

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
X, Y, Z, W, V = 0x1000000, 0x2000000, 0x3000000, 0x4000000, 0x5000000
INVALID, SHAPE, DTYPE, WORKSPACE = -1, -2, -3, -4
BIG = 1 << 24


def test_library_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "dobb_layers.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(dobb_\w+)\s*\(", text)))
    assert len(names) == 11
    L = _layers._lib()
    assert not [n for n in names if not hasattr(L, n)]


def _norm(N=4, n=8, x=X, xt=0, ldx=8, w=W, b=W + 0x1000, wt=0, eps=1e-5, y=Y, yt=0, ldy=8, mean=Z, rstd=Z + 0x100):
    return _layers._lib().dobb_layer_norm(N, n, x, xt, ldx, w, b, wt, eps, y, yt, ldy, mean, rstd, None)


def test_layer_norm_refusals():
    nan, inf = float("nan"), float("inf")
    assert _norm(x=None) == INVALID and _norm(y=None) == INVALID
    assert _norm(N=0) == INVALID and _norm(n=0) == SHAPE and _norm(N=BIG + 1) == SHAPE and _norm(n=BIG + 1, ldx=BIG + 1, ldy=BIG + 1) == SHAPE
    assert _norm(ldx=7) == SHAPE and _norm(ldy=7) == SHAPE and _norm(ldx=1 << 60) == SHAPE and _norm(N=BIG, ldy=1 << 50) == SHAPE
    assert _norm(xt=2) == DTYPE and _norm(yt=-1) == DTYPE and _norm(wt=9) == DTYPE
    assert _norm(eps=-1e-9) == INVALID and _norm(eps=nan) == INVALID and _norm(eps=inf) == INVALID
    assert _norm(x=X + 2) == INVALID and _norm(y=Y + 1, yt=1) == INVALID and _norm(w=W + 2) == INVALID and _norm(mean=Z + 2) == INVALID
    assert _norm(y=X + 4) == INVALID and _norm(y=X, yt=1) == INVALID and _norm(y=X, ldy=9) == INVALID   # in place: the same layout only
    assert _norm(mean=X) == INVALID and _norm(rstd=Z + 4) == INVALID and _norm(mean=W) == INVALID


def _grad(N=4, n=8, dy=X, dyt=0, lddy=8, x=Y, xt=0, ldx=8, mean=Z, rstd=Z + 0x100, w=W, wt=0, dx=V, dxt=0, lddx=8, dw=V + 0x1000,
          db=V + 0x2000, gt=0, ws=0x9000000, wsb=1 << 20):
    return _layers._lib().dobb_layer_norm_backward(N, n, dy, dyt, lddy, x, xt, ldx, mean, rstd, w, wt, dx, dxt, lddx, dw, db, gt, ws, wsb, None)


def test_layer_norm_backward_refusals():
    for k in ("dy", "x", "dx", "mean", "rstd"):
        assert _grad(**{k: None}) == INVALID
    for k in ("dyt", "xt", "dxt", "wt", "gt"):
        assert _grad(**{k: 3}) == DTYPE
    for k in ("lddy", "ldx", "lddx"):
        assert _grad(**{k: 7}) == SHAPE
    assert _grad(N=0) == INVALID and _grad(n=0) == SHAPE and _grad(N=BIG + 1) == SHAPE
    assert _grad(dx=Y) == INVALID and _grad(dx=X, lddx=9) == INVALID and _grad(dw=V) == INVALID and _grad(db=V + 0x1000) == INVALID
    assert _grad(dw=W) == INVALID and _grad(ws=X & ~255) == INVALID
    assert _grad(ws=None) == WORKSPACE and _grad(ws=0x9000010) == WORKSPACE and _grad(wsb=16) == WORKSPACE
    size = _layers._lib().dobb_layer_norm_backward_workspace_size
    assert size(0, 8) == 0 and size(8, 0) == 0 and size(BIG + 1, 8) == 0
    assert size(16384, 1600) <= 512 * 2 * 1600 * 4 and size(BIG, 8) <= BIG * 8 * 4 // 64


def _op(rows=8, k=130, codes=X, scales=X + 0x100000, fmt=0):
    return _layers._CFp8Operand(codes, scales, rows, k, fmt)


def _quant(N=130, n=8, x=Z, xt=0, ldx=8, square=0, rows=None, cols="make"):
    cols = _op(n, N) if cols == "make" else cols
    ref = lambda o: None if o is None else ctypes.byref(o)  # noqa: E731
    return _layers._lib().dobb_fp8_quantize(N, n, x, xt, ldx, square, ref(rows), ref(cols), None)


def test_quantize_refusals():
    assert _quant(cols=None) == INVALID and _quant(x=None) == INVALID
    assert _quant(N=0) == INVALID and _quant(n=0) == SHAPE and _quant(ldx=7) == SHAPE and _quant(xt=5) == DTYPE
    assert _quant(cols=_op(9, 130)) == SHAPE and _quant(cols=_op(8, 131)) == SHAPE and _quant(rows=_op(8, 130, Y, Y + 0x100000)) == SHAPE
    assert _quant(cols=_op(fmt=2)) == DTYPE
    assert _quant(cols=_op(codes=None)) == INVALID and _quant(cols=_op(scales=None)) == INVALID
    assert _quant(cols=_op(codes=X + 8)) == INVALID and _quant(cols=_op(scales=X + 0x100002)) == INVALID
    assert _quant(rows=_op(130, 8, Y, Y + 0x100000, 1)) == DTYPE           # one format
    assert _quant(rows=_op(130, 8, X, Y)) == INVALID                       # operands over each other
    assert _quant(x=X + 64) == INVALID                                     # .. and over X
    assert _quant(N=BIG * 128, n=BIG, ldx=BIG, cols=_op(BIG, BIG * 128)) == SHAPE
    L = _layers._lib()
    a = ctypes.byref(_op())
    assert L.dobb_layer_norm_fp8(130, 8, Z, 0, 8, None, None, 0, 1e-5, None, Y, None, a, None) == INVALID
    assert L.dobb_layer_norm_fp8(130, 8, Z, 0, 8, None, None, 0, -1.0, Y, Y + 0x1000, None, a, None) == INVALID
    assert L.dobb_layer_norm_fp8(130, 8, Z, 0, 8, None, None, 0, 1e-5, X, Y + 0x1000, None, a, None) == INVALID
    assert L.dobb_layer_norm_fp8(130, 8, Z, 0, 8, None, None, 0, 1e-5, Y, Y + 0x1000, None, None, None) == INVALID


def test_dequantize_refusals():
    f = lambda op=None, t=0, out=Z, dt=0, ldo=130: _layers._lib().dobb_fp8_dequantize(ctypes.byref(op or _op()), t, out, dt, ldo, None)  # noqa: E731
    assert f(out=None) == INVALID and f(dt=2) == DTYPE and f(ldo=129) == SHAPE and f(t=1, ldo=7) == SHAPE and f(out=X) == INVALID
    assert f(_op(rows=0)) == SHAPE and f(_op(k=0)) == SHAPE and f(_op(rows=BIG + 1)) == SHAPE and f(_op(codes=None)) == INVALID
    assert _layers._lib().dobb_fp8_dequantize(None, 0, Z, 0, 130, None) == INVALID


def _mm(a=None, b=None, bias=W, bt=0, acc=0, out=Z, dt=0, ldo=16, ws=0x9000000, wsb=1 << 30):
    a, b = a or _op(), b or _op(16, 130, Y, Y + 0x100000)
    return _layers._lib().dobb_fp8_matmul(ctypes.byref(a), ctypes.byref(b), bias, bt, acc, out, dt, ldo, ws, wsb, None)


def test_matmul_refusals():
    assert _mm(a=_op(k=131)) == SHAPE and _mm(a=_op(rows=0)) == SHAPE and _mm(b=_op(16, 130, None, Y)) == INVALID
    assert _mm(a=_op(fmt=7)) == DTYPE and _mm(bt=4) == DTYPE and _mm(dt=3) == DTYPE
    assert _mm(out=None) == INVALID and _mm(ldo=15) == SHAPE and _mm(out=Z + 2) == INVALID
    assert _mm(out=X) == INVALID and _mm(out=Y + 0x100000) == INVALID and _mm(out=W) == INVALID
    size = _layers._lib().dobb_fp8_matmul_workspace_size
    assert size(0, 1, 1) == 0 and size(1, BIG + 1, 1) == 0 and size(1, 1, 0) == 0


def _moment(shapes=((1, 8, 4),), ops=None, N=130, beta=0.0, A=(Z,), ws=0x9000000, wsb=1 << 20, count=None):
    ops = [_op()] if ops is None else ops
    return _layers._lib().dobb_accumulate_moment_fp8_grouped(
        len(shapes) if count is None else count, (_abi.Shape * len(shapes))(*[_abi.Shape(*s) for s in shapes]),
        (_layers._CFp8Operand * len(ops))(*ops), N, beta, (ctypes.c_void_p * len(A))(*A), ws, wsb, None)


def test_moment_refusals():
    nan = float("nan")
    assert _moment(count=0) == INVALID and _moment(N=0) == INVALID and _moment(N=257) == INVALID
    assert _moment(beta=1.0) == INVALID and _moment(beta=-0.1) == INVALID and _moment(beta=nan) == INVALID
    assert _moment(shapes=((1, 8, 3),)) == SHAPE and _moment(shapes=((1, 12, 4),)) == SHAPE and _moment(shapes=((1, 8, 0),)) == SHAPE
    assert _moment(A=(None,)) == INVALID and _moment(A=(Z + 2,)) == INVALID and _moment(A=(X,)) == INVALID
    two = dict(shapes=((1, 8, 4), (1, 8, 8)), A=(Z, Z + 0x1000))
    assert _moment(**two, ops=[_op(), _op(fmt=1)]) == DTYPE and _moment(**two, ops=[_op(), _op(k=300)]) == INVALID
    assert _moment(shapes=two["shapes"], A=(Z, Z), ops=[_op(), _op()]) == INVALID
    long = dict(shapes=((1, 8, 4),), ops=[_op(k=1 << 20, codes=0x100000000, scales=0x200000000)], N=1 << 20)
    assert _moment(**long, ws=None) == WORKSPACE and _moment(**long, ws=0x9000010) == WORKSPACE and _moment(**long, wsb=64) == WORKSPACE
    size = dobb.dobb_moment_fp8_workspace_size
    assert size([(1, 8, 3)], 4) == 0 and size([(1, 8, 4)], 0) == 0 and size([(1, 8, 4)], 1) == 0
    L = _layers._lib()
    assert L.dobb_accumulate_moment_fp8(None, ctypes.byref(_op()), 1, 0.0, Z, None, 0, None) == INVALID


def test_python_refusals_without_a_gpu():
    x = torch.zeros(4, 8)
    op = dobb.Fp8Operand(torch.zeros(1, 8, 4, 16, dtype=torch.uint8), torch.zeros(1, 4, dtype=torch.uint8), 8, "e4m3")
    for call in (lambda: dobb.dobb_layer_norm(x), lambda: dobb.dobb_fp8_quantize(x), lambda: dobb.dobb_fp8_dequantize(op),
                 lambda: dobb.dobb_fp8_matmul(op, op), lambda: dobb.dobb_layer_norm_fp8(x),
                 lambda: dobb.dobb_layer_norm_backward(x, x, x[:, 0], x[:, 0]),
                 lambda: dobb.dobb_accumulate_moment_fp8(op, torch.zeros(1, 4, 4), 4), lambda: dobb.dobb_fp8_matmul(x, op),
                 lambda: dobb.dobb_layer_norm("x"), lambda: dobb.dobb_layer_norm(x, dtype=torch.float16)):
        with pytest.raises(TypeError):
            call()


def _capture(N, n, fmt="e4m3", seed=0):
    g = torch.Generator()
    g.manual_seed(seed)
    T = dobb.fp8_tiles(N)
    return dobb.Fp8Capture(dobb.Fp8Operand(torch.randint(0, 256, (T, 8, n, 16), generator=g, dtype=torch.uint8),
                                           torch.randint(0, 256, (T, (n + 3) // 4 * 4), generator=g, dtype=torch.uint8), N, fmt))


def test_capture_checks_and_cat():
    c = _capture(200, 6)
    assert c.shape == (200, 6) and c.tiles == 2 and c.parts == (200,)
    d = _capture(57, 6, seed=1)
    joined = dobb.Fp8Capture.cat([c, d, c])
    assert joined.parts == (200, 57, 200) and joined.tiles == 5 and joined.shape == (457, 6) and joined.operand.K == 128 * 3 + 200
    assert torch.equal(joined.operand.codes, torch.cat([c.operand.codes, d.operand.codes, c.operand.codes]))
    assert torch.equal(joined.operand.scales, torch.cat([c.operand.scales, d.operand.scales, c.operand.scales]))
    assert dobb.Fp8Capture.cat([c]) is c
    for bad in ([], [c, _capture(57, 7)], [c, _capture(57, 6, "e5m2")]):
        with pytest.raises(ValueError):
            dobb.Fp8Capture.cat(bad)
    codes, scales, K, fmt = c.operand
    for op, parts in (((codes, scales[:, :4], K, fmt), None), ((codes[:, :4], scales, K, fmt), None), ((codes, scales, 300, fmt), None),
                      ((codes, scales, K, "fp8"), None), ((codes, scales, K, fmt), (100,)), ((codes, scales, K, fmt), ()),
                      ((codes, scales, K, fmt), (128, 0)), ((codes.transpose(2, 3), scales, K, fmt), None)):
        with pytest.raises(ValueError):
            dobb.Fp8Capture(dobb.Fp8Operand(*op), parts)
    with pytest.raises(TypeError):
        dobb.Fp8Capture(dobb.Fp8Operand(codes.float(), scales, K, fmt))
    # whole words or not, the bytes are the same
    odd = torch.empty(2 * 8 * 6 * 16 + 1, dtype=torch.uint8)[1:].view(2, 8, 6, 16)
    odd.copy_(codes)
    assert torch.equal(dobb.Fp8Capture.cat([dobb.Fp8Capture(dobb.Fp8Operand(odd, scales, K, fmt)), d]).operand.codes,
                       torch.cat([codes, d.operand.codes]))


def test_optimizer_keeps_captures_that_are_held_already(monkeypatch):
    p = torch.nn.Parameter(torch.zeros(8, 6))
    opt = Dobb([p], block_size=3, capture="all", capture_format="fp8")
    c = _capture(57, 6)
    opt.capture(p, c)
    assert opt._captured[id(p)] == [c]
    seen = []
    monkeypatch.setattr(dobb.Fp8Capture, "quantize", classmethod(lambda cls, x: seen.append(tuple(x.shape)) or _capture(x.shape[0], 6)))
    opt.capture(p, torch.zeros(2, 5, 6))
    assert seen == [(10, 6)] and len(opt._captured[id(p)]) == 2
    opt.capture(p, torch.zeros(0, 6))
    assert len(opt._captured[id(p)]) == 2
    mx = Mx4Capture(torch.zeros(1, 4, 6, 16, dtype=torch.uint8), torch.zeros(1, 6, 4, dtype=torch.uint8), (5,))
    with pytest.raises(ValueError):
        opt.capture(p, mx)
    first = Dobb([p], block_size=3)
    first.capture(p, c)
    first.capture(p, torch.zeros(4, 6))                          # the first of a refresh iteration is kept
    assert first._captured[id(p)] == [c]
    with pytest.raises(ValueError):
        Dobb([p], block_size=3, capture_format="fp4")


def test_group_plans_fp8_captures():
    ws = [torch.zeros(8, 6), torch.zeros(4, 6), torch.zeros(4, 9)]
    g = DobbGroup(ws, [3, 3, 3])
    xs = [_capture(300, 6), torch.zeros(300, 6), _capture(300, 9)]
    (plan,) = g._plan(xs).values()
    assert plan.fp8 == [[0, 2]] and plan.dense == [[1]] and plan.mx4 == []
    xs[2] = _capture(300, 9, "e5m2")
    (plan,) = g._plan(xs).values()
    assert plan.fp8 == [[0], [2]]
    for bad in (_capture(300, 6), dobb.Fp8Capture.cat([_capture(1, 8)])):
        with pytest.raises(ValueError):
            g._plan([xs[0], xs[1], bad])
