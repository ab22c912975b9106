"""The operators of the layers whose weights Dobb trains (include/dobb_layers.h), with the C names: layer norm
forward and backward, FP8 operands and their products, and second moments from operands held as captures.

A training step of a layer norm and a linear map y = norm(x) W^T behind it::

    xr, xc, mean, rstd = dobb_layer_norm_fp8(x, g, b, rows=True, cols=True)
    wr, wc = dobb_fp8_quantize(W, cols=True, square=True)                  # once for each optimizer step
    y = dobb_fp8_matmul(xr, wr, bias=c)
    # backward, from the output gradient dy
    dr, dc = dobb_fp8_quantize(dy, cols=True, fmt="e5m2")
    dh = dobb_fp8_matmul(dr, wc)                                          # gradient of norm(x)
    dW = dobb_fp8_matmul(dc, xc, dtype=torch.float32)
    dx, dg, db = dobb_layer_norm_backward(dh, x, mean, rstd, g)
    # xc is also the capture whose second moment the weight's basis is taken from
    optimizer.capture(W, Fp8Capture(xc))

Tensors are checked and marshalled by the native module (csrc/host_ops.cpp).  Work runs on torch's current
stream of the tensors' own device; with ``stream`` it runs, and what the call allocates is allocated, on
that stream.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _abi
from ._abi import Shape, _check
from ._ops import _call, _host

FP8_TILE = 128


class Fp8Operand(NamedTuple):
    """An FP8 operand of a product: `rows` rows of K entries in tiles of 128 (layout: include/dobb_layers.h)."""
    codes: torch.Tensor        # uint8 (tiles, 8, rows, 16)
    scales: torch.Tensor       # uint8 (tiles, rows rounded up to fours)
    K: int
    fmt: str                   # "e4m3" or "e5m2"

    @property
    def rows(self) -> int:
        return self.codes.shape[2]

    @property
    def tiles(self) -> int:
        return self.codes.shape[0]

    @property
    def tokens(self) -> int:
        """Entries of a row that are no padding: K, but for the operand of a capture of several micro-batches."""
        return self.K


class _JoinedOperand(Fp8Operand):
    """The operand of a capture whose K counts the padding of every micro-batch but the last."""

    @property
    def tokens(self) -> int:
        return self._tokens

    def _replace(self, **kw):
        new = super()._replace(**kw)
        new._tokens = self._tokens
        return new


class _CFp8Operand(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64), ("k", ctypes.c_int64),
                ("format", ctypes.c_int)]


def _c_operand(op: Fp8Operand) -> _CFp8Operand:
    return _CFp8Operand(op.codes.data_ptr(), op.scales.data_ptr(), op.rows, op.K, 1 if op.fmt == "e5m2" else 0)


_bound = False


def _lib() -> ctypes.CDLL:
    """libdobb.so with the C entry points of dobb_layers.h declared."""
    global _bound
    L = _abi.lib()
    if not _bound:
        vp, sz, i64, i32, f32, ci = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_int
        P, op = ctypes.POINTER, ctypes.POINTER(_CFp8Operand)
        norm = [i64, i64, vp, ci, i64, vp, vp, ci, f32]
        L.dobb_layer_norm.argtypes = norm + [vp, ci, i64, vp, vp, vp]
        L.dobb_layer_norm_fp8.argtypes = norm + [vp, vp, op, op, vp]
        L.dobb_layer_norm_backward_workspace_size.argtypes = [i64, i64]
        L.dobb_layer_norm_backward_workspace_size.restype = sz
        L.dobb_layer_norm_backward.argtypes = [i64, i64, vp, ci, i64, vp, ci, i64, vp, vp, vp, ci, vp, ci, i64, vp, vp, ci, vp, sz, vp]
        L.dobb_fp8_quantize.argtypes = [i64, i64, vp, ci, i64, i32, op, op, vp]
        L.dobb_fp8_dequantize.argtypes = [op, i32, vp, ci, i64, vp]
        L.dobb_fp8_matmul_workspace_size.argtypes = [i64, i64, i64]
        L.dobb_fp8_matmul_workspace_size.restype = sz
        L.dobb_fp8_matmul.argtypes = [op, op, vp, ci, i32, vp, ci, i64, vp, sz, vp]
        L.dobb_moment_fp8_workspace_size.argtypes = [ci, P(Shape), i64]
        L.dobb_moment_fp8_workspace_size.restype = sz
        L.dobb_accumulate_moment_fp8.argtypes = [P(Shape), op, i64, f32, vp, vp, sz, vp]
        L.dobb_accumulate_moment_fp8_grouped.argtypes = [ci, P(Shape), op, i64, f32, P(vp), vp, sz, vp]
        for name in ("dobb_layer_norm", "dobb_layer_norm_fp8", "dobb_layer_norm_backward", "dobb_fp8_quantize", "dobb_fp8_dequantize",
                     "dobb_fp8_matmul", "dobb_accumulate_moment_fp8", "dobb_accumulate_moment_fp8_grouped"):
            getattr(L, name).restype = ci
        _bound = True
    return L


def _bf16(dtype, default: int = 0) -> int:
    if dtype is None:
        return default
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    return int(dtype == torch.bfloat16)


def _of(fn, stream, op, *args):
    """fn(*args) on `stream` (see _call), which has to be on the operand's device."""
    return _call(lambda _, *a: fn(*a), stream, op[0] if isinstance(op, tuple) and op else [], *args)


def _operands(got, N: int, n: int, fmt: str):
    rc, rs, cc, cs = got
    return (None if rc is None else Fp8Operand(rc, rs, n, fmt)), (None if cc is None else Fp8Operand(cc, cs, N, fmt))


# ---- layer norm ----------------------------------------------------------------------------------
def dobb_layer_norm(X: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, eps: float = 1e-5,
                    out: torch.Tensor | None = None, dtype: torch.dtype | None = None, mean: torch.Tensor | None = None,
                    rstd: torch.Tensor | None = None, stream=None):
    """(Y, mean, rstd): the layer norm over the columns of every row of X (rows x n, fp32 or bf16, any row
    stride).  weight and bias: n entries, fp32 or bf16, either may be left out.  Y is `out`, or new in `dtype`
    (default: X's); out=X works in place.  mean and rstd: fp32, one entry a row."""
    st, *got = _call(_host().layer_norm, stream, X, weight, bias, eps, out, _bf16(dtype, -1), mean, rstd)
    _check(st, "dobb_layer_norm")
    return tuple(got)


def dobb_layer_norm_fp8(X: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, eps: float = 1e-5,
                        rows: bool = True, cols: bool = False, fmt: str = "e4m3", rows_out: Fp8Operand | None = None,
                        cols_out: Fp8Operand | None = None, mean: torch.Tensor | None = None, rstd: torch.Tensor | None = None,
                        stream=None):
    """(rows, cols, mean, rstd): what dobb_layer_norm writes in X's type, as FP8 operands (see
    dobb_fp8_quantize, bit for bit), without that matrix in between."""
    st, *got = _call(_host().layer_norm_fp8, stream, X, weight, bias, eps, bool(rows), bool(cols), fmt, rows_out, cols_out, mean, rstd)
    _check(st, "dobb_layer_norm_fp8")
    return (*_operands(got[:4], *X.shape, fmt), got[4], got[5])


def dobb_layer_norm_backward(dY: torch.Tensor, X: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                             weight: torch.Tensor | None = None, dX: torch.Tensor | None = None, dtype: torch.dtype | None = None,
                             dweight: torch.Tensor | bool = True, dbias: torch.Tensor | bool = True, ws: torch.Tensor | None = None,
                             stream=None):
    """(dX, dweight, dbias): gradients of X, weight and bias for an output gradient dY, with the mean and rstd
    of the forward pass.  dX is the tensor given, or new in `dtype` (default: X's); dX=dY works in place.  dweight and
    dbias: a tensor to write (fp32 or bf16), True for a new one in the weight's type (fp32 without a weight),
    False for none."""
    given = [None if isinstance(g, bool) else g for g in (dweight, dbias)]
    st, *got = _call(_host().layer_norm_backward, stream, dY, X, mean, rstd, weight, dX, _bf16(dtype, -1), dweight is True, dbias is True,
                     *given, ws)
    _check(st, "dobb_layer_norm_backward")
    return tuple(got)


# ---- FP8 operands --------------------------------------------------------------------------------
def fp8_tiles(K: int) -> int:
    """Tiles of 128 entries that K entries take."""
    return -(-int(K) // FP8_TILE)


def dobb_fp8_quantize(X: torch.Tensor, rows: bool = True, cols: bool = False, fmt: str = "e4m3", square: bool = False,
                      rows_out: Fp8Operand | None = None, cols_out: Fp8Operand | None = None, stream=None):
    """(rows, cols): X (N x n, fp32 or bf16, any row stride) as FP8 operands from one read.  `rows` holds N rows
    of K = n entries, `cols` n rows of K = N (what a product along the tokens takes, and a capture); one that is
    not wanted is None.  A power of two scales 128 entries along K, or 128 x 128 with `square` (weights: both
    operands then hold the same values).  rows_out and cols_out: operands to write."""
    st, *got = _call(_host().fp8_quantize, stream, X, bool(rows), bool(cols), fmt, bool(square), rows_out, cols_out)
    _check(st, "dobb_fp8_quantize")
    return _operands(got, *X.shape, fmt)


def dobb_fp8_dequantize(op: Fp8Operand, dtype: torch.dtype = torch.float32, transpose: bool = False,
                        out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values of an operand (rows x K, or K x rows with `transpose`; fp32 or bf16, or the type of `out`)."""
    st, out = _of(_host().fp8_dequantize, stream, op, op, _bf16(dtype), bool(transpose), out)
    _check(st, "dobb_fp8_dequantize")
    return out


def dobb_fp8_matmul(A: Fp8Operand, B: Fp8Operand, out: torch.Tensor | None = None, dtype: torch.dtype = torch.bfloat16,
                    bias: torch.Tensor | None = None, accumulate: bool = False, ws: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """A B^T (+ bias) (+ out with `accumulate`), A.rows x B.rows, summed in fp32 and rounded once to `dtype`
    (fp32 or bf16) or the type of `out`.  bias: B.rows entries, fp32 or bf16."""
    st, out = _of(_host().fp8_matmul, stream, A, A, B, bias, out, _bf16(dtype), bool(accumulate), ws)
    _check(st, "dobb_fp8_matmul")
    return out


def dobb_fp8_matmul_workspace_size(M: int, N: int, K: int) -> int:
    return int(_lib().dobb_fp8_matmul_workspace_size(int(M), int(N), int(K)))


# ---- captures held in FP8 --------------------------------------------------------------------------
def dobb_moment_fp8_workspace_size(shapes, tiles: int) -> int:
    arr = (Shape * len(shapes))(*[Shape(*s) for s in shapes])
    return int(_lib().dobb_moment_fp8_workspace_size(len(shapes), arr, int(tiles)))


def dobb_accumulate_moment_fp8_grouped(ops, As, nbs, N: int, beta: float = 0.0, ws: torch.Tensor | None = None, stream=None) -> None:
    """As[i] (B x nb x nb fp32, symmetric) <- beta As[i] + (1 - beta)/N sum over all tiles of operand i, along the
    columns of a capture (dobb_fp8_quantize(cols=True)); N is the number of tokens every capture holds, and all have
    the same number of tiles and one format.  beta is rounded to fp32, as in dobb_accumulate_moment."""
    _check(_of(_host().moment_fp8, stream, ops[0] if len(ops) else None, ops, As, nbs, N, beta, ws), "dobb_accumulate_moment_fp8_grouped")


def dobb_accumulate_moment_fp8(op: Fp8Operand, A: torch.Tensor, nb: int, N: int | None = None, beta: float = 0.0,
                               ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dobb_accumulate_moment from a capture held as an FP8 operand along its columns, of N tokens (default: op.tokens, that
    is op.K; for the operand of an Fp8Capture of several micro-batches their tokens, without the padding between
    them)."""
    _check(_of(_host().moment_fp8, stream, op, (op,), (A,), (nb,), op.tokens if N is None else N, beta, ws), "dobb_accumulate_moment_fp8")
    return A


class Fp8Capture:
    """Captured activations or output gradients (tokens x n) held in FP8 along their columns, the operand that
    the weight's gradient takes too: 129/128 byte an entry instead of 2 or 4.  `parts` are the token counts of the
    micro-batches it holds, each from a tile of 128 tokens of its own (default: one, of operand.K tokens)."""

    def __init__(self, operand: Fp8Operand, parts=None):
        operand = Fp8Operand(*operand)
        self.operand = operand = operand._replace(K=int(operand.K))
        self.parts = (int(operand.K),) if parts is None else tuple(int(k) for k in parts)
        c, s = operand.codes, operand.scales
        T, n = (c.shape[0], c.shape[2]) if c.dim() == 4 else (0, 0)
        if tuple(c.shape) != (T, 8, n, 16) or tuple(s.shape) != (T, (n + 3) // 4 * 4):
            raise ValueError("codes must have shape (tiles, 8, columns, 16) and scales (tiles, columns rounded up to fours)")
        if c.dtype != torch.uint8 or s.dtype != torch.uint8:
            raise TypeError("codes and scales must be uint8")
        if not c.is_contiguous() or not s.is_contiguous() or s.device != c.device:
            raise ValueError("codes and scales must be contiguous, on one device")
        if operand.fmt not in ("e4m3", "e5m2"):
            raise ValueError('the format must be "e4m3" or "e5m2"')
        if not self.parts or any(k < 1 for k in self.parts) or sum(fp8_tiles(k) for k in self.parts) != T:
            raise ValueError("the tiles of the parts do not add up to those of the codes")
        if fp8_tiles(operand.K) != T:
            raise ValueError(f"K must be a number of entries that {T} tiles hold, the padding between parts counted; got {operand.K}")
        if sum(self.parts) != operand.K:
            self.operand = _JoinedOperand(*operand)
            self.operand._tokens = sum(self.parts)

    @classmethod
    def quantize(cls, x: torch.Tensor, fmt: str = "e4m3") -> "Fp8Capture":
        """(tokens x n) fp32 or bf16 -> FP8 (dobb_fp8_quantize).  Rows of any stride are read as they are; other
        layouts (a broadcast loss's gradient, a transposed input) are copied first."""
        if x.dim() == 2 and (x.is_neg() or (x.shape[1] > 1 and x.stride(1) != 1) or (x.shape[0] > 1 and x.stride(0) < x.shape[1])):
            x = x.resolve_neg().contiguous()
        return cls(dobb_fp8_quantize(x, rows=False, cols=True, fmt=fmt)[1])

    @classmethod
    def cat(cls, captures) -> "Fp8Capture":
        """Captures of several micro-batches as one."""
        captures = list(captures)
        if len(captures) == 1 and captures[0].aligned:
            return captures[0]
        if not captures or len({(c.shape[1], c.operand.fmt) for c in captures}) != 1:
            raise ValueError("captures of one width and format, at least one")
        parts = [k for c in captures for k in c.parts]
        codes, scales = [c.operand.codes for c in captures], [c.operand.scales for c in captures]
        # in words, which torch copies faster than bytes (both are whole words, tile by tile)
        if all(c.storage_offset() % 8 == 0 and s.storage_offset() % 4 == 0 for c, s in zip(codes, scales)):
            codes = torch.cat([c.view(torch.int64) for c in codes]).view(torch.uint8)
            scales = torch.cat([s.view(torch.int32) for s in scales]).view(torch.uint8)
        else:
            codes, scales = torch.cat(codes), torch.cat(scales)
        K = FP8_TILE * (codes.shape[0] - fp8_tiles(parts[-1])) + parts[-1]
        return cls(Fp8Operand(codes, scales, K, captures[0].operand.fmt), parts)

    def dequantize(self, dtype: torch.dtype = torch.float32) -> torch.Tensor:
        """The (tokens x n) values held (dobb_fp8_dequantize)."""
        out = torch.empty(*self.shape, dtype=dtype, device=self.device)
        tile = row = 0
        for k in self.parts:
            t = fp8_tiles(k)
            op = Fp8Operand(self.operand.codes[tile:tile + t], self.operand.scales[tile:tile + t], k, self.operand.fmt)
            dobb_fp8_dequantize(op, dtype, transpose=True, out=out[row:row + k])
            tile, row = tile + t, row + k
        return out

    @property
    def aligned(self) -> bool:
        """Whether the calls take the tensors as they lie (a copy, `cat`'s too, always is)."""
        return self.operand.codes.data_ptr() % 16 == 0 and self.operand.scales.data_ptr() % 4 == 0

    @property
    def shape(self):
        return (sum(self.parts), self.operand.rows)

    @property
    def tiles(self) -> int:
        return self.operand.tiles

    @property
    def device(self):
        return self.operand.codes.device
