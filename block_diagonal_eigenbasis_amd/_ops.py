"""ctypes binding of the operators around the Dobb step (include/dobb_ops.h), with the C names.

Argument marshalling and checks, as in ``_abi``: gradient norms and clipping over lists of tensors, and
captures held in MXFP4.  Work runs on ``stream`` (default: torch's current stream of the tensors' own
device); tensors and workspaces that a call allocates are recorded on a stream that is passed in.
"""
from __future__ import annotations

import ctypes
from contextlib import contextmanager

import torch

from . import _abi
from ._abi import Shape, _check, _dtype_code, _ptrs

_bound = False


def _lib() -> ctypes.CDLL:
    global _bound
    L = _abi.lib()
    if not _bound:
        vp, sz, i64, f32, ci = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_float, ctypes.c_int
        P = ctypes.POINTER
        nl = [ci, P(i64), P(vp), P(ci)]
        L.dobb_grad_norm_workspace_size.argtypes = [ci, P(i64), P(ci)]
        L.dobb_grad_norm_workspace_size.restype = sz
        L.dobb_grad_norm_grouped.argtypes = nl + [vp, vp, vp, sz, vp]
        L.dobb_clip_grads_grouped.argtypes = nl + [P(vp), P(ci), vp, f32, vp]
        L.dobb_clip_grad_norm_grouped.argtypes = nl + [P(vp), P(ci), f32, vp, vp, vp, sz, vp]
        L.dobb_mx4_quantize.argtypes = [i64, i64, vp, ci, i64, vp, vp, vp]
        L.dobb_mx4_dequantize.argtypes = [i64, i64, vp, vp, vp, ci, i64, vp]
        L.dobb_moment_mx4_workspace_size.argtypes = [ci, P(Shape), i64]
        L.dobb_moment_mx4_workspace_size.restype = sz
        L.dobb_accumulate_moment_mx4.argtypes = [P(Shape), vp, vp, i64, i64, f32, vp, vp, sz, vp]
        L.dobb_accumulate_moment_mx4_grouped.argtypes = [ci, P(Shape), P(vp), P(vp), i64, i64, f32, P(vp), vp, sz, vp]
        for name in ("dobb_grad_norm_grouped", "dobb_clip_grads_grouped", "dobb_clip_grad_norm_grouped", "dobb_mx4_quantize",
                     "dobb_mx4_dequantize", "dobb_accumulate_moment_mx4", "dobb_accumulate_moment_mx4_grouped"):
            getattr(L, name).restype = ci
        _bound = True
    return L


@contextmanager
def _on(device: torch.device, stream, *made):
    """The stream handle for work on `device`, with that device current; the tensors `made` for the call
    are kept from reuse until a stream that was passed in is done with them."""
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream(device).cuda_stream
            return
        # what was allocated here may still be in use by earlier work of the current stream
        if made and stream != torch.cuda.current_stream(device):
            stream.wait_stream(torch.cuda.current_stream(device))
        yield stream.cuda_stream
        for t in made:
            if t is not None:
                t.record_stream(stream)


def _gpu(t, name: str, device=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return t


def _held(t, name: str, dtype, shape, device) -> torch.Tensor:
    _gpu(t, name, device)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _space(nbytes: int, device, ws):
    """(workspace tensor or None, whether it was made here)."""
    if nbytes == 0:
        return None, None
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        return ws, ws
    _gpu(ws, "ws", device)
    if ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 tensor")
    if ws.numel() < nbytes:
        raise ValueError(f"workspace too small: {ws.numel()} < {nbytes} bytes")
    return ws, None


# ---- gradient norm and clipping ------------------------------------------------------------------
class _List:
    """A list of dense tensors on one device, marshalled."""

    def __init__(self, ts, name: str, device=None):
        ts = list(ts)
        if not ts:
            raise ValueError(f"{name}: the list is empty")
        self.device = _gpu(ts[0], name).device if device is None else device
        codes = []
        for t in ts:
            _gpu(t, name, self.device)
            if not t.is_contiguous():
                raise ValueError(f"{name}: every tensor must be contiguous")
            codes.append(_dtype_code(t))
        self.ts = ts
        self.count = len(ts)
        self.numel = (ctypes.c_int64 * self.count)(*[t.numel() for t in ts])
        self.dtypes = (ctypes.c_int * self.count)(*codes)
        self.ptrs = _ptrs(ts)


def _norm_outputs(lst: _List, norms, total):
    made = []
    if norms is not None:
        _held(norms, "norms", torch.float32, (lst.count,), lst.device)
    if total is None:
        total = torch.empty((), dtype=torch.float32, device=lst.device)
        made.append(total)
    else:
        _gpu(total, "total", lst.device)
        if total.dtype != torch.float32 or total.numel() != 1:
            raise ValueError("total must be a float32 tensor of one entry")
    return total, made


def _outs_of(lst: _List, outs) -> _List:
    if outs is None:
        return lst
    o = _List(outs, "outs", lst.device)
    if o.count != lst.count or any(a.shape != b.shape for a, b in zip(o.ts, lst.ts)):
        raise ValueError("outs must have the gradients' shapes")
    return o


def dobb_grad_norm_grouped(Gs, norms: torch.Tensor | None = None, total: torch.Tensor | None = None,
                           ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The l2 norm of all entries of the list Gs (contiguous, fp32 or bf16, mixed; a tensor listed twice
    counts twice) into `total` (fp32 scalar, returned) and, if given, each tensor's into `norms` (fp32,
    one entry a tensor).  Sums are formed in fp64.  Nothing is synchronized."""
    g = _List(Gs, "Gs")
    total, made = _norm_outputs(g, norms, total)
    L = _lib()
    ws, own = _space(int(L.dobb_grad_norm_workspace_size(g.count, g.numel, g.dtypes)), g.device, ws)
    with _on(g.device, stream, *made, own) as sh:
        _check(L.dobb_grad_norm_grouped(g.count, g.numel, g.ptrs, g.dtypes, None if norms is None else norms.data_ptr(),
                                        total.data_ptr(), ws.data_ptr(), ws.numel(), sh), "dobb_grad_norm_grouped")
    return total


def dobb_clip_grads_grouped(Gs, total: torch.Tensor, max_norm: float, outs=None, stream=None):
    """outs[i] <- Gs[i] * min(1, max_norm / (total + 1e-6)), in place without outs; total is a device
    scalar (fp32).  Buffers written may not overlap: a tensor listed twice in place is refused."""
    g = _List(Gs, "Gs")
    o = _outs_of(g, outs)
    total, _ = _norm_outputs(g, None, total if total is not None else _gpu(total, "total"))
    with _on(g.device, stream) as sh:
        _check(_lib().dobb_clip_grads_grouped(g.count, g.numel, g.ptrs, g.dtypes, o.ptrs, o.dtypes, total.data_ptr(),
                                              float(max_norm), sh), "dobb_clip_grads_grouped")
    return o.ts


def dobb_clip_grad_norm_grouped(Gs, max_norm: float, outs=None, norms: torch.Tensor | None = None,
                                total: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                                stream=None) -> torch.Tensor:
    """dobb_grad_norm_grouped, then dobb_clip_grads_grouped with its total, in one call; returns total
    (the norm before clipping)."""
    g = _List(Gs, "Gs")
    o = _outs_of(g, outs)
    total, made = _norm_outputs(g, norms, total)
    L = _lib()
    ws, own = _space(int(L.dobb_grad_norm_workspace_size(g.count, g.numel, g.dtypes)), g.device, ws)
    with _on(g.device, stream, *made, own) as sh:
        _check(L.dobb_clip_grad_norm_grouped(g.count, g.numel, g.ptrs, g.dtypes, o.ptrs, o.dtypes, float(max_norm),
                                             None if norms is None else norms.data_ptr(), total.data_ptr(), ws.data_ptr(),
                                             ws.numel(), sh), "dobb_clip_grad_norm_grouped")
    return total


# ---- captures in MXFP4 -----------------------------------------------------------------------------
MX4_TILE = 128


def mx4_tiles(N: int) -> int:
    """Tiles of 128 tokens that N tokens take."""
    return -(-int(N) // MX4_TILE)


def _rows(x: torch.Tensor, name: str):
    """(tokens, columns, row stride) of a 2-D tensor with unit column stride."""
    if x.dim() != 2:
        raise ValueError(f"{name} must be (tokens x columns)")
    N, n = x.shape
    if N < 1 or n < 1:
        raise ValueError(f"{name} must hold at least one token and one column")
    ld = x.stride(0) if N > 1 else max(x.stride(0), n)
    if (n > 1 and x.stride(1) != 1) or ld < n:
        raise ValueError(f"{name} must have unit column stride and rows that do not overlap")
    return N, n, ld


def _codes_of(codes, scales, device=None):
    """(tiles, columns) of a capture's tensors, checked."""
    _gpu(codes, "codes", device)
    if codes.dim() != 4 or codes.shape[1] != 4 or codes.shape[3] != 16:
        raise ValueError("codes must have shape (tiles, 4, columns, 16)")
    T, _, n, _ = codes.shape
    _held(codes, "codes", torch.uint8, (T, 4, n, 16), codes.device)
    _held(scales, "scales", torch.uint8, (T, n, 4), codes.device)
    return T, n


def dobb_mx4_quantize(X: torch.Tensor, codes: torch.Tensor | None = None, scales: torch.Tensor | None = None, stream=None):
    """(codes, scales) of X (N x n, fp32 or bf16, any row stride) in MXFP4: uint8 (T, 4, n, 16) and
    (T, n, 4) with T = mx4_tiles(N); given tensors are written (slices of tiles of a larger capture, say)."""
    _gpu(X, "X")
    N, n, ld = _rows(X, "X")
    dt = _dtype_code(X)
    T = mx4_tiles(N)
    made = []
    if codes is None:
        codes = torch.empty(T, 4, n, 16, dtype=torch.uint8, device=X.device)
        made.append(codes)
    if scales is None:
        scales = torch.empty(T, n, 4, dtype=torch.uint8, device=X.device)
        made.append(scales)
    _held(codes, "codes", torch.uint8, (T, 4, n, 16), X.device)
    _held(scales, "scales", torch.uint8, (T, n, 4), X.device)
    with _on(X.device, stream, *made) as sh:
        _check(_lib().dobb_mx4_quantize(N, n, X.data_ptr(), dt, ld, codes.data_ptr(), scales.data_ptr(), sh), "dobb_mx4_quantize")
    return codes, scales


def dobb_mx4_dequantize(codes: torch.Tensor, scales: torch.Tensor, N: int, dtype: torch.dtype = torch.float32,
                        out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The first N tokens of a capture as values (N x n; fp32 or bf16, or the type of `out`)."""
    T, n = _codes_of(codes, scales)
    N = int(N)
    if N < 1 or mx4_tiles(N) > T:
        raise ValueError(f"N must be from 1 to {T * MX4_TILE}")
    made = []
    if out is None:
        out = torch.empty(N, n, dtype=dtype, device=codes.device)
        made.append(out)
    _gpu(out, "out", codes.device)
    if tuple(out.shape) != (N, n):
        raise ValueError(f"out must have shape {(N, n)}, got {tuple(out.shape)}")
    _, _, ld = _rows(out, "out")
    dt = _dtype_code(out)
    with _on(codes.device, stream, *made) as sh:
        _check(_lib().dobb_mx4_dequantize(N, n, codes.data_ptr(), scales.data_ptr(), out.data_ptr(), dt, ld, sh),
               "dobb_mx4_dequantize")
    return out


def dobb_moment_mx4_workspace_size(shapes, tiles: int) -> int:
    arr = (Shape * len(shapes))(*[Shape(*s) for s in shapes])
    return int(_lib().dobb_moment_mx4_workspace_size(len(shapes), arr, int(tiles)))


def dobb_accumulate_moment_mx4_grouped(codes, scales, As, nbs, N: int, beta: float = 0.0, ws: torch.Tensor | None = None,
                                       stream=None):
    """As[i] (B x nb x nb fp32, symmetric) <- beta As[i] + (1 - beta)/N sum over all tiles of capture i;
    N is the number of tokens every capture holds, and all have the same number of tiles."""
    codes, scales, As, nbs = list(codes), list(scales), list(As), [int(b) for b in nbs]
    count = len(codes)
    if not count or not (len(scales) == len(As) == len(nbs) == count):
        raise ValueError("codes, scales, As and nbs need the same number of entries, at least one")
    device = _gpu(codes[0], "codes").device
    shapes, T = [], None
    for c, s, A, nb in zip(codes, scales, As, nbs):
        t, n = _codes_of(c, s, device)
        if T is not None and t != T:
            raise ValueError("all captures of a group need the same number of tiles")
        T = t
        if nb < 1 or n % nb:
            raise ValueError(f"block size {nb} does not divide {n}")
        _held(A, "A", torch.float32, (n // nb, nb, nb), device)
        shapes.append((1, n, nb))
    sarr = (Shape * count)(*[Shape(*s) for s in shapes])
    L = _lib()
    ws, own = _space(int(L.dobb_moment_mx4_workspace_size(count, sarr, T)), device, ws)
    with _on(device, stream, own) as sh:
        _check(L.dobb_accumulate_moment_mx4_grouped(count, sarr, _ptrs(codes), _ptrs(scales), T, int(N), float(beta),
                                                    _ptrs(As), None if ws is None else ws.data_ptr(),
                                                    0 if ws is None else ws.numel(), sh),
               "dobb_accumulate_moment_mx4_grouped")
    return As


def dobb_accumulate_moment_mx4(codes: torch.Tensor, scales: torch.Tensor, A: torch.Tensor, nb: int, N: int,
                               beta: float = 0.0, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dobb_accumulate_moment from a capture held in MXFP4 (dobb_mx4_quantize) of N tokens."""
    return dobb_accumulate_moment_mx4_grouped([codes], [scales], [A], [nb], N, beta, ws, stream)[0]
