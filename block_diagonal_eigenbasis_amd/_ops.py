"""The operators around the Dobb step (include/dobb_ops.h), with the C names: gradient norms and clipping
over lists of tensors, and captures held in MXFP4.

Tensors are checked and marshalled by a small native module (csrc/host_ops.cpp), so that a list of some
hundred gradients costs microseconds of host time.  Work runs on torch's current stream of the tensors'
own device; with ``stream`` it runs, and what the call allocates is allocated, on that stream.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import _abi
from ._abi import Shape, _check

_HOST_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_dobb_host.so")
_bound = False
_module = None


def _host():
    """The native marshalling module (raises if it has not been built)."""
    global _module
    if _module is None:
        _abi.lib()
        if not os.path.exists(_HOST_PATH):
            raise RuntimeError(f"{_HOST_PATH} is missing: build it with __graft_entry__.build()")
        from . import _dobb_host
        _module = _dobb_host
    return _module


def _lib() -> ctypes.CDLL:
    """libdobb.so with the C entry points of dobb_ops.h declared."""
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


def _call(fn, stream, of, *args):
    """fn(of, *args) with `stream` current; what it returns beside the status is then kept from reuse until
    the stream that was current before is done with it.  `of` is a tensor or a list of them."""
    if stream is None:
        return fn(of, *args)
    if not isinstance(of, torch.Tensor):
        of = list(of)
    first = of if isinstance(of, torch.Tensor) else of[0] if of else None
    if isinstance(first, torch.Tensor) and first.device != stream.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {first.device}")
    with torch.cuda.device(stream.device):
        before = torch.cuda.current_stream()
        with torch.cuda.stream(stream):
            got = fn(of, *args)
    if isinstance(got, tuple):
        for t in got[1:]:
            if t is not None:
                t.record_stream(before)
    return got


# ---- gradient norm and clipping ------------------------------------------------------------------
def dobb_grad_norm_grouped(Gs, norms: torch.Tensor | None = None, total: torch.Tensor | None = None,
                           ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The l2 norm of all entries of the list Gs (contiguous, fp32 or bf16, mixed; a tensor listed twice
    counts twice) into `total` (fp32 scalar, returned) and, if given, each tensor's into `norms` (fp32,
    one entry a tensor).  Sums are formed in fp64.  Nothing is synchronized."""
    st, total = _call(_host().grads, stream, Gs, 0, None, 0.0, norms, total, ws)
    _check(st, "dobb_grad_norm_grouped")
    return total


def dobb_clip_grads_grouped(Gs, total: torch.Tensor, max_norm: float, outs=None, stream=None) -> None:
    """outs[i] <- Gs[i] * min(1, max_norm / (total + 1e-6)), in place without outs; total is a device
    scalar (fp32).  Buffers written may not overlap: a tensor listed twice in place is refused."""
    st, _ = _call(_host().grads, stream, Gs, 1, outs, max_norm, None, total, None)
    _check(st, "dobb_clip_grads_grouped")


def dobb_clip_grad_norm_grouped(Gs, max_norm: float, outs=None, norms: torch.Tensor | None = None,
                                total: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                                stream=None) -> torch.Tensor:
    """dobb_grad_norm_grouped, then dobb_clip_grads_grouped with its total, in one call; returns total
    (the norm before clipping)."""
    st, total = _call(_host().grads, stream, Gs, 2, outs, max_norm, norms, total, ws)
    _check(st, "dobb_clip_grad_norm_grouped")
    return total


# ---- captures in MXFP4 -----------------------------------------------------------------------------
MX4_TILE = 128


def mx4_tiles(N: int) -> int:
    """Tiles of 128 tokens that N tokens take."""
    return -(-int(N) // MX4_TILE)


def dobb_mx4_quantize(X: torch.Tensor, codes: torch.Tensor | None = None, scales: torch.Tensor | None = None, stream=None):
    """(codes, scales) of X (N x n, fp32 or bf16, any row stride) in MXFP4: uint8 (T, 4, n, 16) and
    (T, n, 4) with T = mx4_tiles(N); given tensors are written (slices of tiles of a larger capture, say)."""
    st, codes, scales = _call(_host().mx4_quantize, stream, X, codes, scales)
    _check(st, "dobb_mx4_quantize")
    return codes, scales


def dobb_mx4_dequantize(codes: torch.Tensor, scales: torch.Tensor, N: int, dtype: torch.dtype = torch.float32,
                        out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The first N tokens of a capture as values (N x n; fp32 or bf16, or the type of `out`)."""
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    st, out = _call(_host().mx4_dequantize, stream, codes, scales, N, dtype == torch.bfloat16, out)
    _check(st, "dobb_mx4_dequantize")
    return out


def dobb_moment_mx4_workspace_size(shapes, tiles: int) -> int:
    arr = (Shape * len(shapes))(*[Shape(*s) for s in shapes])
    return int(_lib().dobb_moment_mx4_workspace_size(len(shapes), arr, int(tiles)))


def dobb_accumulate_moment_mx4_grouped(codes, scales, As, nbs, N: int, beta: float = 0.0, ws: torch.Tensor | None = None,
                                       stream=None) -> None:
    """As[i] (B x nb x nb fp32, symmetric) <- beta As[i] + (1 - beta)/N sum over all tiles of capture i;
    N is the number of tokens every capture holds, and all have the same number of tiles.  beta is rounded to
    fp32 (0.9 to 0.9f: 1 - beta then differs by 2.4e-7 relative), as in dobb_accumulate_moment."""
    _check(_call(_host().moment_mx4, stream, codes, scales, As, nbs, N, beta, ws), "dobb_accumulate_moment_mx4_grouped")


def dobb_accumulate_moment_mx4(codes: torch.Tensor, scales: torch.Tensor, A: torch.Tensor, nb: int, N: int,
                               beta: float = 0.0, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dobb_accumulate_moment from a capture held in MXFP4 (dobb_mx4_quantize) of N tokens."""
    _check(_call(_host().moment_mx4, stream, (codes,), (scales,), (A,), (nb,), N, beta, ws), "dobb_accumulate_moment_mx4")
    return A
