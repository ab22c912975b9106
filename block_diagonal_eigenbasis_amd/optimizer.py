"""Dobb as a torch optimizer over a set of 2-D weights, driving libdobb.so's grouped entry points.

The cadence follows the Dobb paper (arXiv 2610.39412): second moments are captured on refresh
iterations only (Table 17: from the first micro-batch by default, or from all of them), the basis is
refreshed every T steps (Table 14; T = 9 in the principal runs), the first refresh is an exact
eigendecomposition and later ones warm-started orthogonal iteration with k = 1 (Table 15), the basis
may be stored in bf16 (Table 18's principal setting), and the update scale is tau sqrt(max(m, n)/m)
with tau = 0.2 (Table 9).  Dobb-G (Tables 12-13) takes the basis from the output-gradient second
moment instead, with blocks of rows: side="output" (update scale tau sqrt(max(m, n)/n), Table 9).

``DobbGroup`` keeps the optimizer state (M, A, Q) of a matrix set as device tensors, marshals the
per-matrix pointer tables once and owns its workspace, so a step is a handful of ctypes calls.  The
C ABI takes one dtype per argument of a grouped call, so the set is partitioned by weight dtype, and
activations and gradients of mixed dtypes (or token counts) are passed in one call per kind.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import torch

from . import _abi, _layers, _ops
from ._layers import Fp8Capture


def default_update_scale(m: int, n: int, tau: float = 0.2) -> float:
    return tau * math.sqrt(max(m, n) / m)


def default_update_scale_g(m: int, n: int, tau: float = 0.2) -> float:
    """Dobb-G (Table 9): RMS tau sqrt(max(m, n)/n) for the sign update."""
    return tau * math.sqrt(max(m, n) / n)


class Mx4Capture:
    """Captured activations or output gradients (tokens x n) held in MXFP4: 17/32 byte an entry instead of
    2 or 4, from the forward (or backward) pass to the refresh that takes their second moment.  `parts` are
    the token counts of the micro-batches it holds, each from a tile of 128 tokens of its own."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, parts):
        self.codes, self.scales, self.parts = codes, scales, tuple(int(k) for k in parts)
        T, n = (codes.shape[0], codes.shape[2]) if codes.dim() == 4 else (0, 0)
        if tuple(codes.shape) != (T, 4, n, 16) or tuple(scales.shape) != (T, n, 4):
            raise ValueError("codes must have shape (tiles, 4, columns, 16) and scales (tiles, columns, 4)")
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales must be uint8")
        if not codes.is_contiguous() or not scales.is_contiguous() or scales.device != codes.device:
            raise ValueError("codes and scales must be contiguous, on one device")
        if any(k < 1 for k in self.parts) or sum(_ops.mx4_tiles(k) for k in self.parts) != codes.shape[0]:
            raise ValueError("the tiles of the parts do not add up to those of the codes")

    @classmethod
    def quantize(cls, x: torch.Tensor) -> "Mx4Capture":
        """(tokens x n) fp32 or bf16 -> MXFP4 (dobb_mx4_quantize).  Rows of any stride are read as they are; other
        layouts (a broadcast loss's gradient, a transposed input) are copied first."""
        if x.dim() == 2 and (x.is_neg() or (x.shape[1] > 1 and x.stride(1) != 1) or (x.shape[0] > 1 and x.stride(0) < x.shape[1])):
            x = x.resolve_neg().contiguous()
        codes, scales = _ops.dobb_mx4_quantize(x)
        return cls(codes, scales, (x.shape[0],))

    @classmethod
    def cat(cls, captures) -> "Mx4Capture":
        """Captures of several micro-batches as one."""
        captures = list(captures)
        if len(captures) == 1 and captures[0].aligned:
            return captures[0]
        if not captures or len({c.shape[1] for c in captures}) != 1:
            raise ValueError("captures of one width, at least one")
        codes, scales, parts = [c.codes for c in captures], [c.scales for c in captures], [k for c in captures for k in c.parts]
        # torch copies bytes one a lane: 8193 tokens of 6400 columns in three parts take 43.1 us as bytes and 17.5 as
        # words, four parts of 4096 tokens 72.9 and 21.9.  Below 16 MB the views' host time is what counts: four
        # parts of 4096 tokens of 1600 columns (13 MB) 22.4 and 22.1, 8193 tokens of them 14.6 and 17.4.
        if sum(c.numel() for c in codes) >= 1 << 24 and all(
                c.storage_offset() % 8 == 0 and s.storage_offset() % 4 == 0 for c, s in zip(codes, scales)):
            return cls(torch.cat([c.view(torch.int64) for c in codes]).view(torch.uint8),
                       torch.cat([s.view(torch.int32) for s in scales]).view(torch.uint8), parts)
        return cls(torch.cat(codes), torch.cat(scales), parts)

    def dequantize(self, dtype: torch.dtype = torch.float32) -> torch.Tensor:
        """The (tokens x n) values held (dobb_mx4_dequantize)."""
        out = torch.empty(*self.shape, dtype=dtype, device=self.device)
        tile = row = 0
        for k in self.parts:
            t = _ops.mx4_tiles(k)
            _ops.dobb_mx4_dequantize(self.codes[tile:tile + t], self.scales[tile:tile + t], k, dtype, out=out[row:row + k])
            tile, row = tile + t, row + k
        return out

    @property
    def aligned(self) -> bool:
        """Whether the moment takes the tensors as they lie (a copy, `cat`'s too, always is)."""
        return self.codes.data_ptr() % 16 == 0 and self.scales.data_ptr() % 4 == 0

    @property
    def shape(self):
        return (sum(self.parts), self.codes.shape[2])

    @property
    def tiles(self) -> int:
        return self.codes.shape[0]

    @property
    def device(self):
        return self.codes.device


def clip_grad_norm_(parameters, max_norm: float) -> torch.Tensor:
    """Scale the gradients of the parameters (or one parameter) in place so that their global l2 norm is at
    most max_norm, by min(1, max_norm / (norm + 1e-6)); returns the norm before, as a scalar on their device.
    Gradients are contiguous, fp32 or bf16, on one device; parameters without one are passed over, a
    gradient shared by several counts once, and one that is part of another is refused.  Call it over a
    whole model's parameters where several optimizers share them (``Dobb(max_grad_norm=...)`` clips over
    its own).  The norm is this process's: it is the model's where every process holds all gradients, reduced.
    Where each holds a shard, take the shards' norms (dobb_grad_norm_grouped), combine them over the
    processes, and scale by the total (dobb_clip_grads_grouped)."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    grads, seen, device = [], set(), None
    for p in parameters:
        device = device or p.device
        g = p.grad
        if g is None:
            continue
        key = (g.device, g.data_ptr(), g.numel(), g.dtype)
        if g.numel() == 0 or key not in seen:
            seen.add(key)
            grads.append(g)
    if not grads:
        return torch.zeros((), dtype=torch.float32, device=device)
    return _ops.dobb_clip_grad_norm_grouped(grads, max_norm)


def _arr(ptrs):
    return (ctypes.c_void_p * len(ptrs))(*ptrs)


def _split(idx, key):
    """idx partitioned by key(i), in first-seen order."""
    out = {}
    for i in idx:
        out.setdefault(key(i), []).append(i)
    return list(out.values())


class _Part:
    """Pre-marshalled launch arguments and a workspace for a subset of a DobbGroup's weights (all of
    one weight dtype)."""

    def __init__(self, g: "DobbGroup", idx, stream):
        self.idx = list(idx)
        self.count = len(self.idx)
        self.stream = stream
        shapes = [g.shapes[i] for i in self.idx]
        self.shapes = shapes
        self.sh = (_abi.Shape * self.count)(*[_abi.Shape(*s) for s in shapes])
        # the moments and bases live on the captured axis: inputs (n) for Dobb, outputs (m) for Dobb-G
        self.cshapes = [(1, g.cap_dim(i), g.nb[i]) for i in self.idx]
        self.ash = (_abi.Shape * self.count)(*[_abi.Shape(*c) for c in self.cshapes])
        self.w_dtype = _abi._dtype_code(g.W[self.idx[0]])
        self.W = _arr([g.W[i].data_ptr() for i in self.idx])
        self.M = _arr([g.M[i].data_ptr() for i in self.idx])
        self.A = _arr([g.A[i].data_ptr() for i in self.idx])
        self.Q = _arr([g.Q[i].data_ptr() for i in self.idx])
        self.lam = _arr([g.lam[i].data_ptr() for i in self.idx])
        self.info = _arr([g.info[i].data_ptr() for i in self.idx])
        self.ldx = (ctypes.c_int64 * self.count)(*[c[1] for c in self.cshapes])
        self.hp = (_abi.HParams * self.count)(*[g.hp[i] for i in self.idx])
        self.device = g.device
        self.ws = torch.empty(max(self.need(g, g.n_tokens), 256), dtype=torch.uint8, device=self.device)

    def need(self, g, n_tokens):
        qv = _abi.DOBB_WS_BF16_BASIS if g.q_dtype == _abi.DOBB_BF16 else 0
        ash = self.cshapes
        return max(_abi.dobb_workspace_size(g.step_op, self.shapes, 0, g.norm | qv),
                   _abi.dobb_workspace_size(_abi.DOBB_OP_REFRESH, ash, 0, qv),
                   _abi.dobb_workspace_size(_abi.DOBB_OP_ACCUMULATE, ash, max(n_tokens, 1)))

    def reserve(self, nbytes, stream):
        """The workspace, of at least nbytes, for calls on `stream`.  A larger one is allocated in that stream's
        order, and one that was allocated in another stream's is recorded on it: what it leaves behind is not
        given away before every call that used it is done."""
        if nbytes > self.ws.numel():
            with torch.cuda.device(self.device), torch.cuda.stream(stream):
                self.ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self.ws.record_stream(stream)

    def refresh_hp(self, g):
        for k, i in enumerate(self.idx):
            self.hp[k] = g.hp[i]


class _Plan(NamedTuple):
    """The calls of one part that take a set of captures: lists of weights, and the bytes of workspace."""
    mx4: list
    fp8: list
    dense: list
    need: int


class DobbGroup:
    """Optimizer state and pre-marshalled launch arguments for a list of weights.

    streams=2 splits the set into the weights with blocks of at most 128 columns and the wider ones
    and runs the two on separate streams (each with its own workspace), joined back into the
    caller's stream: the two kernel families then overlap (the wide blocks' refresh is a chain of
    latency-bound panel launches).  basis_dtype=torch.bfloat16 stores every Q_b in bf16.
    side="output" runs Dobb-G: block_sizes divide the output dimensions, the moments are captured from
    output gradients (accumulate takes N x m tensors) and the step is dobb_step_g.
    Captures may be tensors, ``Mx4Capture``s or ``Fp8Capture``s, mixed.  With max_grad_norm, step and refresh_step first clip
    the gradients in place to that global norm over the set, as this process holds it (``clip_grad_norm_`` says
    what shards take instead); `grad_norm` (device scalar) then holds the norm before."""

    def __init__(self, weights, block_sizes, grads=None, n_tokens: int = 0, lr: float = 2.5e-3,
                 weight_decay: float = 0.0, momentum: float = 0.9, tau: float = 0.2, nesterov: bool = False,
                 norm: int = _abi.DOBB_NORM_SIGN, update_scales=None, streams: int = 1,
                 basis_dtype: torch.dtype = torch.float32, side: str = "input"):
        if side not in ("input", "output"):
            raise ValueError('side must be "input" (Dobb) or "output" (Dobb-G)')
        self.side = side
        self.step_op = _abi.DOBB_OP_STEP if side == "input" else _abi.DOBB_OP_STEP_G
        self.W = list(weights)
        self.nb = [int(b) for b in block_sizes]
        if len(self.nb) != len(self.W):
            raise ValueError("one block size per weight")
        dev = self.W[0].device
        self.device = dev
        self.count = len(self.W)
        for w in self.W:
            _abi._dtype_code(w)
            if w.dim() != 2 or not w.is_contiguous() or w.device != dev:
                raise ValueError("weights must be contiguous 2-D tensors on one device")
        self.shapes = [(w.shape[0], w.shape[1], nb) for w, nb in zip(self.W, self.nb)]
        for i, nb in enumerate(self.nb):
            if self.cap_dim(i) % nb:
                raise ValueError(f"block size {nb} does not divide {self.cap_dim(i)}")
        if basis_dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("basis_dtype must be torch.float32 or torch.bfloat16")
        self.q_dtype = _abi.DOBB_BF16 if basis_dtype == torch.bfloat16 else _abi.DOBB_F32
        self.M = [torch.zeros(w.shape, dtype=torch.float32, device=dev) for w in self.W]
        nblk = [self.cap_dim(i) // nb for i, nb in enumerate(self.nb)]
        self.A = [torch.zeros(B, nb, nb, dtype=torch.float32, device=dev) for B, nb in zip(nblk, self.nb)]
        # Q = I before the first refresh (the step is then sign(M)); the identity is exact in bf16
        self.Q = [torch.eye(nb, dtype=basis_dtype, device=dev).expand(B, nb, nb).contiguous()
                  for B, nb in zip(nblk, self.nb)]
        self.lam = [torch.zeros(B, nb, dtype=torch.float32, device=dev) for B, nb in zip(nblk, self.nb)]
        self.info = [torch.zeros(B, dtype=torch.int32, device=dev) for B in nblk]
        self.G = list(grads) if grads is not None else None
        scale_fn = default_update_scale if side == "input" else default_update_scale_g
        scales = update_scales or [scale_fn(m, n, tau) for (m, n, _) in self.shapes]
        self.hp = [_abi.make_hparams(lr, weight_decay, momentum, s, nesterov, norm) for s in scales]
        self.norm = norm
        self.n_tokens = n_tokens
        self._parts = []
        self._bound = []                      # workspaces that graphs captured by the caller use
        self.set_streams(streams)
        self.refreshes = 0
        self.grad_norm = torch.zeros((), dtype=torch.float32, device=dev)

    def cap_dim(self, i: int) -> int:
        """The dimension the moments of weight i are captured on: n (inputs) or m (outputs, Dobb-G)."""
        return self.W[i].shape[1] if self.side == "input" else self.W[i].shape[0]

    def set_streams(self, streams: int) -> None:
        """Partition the weights for `streams` streams (1 or 2), and by weight dtype; the state
        tensors are kept."""
        narrow = [i for i, nb in enumerate(self.nb) if nb <= 128]
        wide = [i for i, nb in enumerate(self.nb) if nb > 128]
        wdt = lambda i: self.W[i].dtype  # noqa: E731
        self._parts = []
        if streams > 1 and narrow and wide:
            side = torch.cuda.Stream(self.device)
            self._parts = [_Part(self, sub, None) for sub in _split(wide, wdt)]
            self._parts += [_Part(self, sub, side) for sub in _split(narrow, wdt)]
        else:
            self._parts = [_Part(self, sub, None) for sub in _split(range(self.count), wdt)]

    def set_hparams(self, idx=None, lr=None, weight_decay=None, momentum=None) -> None:
        """Change lr, weight decay or momentum of the weights idx (default: all) for later steps."""
        for i in range(self.count) if idx is None else idx:
            h = self.hp[i]
            self.hp[i] = _abi.make_hparams(h.lr if lr is None else lr,
                                           h.weight_decay if weight_decay is None else weight_decay,
                                           h.momentum if momentum is None else momentum,
                                           h.update_scale, bool(h.nesterov), h.norm)
        for part in self._parts:
            part.refresh_hp(self)

    def _run(self, stream, fn, plans=None):
        """fn(part, stream handle) for every part: those without a stream of their own on the caller's
        stream, the others on theirs, forked from and joined back into the caller's stream.  Workspaces have
        the size of `plans` (by _plan) before the streams fork: one that grew between two calls of a part would be
        freed while the first still runs, and another part's stream does not wait for that."""
        main = torch.cuda.current_stream(self.device) if stream is None else stream
        capturing = torch.cuda.is_current_stream_capturing()
        sides = []
        for part in self._parts:
            if part.stream is not None and part.stream not in sides:
                sides.append(part.stream)
            part.reserve(plans[part].need if plans else 0, main if part.stream is None else part.stream)
            if capturing and not any(w is part.ws for w in self._bound):
                self._bound.append(part.ws)
        for s in sides:
            s.wait_stream(main)
        with torch.cuda.device(self.device):
            for part in self._parts:
                fn(part, _abi._stream(main if part.stream is None else part.stream))
        for s in sides:
            main.wait_stream(s)

    @staticmethod
    def _dense_tokens(xs) -> int:
        """Tokens of the longest capture given as a tensor (those in MXFP4 or FP8 size their own workspace)."""
        return max((x.shape[0] for x in xs if not isinstance(x, (Mx4Capture, Fp8Capture))), default=0)

    def _plan(self, xs):
        """{part: its calls that take the captures xs, and the workspace they need}: one call per (tiles, token
        count) of those in MXFP4, per (tiles, token count, format) of those in FP8, and per (activation dtype, token
        count) of the tensors.  Every capture is checked here, before anything is enqueued."""
        N = self._dense_tokens(xs)
        plans = {}
        for part in self._parts:
            need = part.need(self, N) if N > self.n_tokens else 0
            mx4 = [i for i in part.idx if isinstance(xs[i], Mx4Capture)]
            fp8 = [i for i in part.idx if isinstance(xs[i], Fp8Capture)]
            dense = [i for i in part.idx if not isinstance(xs[i], (Mx4Capture, Fp8Capture))] if mx4 or fp8 else part.idx
            for i in part.idx:
                self._check_capture(i, xs[i])
            mx4 = _split(mx4, lambda i: (xs[i].tiles, xs[i].shape[0]))
            fp8 = _split(fp8, lambda i: (xs[i].tiles, xs[i].shape[0], xs[i].operand.fmt))
            dense = _split(dense, lambda i: (xs[i].dtype, xs[i].shape[0]))
            for sub in mx4:
                need = max(need, _ops.dobb_moment_mx4_workspace_size(self._cap_shapes(sub), xs[sub[0]].tiles))
            for sub in fp8:
                need = max(need, _layers.dobb_moment_fp8_workspace_size(self._cap_shapes(sub), xs[sub[0]].tiles))
            for sub in dense:
                need = max(need, _abi.dobb_workspace_size(_abi.DOBB_OP_ACCUMULATE, self._cap_shapes(sub), xs[sub[0]].shape[0]))
            plans[part] = _Plan(mx4, fp8, dense, need)
        return plans

    def _check_capture(self, i: int, x) -> None:
        """Refuse a capture that the calls for weight i would not take."""
        if isinstance(x, (Mx4Capture, Fp8Capture)):
            if x.shape[1] != self.cap_dim(i) or x.device != self.device:
                raise ValueError(f"capture {i} must hold (tokens x {self.cap_dim(i)}) on {self.device}")
            if not x.aligned:
                raise ValueError(f"capture {i}: codes must be aligned to 16 bytes and scales to 4")
            return
        if x.dim() != 2 or x.shape[1] != self.cap_dim(i) or not x.is_contiguous() or x.device != self.device:
            raise ValueError(f"capture {i} must be a contiguous (tokens x {self.cap_dim(i)}) tensor")
        _abi._dtype_code(x)

    def _cap_shapes(self, sub):
        return [(1, self.cap_dim(i), self.nb[i]) for i in sub]

    def _accumulate(self, part, plan, sh, xs, beta):
        for sub in plan.mx4:
            c = [xs[i] for i in sub]
            _abi._check(_ops._lib().dobb_accumulate_moment_mx4_grouped(
                len(sub), (_abi.Shape * len(sub))(*[_abi.Shape(*s) for s in self._cap_shapes(sub)]),
                _arr([x.codes.data_ptr() for x in c]), _arr([x.scales.data_ptr() for x in c]), c[0].tiles, c[0].shape[0],
                float(beta), _arr([self.A[i].data_ptr() for i in sub]), part.ws.data_ptr(), part.ws.numel(), sh),
                "dobb_accumulate_moment_mx4_grouped")
        for sub in plan.fp8:
            c = [xs[i] for i in sub]
            _abi._check(_layers._lib().dobb_accumulate_moment_fp8_grouped(
                len(sub), (_abi.Shape * len(sub))(*[_abi.Shape(*s) for s in self._cap_shapes(sub)]),
                (_layers._CFp8Operand * len(sub))(*[_layers._c_operand(x.operand) for x in c]), c[0].shape[0], float(beta),
                _arr([self.A[i].data_ptr() for i in sub]), part.ws.data_ptr(), part.ws.numel(), sh),
                "dobb_accumulate_moment_fp8_grouped")
        for sub in plan.dense:
            if len(sub) == part.count:
                ash, A, ldx = part.ash, part.A, part.ldx
            else:
                ash = (_abi.Shape * len(sub))(*[_abi.Shape(*s) for s in self._cap_shapes(sub)])
                A = _arr([self.A[i].data_ptr() for i in sub])
                ldx = (ctypes.c_int64 * len(sub))(*[self.cap_dim(i) for i in sub])
            _abi._check(_abi.lib().dobb_accumulate_moment_grouped(
                len(sub), ash, _arr([xs[i].data_ptr() for i in sub]), _abi._dtype_code(xs[sub[0]]), xs[sub[0]].shape[0], ldx,
                float(beta), A, part.ws.data_ptr(), part.ws.numel(), sh), "dobb_accumulate_moment_grouped")

    def _refresh(self, part, sh, mode, iters, warm_start, tol, with_lam):
        _abi._check(_abi.lib().dobb_refresh_basis_grouped(
            part.count, part.ash, part.A, part.Q, self.q_dtype, part.lam if with_lam else None, int(mode),
            int(iters), int(bool(warm_start)), float(tol), part.info, part.ws.data_ptr(), part.ws.numel(), sh),
            "dobb_refresh_basis_grouped")

    def _checked(self, grads):
        """The gradients of a step, checked: before anything is enqueued, and before they are clipped in place."""
        G = grads if grads is not None else self.G
        for i, w in enumerate(self.W):
            g = G[i]
            if tuple(g.shape) != tuple(w.shape) or not g.is_contiguous() or g.device != self.device:
                raise ValueError(f"gradient {i} must be a contiguous tensor of shape {tuple(w.shape)}")
            _abi._dtype_code(g)
        return G

    def _step(self, part, sh, G):
        """One grouped step per gradient dtype among the part's weights."""
        for sub in _split(part.idx, lambda i: G[i].dtype):
            if len(sub) == part.count:
                shp, Wp, Mp, Qp, hp = part.sh, part.W, part.M, part.Q, part.hp
            else:
                pos = {i: k for k, i in enumerate(part.idx)}
                shp = (_abi.Shape * len(sub))(*[_abi.Shape(*self.shapes[i]) for i in sub])
                Wp = _arr([self.W[i].data_ptr() for i in sub])
                Mp = _arr([self.M[i].data_ptr() for i in sub])
                Qp = _arr([self.Q[i].data_ptr() for i in sub])
                hp = (_abi.HParams * len(sub))(*[part.hp[pos[i]] for i in sub])
            fn = _abi.lib().dobb_step_grouped if self.side == "input" else _abi.lib().dobb_step_g_grouped
            _abi._check(fn(len(sub), shp, Wp, part.w_dtype, _arr([G[i].data_ptr() for i in sub]),
                           _abi._dtype_code(G[sub[0]]), Mp, Qp, self.q_dtype, hp, None, None, part.ws.data_ptr(),
                           part.ws.numel(), sh), "dobb_step_grouped" if self.side == "input" else "dobb_step_g_grouped")

    def accumulate(self, xs, beta: float, stream=None) -> None:
        """Capture: A_b <- beta A_b + (1-beta)/N X_b^T X_b for every weight (xs[i] is N_i x n_i, or the
        N_i x m_i output gradients for Dobb-G), as tensors, in MXFP4 or in FP8."""
        plans = self._plan(xs)
        self._run(stream, lambda part, sh: self._accumulate(part, plans[part], sh, xs, beta), plans)
        self.n_tokens = max(self.n_tokens, self._dense_tokens(xs))

    def refresh(self, mode: int, iters: int, warm_start: bool = True, tol: float = 0.0, want_lambda: bool = False,
                stream=None) -> None:
        """Refresh every basis; lambda is filled for the exact mode, and for orthogonal iteration only
        when want_lambda (Rayleigh quotients cost an extra product per block)."""
        with_lam = want_lambda or mode == _abi.DOBB_REFRESH_EXACT
        self._run(stream, lambda part, sh: self._refresh(part, sh, mode, iters, warm_start, tol, with_lam))
        self.refreshes += 1

    def clip_grads(self, max_norm: float, grads=None, stream=None) -> torch.Tensor:
        """Clip the gradients in place to a global norm over the set (dobb_clip_grad_norm_grouped); returns
        `grad_norm`, which receives the norm before."""
        G = grads if grads is not None else self.G
        return _ops.dobb_clip_grad_norm_grouped(G, max_norm, total=self.grad_norm, stream=stream)

    def step(self, grads=None, stream=None, max_grad_norm: float | None = None) -> None:
        G = self._checked(grads)
        if max_grad_norm is not None:
            self.clip_grads(max_grad_norm, G, stream)
        self._run(stream, lambda part, sh: self._step(part, sh, G))

    def refresh_step(self, xs, beta: float, mode: int, iters: int, grads=None, warm_start: bool = True,
                     tol: float = 0.0, want_lambda: bool = False, stream=None,
                     max_grad_norm: float | None = None) -> None:
        """accumulate, refresh and step in one call: each part runs the three phases back to back on
        its own stream, so with streams=2 one part's refresh overlaps the other's capture and step.
        The result is the same as the three calls in turn."""
        plans = self._plan(xs)
        G = self._checked(grads)
        if max_grad_norm is not None:
            self.clip_grads(max_grad_norm, G, stream)
        with_lam = want_lambda or mode == _abi.DOBB_REFRESH_EXACT

        def go(part, sh):
            self._accumulate(part, plans[part], sh, xs, beta)
            self._refresh(part, sh, mode, iters, warm_start, tol, with_lam)
            self._step(part, sh, G)
        self._run(stream, go, plans)
        self.n_tokens = max(self.n_tokens, self._dense_tokens(xs))
        self.refreshes += 1

    def capture_refresh_step(self, xs, beta: float, mode: int, iters: int, grads=None, warm_start: bool = True,
                             max_grad_norm: float | None = None) -> "torch.cuda.CUDAGraph":
        """A HIP graph of refresh_step(xs, beta, mode, iters, grads): replaying it runs the same
        kernels on the same buffers without the per-launch host work and gaps.  xs, the gradients and
        the optimizer state are bound by address, so the caller refills them in place between replays.
        Capturing runs nothing; the workspaces must already have their size, so call refresh_step once
        (or accumulate with the same token counts) first.  Each replay counts as one refresh.  The graph
        holds the group and all tensors bound, and its workspaces, should a later call replace them: it has
        to outlive its last replay."""
        if self._dense_tokens(xs) > self.n_tokens or any(plan.need > part.ws.numel() for part, plan in self._plan(xs).items()):
            raise RuntimeError("call refresh_step once before capturing it (the workspaces are sized there)")
        graph = torch.cuda.CUDAGraph()
        refreshes, bound = self.refreshes, list(self._bound)
        with torch.cuda.device(self.device), torch.cuda.graph(graph):
            self.refresh_step(xs, beta, mode, iters, grads=grads, warm_start=warm_start, max_grad_norm=max_grad_norm)
        self.refreshes, self._bound = refreshes, bound
        graph.holds = (self, list(xs), list(grads if grads is not None else self.G), [part.ws for part in self._parts])
        return graph


def _held_as(x) -> str:
    return f"{type(x).__name__} in {x.operand.fmt}" if isinstance(x, Fp8Capture) else type(x).__name__


class Dobb(torch.optim.Optimizer):
    """torch.optim interface: 2-D parameters only, each with a block size (default: n // blocks).

    lr, weight_decay and momentum are read from each parameter group at every step, so learning-rate
    schedulers and later edits of ``param_groups`` take effect.  Activations are supplied by the
    caller with ``capture(param, x)`` (or the forward hooks from ``attach_capture_hooks``) before
    ``step()`` on refresh iterations; ``wants_capture()`` says whether the coming step refreshes.
    capture="first" keeps a weight's first micro-batch of a refresh iteration (the principal policy
    of Table 17), capture="all" every micro-batch (their tokens are pooled into one capture).
    basis="output_gradient" runs Dobb-G (Tables 12-13): blocks of rows (m // blocks, or block_size),
    bases of the output-gradient second moment, captured by the backward hooks of
    ``attach_capture_hooks`` (or ``capture(param, grad_output)``).
    capture_format="mx4" holds captures in MXFP4 from the moment they are taken (``Mx4Capture``): 0.27 of bf16's
    bytes an entry between the forward pass and the refresh, and in the refresh's moment; "native" keeps the
    tensors.  Every weight's capture is quantised and held by itself, where "native" holds one tensor for all
    weights that see it (0.41 of bf16's memory for a layer with separate q, k, v and gate, up of equal width).
    capture_format="fp8" holds them in FP8 (``Fp8Capture``; 0.50 of bf16's bytes).  ``capture`` also takes captures
    that are held already, an ``Fp8Capture`` of the operand that the weight's gradient takes in FP8 among them: it
    then costs neither time nor memory of its own.
    max_grad_norm clips the gradients of this optimizer's parameters in place, by their global norm in this
    process (``clip_grad_norm_`` says what shards take instead), before every step; ``grad_norm`` then holds the
    norm before (a scalar on the parameters' device).
    """

    def __init__(self, params, lr: float = 2.5e-3, weight_decay: float = 0.0, momentum: float = 0.9,
                 blocks: int = 16, block_size: int | None = None, refresh_period: int = 9, orth_iters: int = 1,
                 beta: float = 0.9, tau: float = 0.2, nesterov: bool = False, streams: int = 1,
                 capture: str = "first", basis_dtype: torch.dtype = torch.float32, basis: str = "activation",
                 capture_format: str = "native", max_grad_norm: float | None = None):
        super().__init__(params, dict(lr=lr, weight_decay=weight_decay, momentum=momentum))
        if capture not in ("first", "all"):
            raise ValueError('capture must be "first" or "all"')
        if basis not in ("activation", "output_gradient"):
            raise ValueError('basis must be "activation" (Dobb) or "output_gradient" (Dobb-G)')
        if capture_format not in ("native", "mx4", "fp8"):
            raise ValueError('capture_format must be "native", "mx4" or "fp8"')
        if max_grad_norm is not None and not max_grad_norm >= 0:
            raise ValueError("max_grad_norm must not be negative")
        params = [p for grp in self.param_groups for p in grp["params"]]
        for p in params:
            if p.dim() != 2:
                raise ValueError("Dobb handles 2-D weights; use another optimizer for the rest")
        self.side = "input" if basis == "activation" else "output"
        axis = 1 if self.side == "input" else 0
        nbs = [block_size or p.shape[axis] // blocks for p in params]
        self._params = params
        self._index = {id(p): i for i, p in enumerate(params)}
        self._group = DobbGroup([p.data for p in params], nbs, lr=lr, weight_decay=weight_decay,
                                momentum=momentum, tau=tau, nesterov=nesterov, streams=streams,
                                basis_dtype=basis_dtype, side=self.side)
        self._slots = []                      # per param group: the weight indices
        k = 0
        for grp in self.param_groups:
            self._slots.append(list(range(k, k + len(grp["params"]))))
            k += len(grp["params"])
        self._applied = [None] * len(self.param_groups)
        self.capture_policy = capture
        self.capture_format = capture_format
        self.max_grad_norm = max_grad_norm
        self.grad_norm: torch.Tensor | None = None
        self.T = int(refresh_period)
        self.k = int(orth_iters)
        self.beta = float(beta)
        self.t = 0
        self._captured: dict[int, list] = {}

    def wants_capture(self) -> bool:
        return self.t % self.T == 0

    def capture(self, param, x) -> None:
        """Record (tokens x n) input activations of `param` (Dobb), or (tokens x m) output gradients
        (Dobb-G), for the next refresh: the first call per refresh iteration, or every call with
        capture="all".  A call without tokens is passed over.  x is a tensor, or a capture that is held already (an
        ``Mx4Capture`` or ``Fp8Capture``: kept as it is, copied only if it is not aligned, with capture="all" for every
        micro-batch).  What a step could not take is refused here: another width, device or type, or another format
        than the weight's captures before."""
        held = isinstance(x, (Mx4Capture, Fp8Capture))
        if not held:
            x = x.detach().reshape(-1, x.shape[-1])
        if not x.shape[0] or (self.capture_policy != "all" and id(param) in self._captured):
            return
        if not held:
            x = (Mx4Capture.quantize(x) if self.capture_format == "mx4" else
                 Fp8Capture.quantize(x) if self.capture_format == "fp8" else x.contiguous())
        if held and not x.aligned:
            x = type(x).cat([x])
        if id(param) in self._index:
            self._group._check_capture(self._index[id(param)], x)
        before = self._captured.get(id(param), [])
        if before and _held_as(before[0]) != _held_as(x):
            raise ValueError(f"captures of one weight must be held alike: {_held_as(before[0])} before, now {_held_as(x)}")
        self._captured[id(param)] = before + [x]

    def attach_capture_hooks(self, modules):
        """Hooks on nn.Linear modules whose weights this optimizer owns: on refresh iterations their
        inputs (forward pre-hooks; Dobb) or output gradients (backward hooks; Dobb-G) are captured,
        from the first micro-batch, or all of them with capture="all"."""
        handles = []
        owned = {id(p) for p in self._params}
        for mod in modules:
            w = getattr(mod, "weight", None)
            if w is None or id(w) not in owned:
                continue
            if self.side == "input":
                def hook(module, inputs, w=w):
                    if self.wants_capture():
                        self.capture(w, inputs[0])
                handles.append(mod.register_forward_pre_hook(hook))
            else:
                def bhook(module, grad_input, grad_output, w=w):
                    if self.wants_capture() and grad_output[0] is not None:
                        self.capture(w, grad_output[0])
                handles.append(mod.register_full_backward_hook(bhook))
        return handles

    def _sync_hparams(self) -> None:
        for gi, grp in enumerate(self.param_groups):
            cur = (float(grp["lr"]), float(grp["weight_decay"]), float(grp["momentum"]))
            if cur != self._applied[gi]:
                self._group.set_hparams(self._slots[gi], lr=cur[0], weight_decay=cur[1], momentum=cur[2])
                self._applied[gi] = cur

    @torch.no_grad()
    def step(self, closure=None):
        loss = closure() if closure is not None else None
        self._sync_hparams()
        g = self._group
        if self.max_grad_norm is not None:
            self.grad_norm = clip_grad_norm_(self._params, self.max_grad_norm)
        grads = [p.grad if p.grad is not None else torch.zeros_like(p) for p in self._params]
        if self.wants_capture() and len(self._captured) == len(self._params):
            xs = []
            for p in self._params:
                parts = self._captured[id(p)]
                if len(parts) > 1:               # the joined capture takes the place of its parts, weight by weight
                    held = isinstance(parts[0], (Mx4Capture, Fp8Capture))
                    self._captured[id(p)] = parts = [type(parts[0]).cat(parts) if held else torch.cat(parts, 0)]
                xs.append(parts[0])
            if g.refreshes == 0:
                g.refresh_step(xs, 0.0, _abi.DOBB_REFRESH_EXACT, 0, grads, warm_start=False)
            else:
                g.refresh_step(xs, self.beta, _abi.DOBB_REFRESH_ORTH_ITER, self.k, grads)
        else:
            g.step(grads)
        self._captured.clear()
        self.t += 1
        return loss
