"""The layer operators (include/dobb_layers.h) from their definitions in 64 bits, for the tests."""
import numpy as np
import torch

U = 2.0 ** -24
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}


def host(t):
    return t.detach().to("cpu", torch.float64).numpy()


def levels(fmt):
    """Every value from zero up that a format holds, by its code."""
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    code = np.arange(1 << 7)
    e, f = code >> bits, code & ((1 << bits) - 1)
    v = np.where(e == 0, f * 2.0 ** (low - bits), (1 + f / 2.0 ** bits) * 2.0 ** (e - 1.0 + low))
    return v[v <= LARGEST[fmt]]


def quantize(x, fmt, square=False):
    """(codes T x 8 x R x 16, scales T x R', values R x K) of a float64 array x (R x K) as an FP8 operand."""
    lev = levels(fmt)
    R, K = x.shape
    T = -(-K // 128)
    p = np.zeros((R, T, 128))
    p.reshape(R, T * 128)[:, :K] = x
    top = np.abs(p).max(2)                                        # NaN stays NaN
    if square:
        top = np.concatenate([np.broadcast_to(top[r:r + 128].max(0), top[r:r + 128].shape) for r in range(0, R, 128)])
    bad = ~np.isfinite(top)
    m, e = np.frexp(np.where(bad | (top == 0), 1.0, top))         # top = m 2^e with m in [0.5, 1)
    lm, le = np.frexp(LARGEST[fmt])
    S = np.maximum(np.where(top == 0, -127, e - le + (m > lm)), -127)
    y = np.where(bad[:, :, None], 0.0, np.abs(p)) / (2.0 ** S)[:, :, None]
    k = np.searchsorted((lev[1:] + lev[:-1]) / 2, y)              # midpoints below y
    mid = np.concatenate([(lev[1:] + lev[:-1]) / 2, [np.inf]])
    k = k + ((y == mid[k]) & (k % 2 == 1))                        # a tie goes to the even code
    neg = np.signbit(p)
    code = np.where(bad[:, :, None], 0x7f, k + 128 * neg).astype(np.uint8)
    val = np.where(bad[:, :, None], np.nan, lev[k] * np.where(neg, -1, 1) * (2.0 ** S)[:, :, None])
    scales = np.zeros((T, -(-R // 4) * 4), np.uint8)
    scales[:, :R] = np.where(bad, 255, S + 127).T
    return code.reshape(R, T, 8, 16).transpose(1, 2, 0, 3), scales, val.reshape(R, T * 128)[:, :K]


def norm(x, w, b, eps):
    """(y, mean, rstd, h) over the columns of every row."""
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1 / np.sqrt((c * c).mean(1) + eps)
    h = c * rstd[:, None]
    return h * (1.0 if w is None else w) + (0.0 if b is None else b), mean, rstd, h


def norm_depth(n):
    """Additions in a row that a sum over a row takes: of one thread's entries, then of the threads."""
    return (16 if n <= 16384 else 8 * -(-n // 8192)) + 6 + 16


def norm_bounds(x, w, b, eps, out_eps):
    """How far y, mean and rstd may be off.  Sums run around a first mean m0 that is D u mean|x| off at most:
    mean = m0 + d with d within (D + 2) u mean|x - m0|, the squares within (D + 4) u of theirs and half of that
    in rstd (three roundings more there); y takes mean's error, rstd's and two roundings, the factor w, and its own."""
    y, mean, rstd, h = norm(x, w, b, eps)
    D = norm_depth(x.shape[1])
    spread = np.abs(x - mean[:, None]).mean(1) + D * U * np.abs(x).mean(1)
    m = (D + 3) * U * spread + 3 * U * np.abs(mean)
    # the square of d, which is taken off again, is known to 2 |d| (D + 3) u spread
    d2 = 2 * (D * U * np.abs(x).mean(1)) * (D + 3) * U * spread
    r = rstd * ((D + 4) / 2 + 3) * U + 0.5 * rstd ** 3 * (d2 + 4 * U * (D * U * np.abs(x).mean(1)) ** 2)
    aw = 1.0 if w is None else np.abs(w)
    hb = m[:, None] * rstd[:, None] + np.abs(h) * ((r / rstd)[:, None] + 2 * U)
    return hb * aw + (U + out_eps / 2) * np.abs(y) + U * np.abs(h * aw) + 1e-44, m + 1e-44, r


def norm_grad(dy, x, mean, rstd, w):
    """(dx, dw, db) and how far each may be off before its rounding."""
    n = x.shape[1]
    D = norm_depth(n)
    h = (x - mean[:, None]) * rstd[:, None]
    g = dy * (1.0 if w is None else w)
    a, c = g.mean(1, keepdims=True), (g * h).mean(1, keepdims=True)
    ag, agh = np.abs(g).mean(1, keepdims=True), np.abs(g * h).mean(1, keepdims=True)
    dx = rstd[:, None] * (g - a - h * c)
    bound = rstd[:, None] * U * (4 * np.abs(g) + (D + 5) * ag + (D + 9) * np.abs(h) * agh)
    # a column's sum: a thread's rows (of at least 64 groups), then up to 32 threads of a group; the groups in fp64
    rows = -(-x.shape[0] // 64) + 32
    return (dx, (dy * h).sum(0), dy.sum(0)), (bound, (rows + 3) * U * np.abs(dy * h).sum(0), rows * U * np.abs(dy).sum(0))
