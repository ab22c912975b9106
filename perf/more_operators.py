"""Cases of the layer norm, FP8 operand, FP8 product and FP8 capture operators, with their plain forms.

A layer whose weight Dobb trains is a layer norm and a linear map behind it.  In training its activations
are needed three times: as the operand of the product with the weight, as the operand of the weight's
gradient, and as the capture whose second moment the basis is taken from.  The kinds of case:

* norm      y = (x - mean) rstd w + b over the columns of every row, with mean and rstd;
* normgrad  its backward pass: gradients of x, w and b, the last two summed over all rows;
* quantise  a matrix as FP8 operands (e4m3 or e5m2 elements, a power of two over every 128 entries along
            the contracted axis, or over squares of 128 x 128), along its rows and along its columns, and
            the values read back;
* product   out = A B^T + bias from two FP8 operands;
* backward  of a linear layer in FP8: the output gradient quantised, then the input's and the weight's
            gradients as two products;
* layer     layer norm, its output as FP8 operands, the product with the weight, and the second moment
            from the same operand: a refresh iteration's forward pass;
* moment    captures held in FP8 into the second-moment blocks A_b <- beta A_b + (1 - beta)/N sum_t x_t x_t^T;
* capture   micro-batches quantised as they come, then the moment from all of them.

An FP8 operand holds R rows of K entries in T = ceil(K / 128) tiles: codes (T, 8, R, 16), entry
[t][h][r] being row r's entries 128 t + 16 h on, and scales (T, R rounded up to fours): the exponent of a tile's
power of two, + 127.  The missing entries of the last tile are zeros.  The power is the least that brings the block's largest
magnitude to the format's largest value or below (2^-127 at least).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "bf16": 2}
# largest value, mantissa bits, least exponent of a normal value, torch's type
FORMATS = {"e4m3": (448.0, 3, -6, torch.float8_e4m3fn), "e5m2": (57344.0, 2, -14, torch.float8_e5m2)}
EPS = 1e-5

# the weights of a GPT-2 XL layer (rows, columns) and their block widths
XL = [(4800, 1600, 100), (1600, 1600, 100), (6400, 1600, 100), (1600, 6400, 400)]


def listed():
    return [
        # the last position's norm in a small model: the call's latency
        dict(name="norm one token", kind="norm", rows=1, n=768, ld=768, dtype="fp32", out="fp32"),
        # every token of a GPT-2 XL batch, bf16
        dict(name="norm xl tokens", kind="norm", rows=16384, n=1600, ld=1600, dtype="bf16", out="bf16"),
        # rows of a slice, an odd width, fp32
        dict(name="norm backward odd slice", kind="normgrad", rows=997, n=1601, ld=4800, dtype="fp32"),
        # the GPT-2 XL batch again, backward
        dict(name="norm backward xl tokens", kind="normgrad", rows=16384, n=1600, ld=1600, dtype="bf16"),
        # a weight of the 7B-style stack after an optimizer step: squares, so that both operands agree
        dict(name="quantise 7b weight", kind="quantise", rows=11008, n=4096, ld=4096, dtype="fp32", fmt="e4m3", square=True),
        # output gradients of a batch that is no whole number of tiles
        dict(name="quantise odd gradients", kind="quantise", rows=997, n=4800, ld=4800, dtype="bf16", fmt="e5m2", square=False),
        # one token through a projection of the 7B-style stack: the weight is read once
        dict(name="product one token", kind="product", m=1, n=11008, k=4096, out="bf16", bias=False, fa="e4m3", fb="e4m3"),
        # the projection back of a GPT-2 XL layer, the whole batch
        dict(name="product xl fc-proj", kind="product", m=16384, n=1600, k=6400, out="bf16", bias=True, fa="e4m3", fb="e4m3"),
        # a projection of the 7B-style stack backward, an odd number of tokens
        dict(name="backward 7b projection", kind="backward", tokens=4093, m=11008, n=4096),
        # norm, projection to q, k and v, and the capture's moment of a GPT-2 XL layer
        dict(name="layer xl qkv", kind="layer", tokens=16384, m=4800, n=1600, nb=100, beta=0.0),
        # twelve layers of the GPT-2 XL set in one grouped call
        dict(name="moment xl 12 layers", kind="moment", layers=12, tokens=16384, beta=0.9),
        # a capture of a few tokens
        dict(name="capture few tokens", kind="capture", n=400, nb=100, tokens=37, parts=1, dtype="fp32", beta=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "normgrad", "quantise", "product", "backward", "layer", "capture"])
    if kind in ("norm", "normgrad", "quantise"):
        rows = _log(rng, 1, 16384)
        # (a norm over two or three entries says little: its gradient is what rounding leaves)
        n = _log(rng, 1 if kind == "quantise" else 8, min(16384, 16384 * 1600 // rows))
        c = dict(kind=kind, rows=rows, n=n, ld=n + rng.choice([0, 0, 1, 8, n]), dtype=rng.choice(["fp32", "bf16"]))
        if kind == "norm":
            c.update(out=rng.choice(["fp32", "bf16"]))
        if kind == "quantise":
            c.update(fmt=rng.choice(["e4m3", "e5m2"]), square=rng.random() < 0.4)
        return c
    if kind == "product":
        m = _log(rng, 1, 16384)
        n, k = _log(rng, 1, 11008), _log(rng, 16, 11008)
        return dict(kind=kind, m=min(m, max(1, 16384 * 1600 * 6400 // (n * k))), n=n, k=k, out=rng.choice(["fp32", "bf16"]),
                    bias=rng.random() < 0.5, fa=rng.choice(["e4m3", "e5m2"]), fb="e4m3")
    if kind == "backward":
        tokens = _log(rng, 1, 4096)
        return dict(kind=kind, tokens=tokens, m=_log(rng, 16, 11008), n=_log(rng, 16, 4096))
    nb = _log(rng, 8, 512)
    n = nb * _log(rng, 1, max(1, min(16, 6400 // nb)))
    if kind == "layer":
        return dict(kind=kind, tokens=_log(rng, 1, 8192), m=_log(rng, 16, 6400), n=n, nb=nb, beta=rng.choice([0.0, 0.5, 0.9]))
    tokens = _log(rng, 1, 16384)
    return dict(kind=kind, n=n, nb=nb, tokens=tokens, parts=min(tokens, rng.choice([1, 2, 5])), dtype=rng.choice(["fp32", "bf16"]),
                beta=rng.choice([0.0, 0.5, 0.9]))


# ---- shapes ------------------------------------------------------------------------------------
def _tiles(k):
    return (k + 127) // 128


def _parts(case):
    """Tokens of every micro-batch of a capture case: as even as they come."""
    N, P = case["tokens"], case["parts"]
    return [N * (i + 1) // P - N * i // P for i in range(P)]


def _weights(case):
    """(columns, block width) of every capture of a moment case."""
    return [(n, nb) for _ in range(case["layers"]) for _, n, nb in XL]


def _operand_bytes(r, k):
    return _tiles(k) * r + r * k


def work(case):
    kind = case["kind"]
    if kind in ("norm", "normgrad"):
        e, n, r = case["rows"] * case["n"], case["n"], case["rows"]
        if kind == "norm":
            return {"bytes": e * (SIZE[case["dtype"]] + SIZE[case["out"]]) + 8 * n + 8 * r, "flops": 7 * e}
        return {"bytes": e * 3 * SIZE[case["dtype"]] + 12 * n + 8 * r, "flops": 14 * e}
    if kind == "quantise":
        r, n = case["rows"], case["n"]
        return {"bytes": r * n * (SIZE[case["dtype"]] + 4) + _operand_bytes(r, n) + _operand_bytes(n, r), "flops": 4 * r * n}
    if kind == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": _operand_bytes(m, k) + _operand_bytes(n, k) + m * n * SIZE[case["out"]], "flops": 2 * m * n * k}
    if kind == "backward":
        t, m, n = case["tokens"], case["m"], case["n"]
        return {"bytes": 2 * t * m + _operand_bytes(n, m) + _operand_bytes(n, t) + 2 * t * n + 4 * m * n, "flops": 4 * t * m * n}
    if kind == "layer":
        t, m, n, nb = case["tokens"], case["m"], case["n"], case["nb"]
        return {"bytes": 2 * t * n + _operand_bytes(m, n) + 2 * t * m + 8 * t + n * nb * (8 if case["beta"] > 0 else 4),
                "flops": 2 * t * m * n + t * n * (nb + 1)}
    N = case["tokens"]
    b = f = 0
    for n, nb in _weights(case) if kind == "moment" else [(case["n"], case["nb"])]:
        b += n * nb * (8 if case["beta"] > 0 else 4)
        b += _operand_bytes(n, N) if kind == "moment" else N * n * SIZE[case["dtype"]]
        f += N * n * (nb + 1)
    return {"bytes": b, "flops": f}


# ---- inputs ------------------------------------------------------------------------------------
def _activations(N, n, gen):
    """Rows of tokens: normal entries around a mean, columns of log-normal size with a few far larger ones, and
    tokens of differing size, as the residual stream and the inputs of linear layers come."""
    col = torch.randn(n, generator=gen, device=DEV).mul_(0.5).exp_()
    col = torch.where(torch.rand(n, generator=gen, device=DEV) < 0.01, 20 * col, col)
    tok = torch.randn(N, 1, generator=gen, device=DEV).mul_(0.3).exp_()
    return torch.randn(N, n, generator=gen, device=DEV).add_(0.1).mul_(col).mul_(tok)


def _gradients(N, n, gen):
    """Output gradients: small, with rows and columns of differing size."""
    col = torch.randn(n, generator=gen, device=DEV).exp_()
    tok = torch.randn(N, 1, generator=gen, device=DEV).exp_()
    return torch.randn(N, n, generator=gen, device=DEV).mul_(col).mul_(tok).mul_(1e-4)


def _weight(m, n, gen):
    return torch.randn(m, n, generator=gen, device=DEV).mul_(n ** -0.5)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = {"case": case}
    kind = case["kind"]
    if kind in ("norm", "normgrad", "quantise"):
        r, n, ld, dt = case["rows"], case["n"], case["ld"], DT[case["dtype"]]
        if kind == "quantise":
            make = _weight if case["square"] else _gradients if case["fmt"] == "e5m2" else _activations
            s["x"] = make(r, ld, gen).to(dt)[:, :n]
            return s
        s["x"] = _activations(r, ld, gen).to(dt)[:, :n]
        s["w"] = torch.randn(n, generator=gen, device=DEV).mul_(0.2).add_(1.0)
        s["b"] = torch.randn(n, generator=gen, device=DEV).mul_(0.1)
        if kind == "normgrad":
            s["dy"] = _gradients(r, ld, gen).to(dt)[:, :n]
            _, s["mean"], s["rstd"] = _norm(s["x"].float(), s["w"], s["b"])
        return s
    if kind == "product":
        m, n, k = case["m"], case["n"], case["k"]
        a = _gradients(m, k, gen) if case["fa"] == "e5m2" else _activations(m, k, gen)
        s["a"] = _pack(a, case["fa"], False)
        s["b"] = _pack(_weight(n, k, gen), case["fb"], True)
        if case["bias"]:
            s["bias"] = torch.randn(n, generator=gen, device=DEV).mul_(0.1)
        return s
    if kind == "backward":
        t, m, n = case["tokens"], case["m"], case["n"]
        s["dy"] = _gradients(t, m, gen).to(torch.bfloat16)
        s["x"] = _pack(_activations(t, n, gen).t(), "e4m3", False)
        s["w"] = _pack(_weight(m, n, gen).t(), "e4m3", True)
        return s
    if kind == "layer":
        t, m, n = case["tokens"], case["m"], case["n"]
        s["x"] = _activations(t, n, gen).to(torch.bfloat16)
        s["w"] = torch.randn(n, generator=gen, device=DEV).mul_(0.2).add_(1.0)
        s["b"] = torch.randn(n, generator=gen, device=DEV).mul_(0.1)
        s["weight"] = _pack(_weight(m, n, gen), "e4m3", True)
        s["bias"] = torch.randn(m, generator=gen, device=DEV).mul_(0.1)
        shapes = [(n, case["nb"])]
    elif kind == "moment":
        shapes = _weights(case)
        s["held"] = [_pack(_activations(case["tokens"], n, gen).t(), "e4m3", False) for n, _ in shapes]
    else:
        s["x"] = [_activations(k, case["n"], gen).to(DT[case["dtype"]]) for k in _parts(case)]
        shapes = [(case["n"], case["nb"])]
    a = [torch.randn(n // nb, nb, nb, generator=gen, device=DEV) for n, nb in shapes]
    s["A"] = [x + x.transpose(1, 2) for x in a]
    return s


# ---- the plain forms ---------------------------------------------------------------------------
def _norm(x, w, b):
    """(y, mean, rstd) over the columns of every row."""
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = (c.square().mean(1) + EPS).rsqrt()
    return c * rstd[:, None] * w + b, mean, rstd


def _norm_grad(dy, x, mean, rstd, w):
    """Gradients of x, w and b; the sums over all rows in 64 bits."""
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0, dtype=torch.float64).float(), dy.sum(0, dtype=torch.float64).float()


def _pow2(e):
    """2^e for whole e from -127 to 127, exact (a library power need not be)."""
    return torch.where(e == -127, 1 << 22, (e + 127) << 23).to(torch.int32).view(torch.float32)


def _padded(x, rows):
    """x (R x K) with zeros up to a whole number of tiles along K (and along R if `rows`)."""
    R, K = x.shape
    p = torch.zeros(_tiles(R) * 128 if rows else R, _tiles(K) * 128, device=x.device)
    p[:R, :K] = x
    return p


def _elements(x, fmt, square):
    """(values in units of their block's power of two, exponents) of x (R x K, 32 bits), both R' x T x 128 or
    to be broadcast to it: blocks of 128 along K, or of 128 x 128."""
    largest, bits, low, _ = FORMATS[fmt]
    t = _padded(x, square).view(-1, _tiles(x.shape[1]), 128)
    top = t.abs().amax(2, keepdim=True)
    if square:
        R, T, _ = t.shape
        top = top.view(R // 128, 128, T, 1).amax(1, keepdim=True).expand(-1, 128, -1, -1).reshape(R, T, 1)
    half, e = torch.frexp(top)                       # top = half 2^e with half in [0.5, 1)
    e = e - int(math.log2(largest)) - 1 + (half > largest / 2.0 ** (int(math.log2(largest)) + 1)).int()
    e = torch.where(top > 0, e, -127).clamp(-127, 127)
    y = t * _pow2(-e)
    step = _pow2((torch.frexp(y)[1] - 1).clamp(min=low) - bits)
    return torch.round(y / step) * step, e


def _values(x, fmt, square):
    """x (R x K) as its FP8 operand's values."""
    v, e = _elements(x, fmt, square)
    return (v * _pow2(e)).view(v.shape[0], -1)[:x.shape[0], :x.shape[1]]


def _pack(x, fmt, square):
    """x (R x K) as an FP8 operand: (codes, scales, K, format)."""
    v, e = _elements(x, fmt, square)
    R, K = x.shape
    T = _tiles(K)
    v = v[:R].to(FORMATS[fmt][3]).view(torch.uint8).view(R, T, 8, 16)
    scales = torch.zeros(T, (R + 3) // 4 * 4, dtype=torch.uint8, device=x.device)
    scales[:, :R] = (e[:R, :, 0] + 127).t()
    return v.permute(1, 2, 0, 3).contiguous(), scales, K, fmt


def _unpack(op):
    """The values of an FP8 operand, R x K."""
    codes, scales, K, fmt = op
    T, _, R, _ = codes.shape
    v = codes.permute(2, 0, 1, 3).contiguous().view(FORMATS[fmt][3]).float().view(R, T, 128)
    return (v * _pow2(scales[:, :R].t().int()[:, :, None] - 127)).view(R, T * 128)[:, :K]


def _moment(x, nb, N, beta, A):
    """A <- beta A + (1 - beta) / N X_b^T X_b over blocks of nb columns (x: columns x tokens); products over 1024
    tokens in 32 bits, those added in 64 (the diagonal's terms are all of one sign)."""
    n, rows = x.shape
    C = (rows + 1023) // 1024
    p = torch.zeros(n, C * 1024, device=x.device)
    p[:, :rows] = x
    xb = p.view(n // nb, nb, C, 1024).transpose(1, 2).reshape(-1, nb, 1024)
    g = torch.bmm(xb, xb.transpose(1, 2).contiguous()).view(n // nb, C, nb, nb).sum(1, dtype=torch.float64)
    A.copy_(beta * A + (1 - beta) / N * g if beta > 0 else g / N)


# ---- one pass ----------------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    kind = case["kind"]
    if kind == "norm":
        y, mean, rstd = _norm(s["x"].float(), s["w"], s["b"])
        return {"y": y.to(DT[case["out"]]), "mean": mean, "rstd": rstd}
    if kind == "normgrad":
        dx, dw, db = _norm_grad(s["dy"].float(), s["x"].float(), s["mean"], s["rstd"], s["w"])
        return {"dx": dx.to(DT[case["dtype"]]), "dw": dw, "db": db}
    if kind == "quantise":
        x = s["x"].float()
        return {"rows": _values(x, case["fmt"], case["square"]).to(torch.bfloat16),
                "cols": _values(x.t(), case["fmt"], case["square"]).t().to(torch.bfloat16)}
    if kind == "product":
        out = _unpack(s["a"]) @ _unpack(s["b"]).t()
        return (out + s["bias"] if case["bias"] else out).to(DT[case["out"]])
    if kind == "backward":
        dy = s["dy"].float()
        dx = _values(dy, "e5m2", False) @ _unpack(s["w"]).t()
        return {"dx": dx.to(torch.bfloat16), "dw": _values(dy.t(), "e5m2", False) @ _unpack(s["x"]).t()}
    if kind == "layer":
        y, mean, rstd = _norm(s["x"].float(), s["w"], s["b"])
        y = y.to(torch.bfloat16).float()
        out = _values(y, "e4m3", False) @ _unpack(s["weight"]).t() + s["bias"]
        _moment(_values(y.t(), "e4m3", False), case["nb"], case["tokens"], case["beta"], s["A"][0])
        return {"out": out.to(torch.bfloat16), "mean": mean, "rstd": rstd, "A": s["A"][0]}
    if kind == "moment":
        [_moment(_unpack(op), nb, case["tokens"], case["beta"], A) for op, A, (_, nb) in zip(s["held"], s["A"], _weights(case))]
        return s["A"]
    x = torch.cat([_values(x.float().t(), "e4m3", False) for x in s["x"]], 1)
    _moment(x, case["nb"], case["tokens"], case["beta"], s["A"][0])
    return s["A"]


def _run_own(s, case):
    import block_diagonal_eigenbasis_amd as dobb
    kind = case["kind"]
    if kind == "norm":
        y, mean, rstd = dobb.dobb_layer_norm(s["x"], s["w"], s["b"], EPS, dtype=DT[case["out"]])
        return {"y": y, "mean": mean, "rstd": rstd}
    if kind == "normgrad":
        dx, dw, db = dobb.dobb_layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
        return {"dx": dx, "dw": dw, "db": db}
    if kind == "quantise":
        rows, cols = dobb.dobb_fp8_quantize(s["x"], rows=True, cols=True, fmt=case["fmt"], square=case["square"])
        return {"rows": dobb.dobb_fp8_dequantize(rows, torch.bfloat16),
                "cols": dobb.dobb_fp8_dequantize(cols, torch.bfloat16, transpose=True)}
    if kind == "product":
        return dobb.dobb_fp8_matmul(dobb.Fp8Operand(*s["a"]), dobb.Fp8Operand(*s["b"]), bias=s.get("bias"), dtype=DT[case["out"]])
    if kind == "backward":
        rows, cols = dobb.dobb_fp8_quantize(s["dy"], rows=True, cols=True, fmt="e5m2")
        return {"dx": dobb.dobb_fp8_matmul(rows, dobb.Fp8Operand(*s["w"]), dtype=torch.bfloat16),
                "dw": dobb.dobb_fp8_matmul(cols, dobb.Fp8Operand(*s["x"]), dtype=torch.float32)}
    if kind == "layer":
        rows, cols, mean, rstd = dobb.dobb_layer_norm_fp8(s["x"], s["w"], s["b"], EPS, rows=True, cols=True)
        out = dobb.dobb_fp8_matmul(rows, dobb.Fp8Operand(*s["weight"]), bias=s["bias"], dtype=torch.bfloat16)
        dobb.dobb_accumulate_moment_fp8(cols, s["A"][0], case["nb"], case["tokens"], case["beta"])
        return {"out": out, "mean": mean, "rstd": rstd, "A": s["A"][0]}
    if kind == "moment":
        dobb.dobb_accumulate_moment_fp8_grouped([dobb.Fp8Operand(*op) for op in s["held"]], s["A"], [nb for _, nb in _weights(case)],
                                                case["tokens"], case["beta"])
        return s["A"]
    held = [dobb.Fp8Capture.quantize(x) for x in s["x"]]
    held = dobb.Fp8Capture.cat(held)
    dobb.dobb_accumulate_moment_fp8(held.operand, s["A"][0], case["nb"], case["tokens"], case["beta"])
    return s["A"]


# ---- the definition in 64 bits -------------------------------------------------------------------
def _levels(fmt):
    """Every value from zero up that a format holds, by its code."""
    largest, bits, low, _ = FORMATS[fmt]
    code = np.arange(1 << 7)
    e, f = code >> bits, code & ((1 << bits) - 1)
    v = np.where(e == 0, f * 2.0 ** (low - bits), (1 + f / 2.0 ** bits) * 2.0 ** (e - 1.0 + low))
    return v[v <= largest]


def _two_to(k):
    """2^k in 64 bits for a tensor of whole numbers k."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _fp8_exact(x, fmt, square):
    """x (R x K) in FP8, in 64 bits: each entry takes the nearest level, of two equally near ones that with the
    even code, over its block's power of two."""
    lev = torch.tensor(_levels(fmt), dtype=torch.float64, device=x.device)
    mid = (lev[1:] + lev[:-1]) / 2
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for k in range(0, x.shape[1], 128):
        g = x[:, k:k + 128].double()
        top = g.abs().amax(1)
        if square:
            top = torch.cat([q.max().expand(len(q)) for q in top.split(128)])
        e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -160) / lev[-1]))
        e = torch.where(lev[-1] * _two_to(e - 1) >= top, e - 1, torch.where(lev[-1] * _two_to(e) < top, e + 1, e)).clamp(-127, 127)
        y = (g / _two_to(e)[:, None]).abs()
        # how many midpoints lie below y; one that y equals counts where the level above it is even
        i = torch.bucketize(y, mid)
        on = (mid[i.clamp(max=len(mid) - 1)] == y) & (i % 2 == 1)
        out[:, k:k + 128] = lev[i + on.long()] * torch.sign(g) * _two_to(e)[:, None]
    return out


def _operand_exact(op):
    """The values of an FP8 operand, R x K, in 64 bits."""
    codes, scales, K, fmt = op
    lev = torch.tensor(_levels(fmt), dtype=torch.float64, device=codes.device)
    T, _, R, _ = codes.shape
    out = torch.empty(R, T, 128, dtype=torch.float64, device=codes.device)
    for h in range(8):
        c = codes[:, h].permute(1, 0, 2).long()
        out[:, :, 16 * h:16 * h + 16] = torch.where(c >= 128, -1.0, 1.0).double() * lev[c & 127]
    return (out * _two_to(scales[:, :R].t().long() - 127)[:, :, None]).view(R, T * 128)[:, :K]


def _norm_exact(s):
    x, w, b = s["x"].double(), s["w"].double(), s["b"].double()
    var, mean = torch.var_mean(x, 1, correction=0)
    rstd = 1 / torch.sqrt(var + EPS)
    return torch.addcmul(b, (x - mean[:, None]) * rstd[:, None], w), mean, rstd


def _moment_exact(x, nb, N, beta, A):
    """x: columns x tokens."""
    g = torch.stack([x[b:b + nb] @ x[b:b + nb].T for b in range(0, x.shape[0], nb)])
    return beta * A.double() + (1 - beta) / N * g


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        return dict(zip(("y", "mean", "rstd"), _norm_exact(s)))
    if kind == "normgrad":
        # the gradient in terms of the centred rows: with u = x - mean and v = w dy,
        # dx = rstd (v - mean(v)) - rstd^3 u mean(u v)
        u, dy, r = s["x"].double() - s["mean"].double()[:, None], s["dy"].double(), s["rstd"].double()[:, None]
        v = dy * s["w"].double()
        return {"dx": r * (v - v.mean(1, keepdim=True)) - r ** 3 * u * (u * v).mean(1, keepdim=True),
                "dw": torch.einsum("tn,tn,t->n", dy, u, r[:, 0]), "db": dy.sum(0)}
    if kind == "quantise":
        x = s["x"]
        return {"rows": _fp8_exact(x, case["fmt"], case["square"]), "cols": _fp8_exact(x.t(), case["fmt"], case["square"]).t()}
    if kind == "product":
        out = _operand_exact(s["a"]) @ _operand_exact(s["b"]).T
        return out + s["bias"].double() if case["bias"] else out
    if kind == "backward":
        return {"dx": _fp8_exact(s["dy"], "e5m2", False) @ _operand_exact(s["w"]).T,
                "dw": _fp8_exact(s["dy"].t(), "e5m2", False) @ _operand_exact(s["x"]).T}
    if kind == "layer":
        y, mean, rstd = _norm_exact(s)
        y = y.to(torch.bfloat16)
        return {"out": _fp8_exact(y, "e4m3", False) @ _operand_exact(s["weight"]).T + s["bias"].double(), "mean": mean, "rstd": rstd,
                "A": _moment_exact(_fp8_exact(y.t(), "e4m3", False), case["nb"], case["tokens"], case["beta"], s["A"][0])}
    if kind == "moment":
        return [_moment_exact(_operand_exact(op), nb, case["tokens"], case["beta"], A)
                for op, A, (_, nb) in zip(s["held"], s["A"], _weights(case))]
    x = torch.cat([_fp8_exact(x.t(), "e4m3", False) for x in s["x"]], 1)
    return [_moment_exact(x, case["nb"], case["tokens"], case["beta"], s["A"][0])]
