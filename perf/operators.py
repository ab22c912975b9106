"""Cases of the operators around the Dobb step: gradient norm and clipping, and MXFP4 captures.

The kinds of case, as a training program meets them:

* norm     the norms of every gradient of a list, and the global norm (what a run logs each step);
* clip     the same, and the gradients scaled by min(1, max_norm / (total + 1e-6)) into the optimizer's
           own buffers (same type, or bf16 gradients into fp32 main gradients);
* quantise activations to MXFP4 (e2m1 elements, one power-of-two scale per 32 tokens of a column), and
           the values read back;
* moment   captures held in MXFP4 into the second-moment blocks
           A_b <- beta A_b + (1 - beta)/N sum_t x_t x_t^T;
* capture  the two in a row: micro-batches quantised as they come, then the moment from all of them.

Gradients are views of one flat buffer per type, as gradient buckets hold them, with no padding
between tensors, so that odd sizes leave the next tensor unaligned.  Captures in MXFP4 are held in tiles
of 128 tokens: codes (tiles, 4 groups of 32 tokens, columns, 16 bytes; the even token in the low half of
a byte) and scales (tiles, columns, 4 groups), the missing tokens of the last tile being zeros.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}

# the weights of a layer (rows, columns) and their block widths: the GPT-2 XL set with 16 blocks a
# weight, and the 7B-style stack with blocks of 128
XL = [(4800, 1600, 100), (1600, 1600, 100), (6400, 1600, 100), (1600, 6400, 400)]
SEVEN = [(4096, 4096, 128)] * 4 + [(11008, 4096, 128)] * 2 + [(4096, 11008, 128)]
SETS = {"xl": XL, "7b": SEVEN}


def listed():
    return [
        # one small weight: the call's latency
        dict(name="norm one 768x768", kind="norm", sizes="one", numel=768 * 768, dtype="fp32", norm=0.7),
        # one layer of the 7B-style stack, bf16 gradients
        dict(name="norm 7b layer bf16", kind="norm", sizes="7b", layers=1, dtype="bf16", norm=2.0),
        # one layer of the GPT-2 XL set in fp32, clipped
        dict(name="clip xl layer fp32", kind="clip", sizes="xl", layers=1, dtype="fp32", out="fp32", norm=3.7, max_norm=1.0),
        # every parameter of a small model: many little tensors of odd sizes, both types, unaligned views
        dict(name="clip ragged mixed", kind="clip", sizes="ragged", count=331, lo=1, hi=200000, shape_seed=5, dtype="mixed",
             out="same", norm=1.9, max_norm=0.5),
        # all 192 weights of the GPT-2 XL set, bf16 gradients
        dict(name="clip xl set bf16", kind="clip", sizes="xl", layers=48, dtype="bf16", out="bf16", norm=5.0, max_norm=1.0),
        # a slice of wider rows, a token count that ends inside a group of 32
        dict(name="quantise rows of a slice", kind="quantise", tokens=997, n=1600, ld=4800, dtype="fp32", out="fp32"),
        # the widest capture of the GPT-2 XL set
        dict(name="quantise fc-proj", kind="quantise", tokens=16384, n=6400, ld=6400, dtype="bf16", out="bf16"),
        # the single-weight configuration
        dict(name="moment one 768", kind="moment", sizes="one", n=768, nb=192, tokens=4096, beta=0.0),
        # twelve layers of the GPT-2 XL set in one grouped call
        dict(name="moment xl 12 layers", kind="moment", sizes="xl", layers=12, tokens=16384, beta=0.9),
        # a layer of the 7B-style stack
        dict(name="moment 7b layer", kind="moment", sizes="7b", layers=1, tokens=4096, beta=0.9),
        # a capture of a few tokens
        dict(name="capture few tokens", kind="capture", n=400, nb=100, tokens=37, parts=1, dtype="fp32", beta=0.0),
        # three micro-batches of a wide weight, none of them a whole number of tiles
        dict(name="capture fc-proj parts", kind="capture", n=6400, nb=400, tokens=8193, parts=3, dtype="bf16", beta=0.9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "clip", "quantise", "moment", "capture"])
    if kind in ("norm", "clip"):
        c = dict(kind=kind, sizes="ragged", count=_log(rng, 1, 400), lo=1, hi=_log(rng, 1000, 3000000), shape_seed=rng.randrange(1 << 20),
                 dtype=rng.choice(["fp32", "bf16", "mixed"]), norm=round(rng.uniform(0.3, 6.0), 3))
        if kind == "clip":
            c.update(out=rng.choice(["same", "fp32", "bf16"]), max_norm=rng.choice([0.5, 1.0, 2.0]))
        return c
    if kind == "quantise":
        tokens = _log(rng, 1, 16384)
        n = _log(rng, 1, min(11008, 16384 * 6400 // tokens))
        return dict(kind=kind, tokens=tokens, n=n, ld=n + rng.choice([0, 0, 1, 8, n]), dtype=rng.choice(["fp32", "bf16"]),
                    out=rng.choice(["fp32", "bf16"]))
    nb = _log(rng, 1, 1024)
    n = nb * _log(rng, 1, max(1, min(32, 8192 // nb)))
    tokens = _log(rng, 1, 16384)
    c = dict(kind=kind, n=n, nb=nb, tokens=tokens, beta=rng.choice([0.0, 0.5, 0.9]))
    if kind == "moment":
        c.update(sizes="one")
    else:
        c.update(parts=min(tokens, rng.choice([1, 2, 5])), dtype=rng.choice(["fp32", "bf16"]))
    return c


# ---- shapes ------------------------------------------------------------------------------------
def _numels(case):
    """(elements, type) of every gradient of a norm or clip case."""
    if case["sizes"] == "one":
        numels = [case["numel"]]
    elif case["sizes"] == "ragged":
        r = random.Random(case["shape_seed"])
        numels = [_log(r, case["lo"], case["hi"]) for _ in range(case["count"])]
    else:
        numels = [m * n for _ in range(case["layers"]) for m, n, _ in SETS[case["sizes"]]]
    kinds = ["fp32", "bf16"] if case["dtype"] == "mixed" else [case["dtype"]]
    return [(k, kinds[i % len(kinds)]) for i, k in enumerate(numels)]


def _weights(case):
    """(columns, block width) of every capture of a moment or capture case."""
    if case.get("sizes", "one") == "one":
        return [(case["n"], case["nb"])]
    return [(n, nb) for _ in range(case["layers"]) for _, n, nb in SETS[case["sizes"]]]


def _out_type(case, dtype):
    return dtype if case["out"] == "same" else case["out"]


def _parts(case):
    """Tokens of every micro-batch of a capture case: as even as they come."""
    N, P = case["tokens"], case["parts"]
    return [N * (i + 1) // P - N * i // P for i in range(P)]


def _views(flat, numels):
    out, at = [], {k: 0 for k in flat}
    for k, dt in numels:
        out.append(flat[dt][at[dt]:at[dt] + k])
        at[dt] += k
    return out


def work(case):
    size = {"fp32": 4, "bf16": 2}
    if case["kind"] in ("norm", "clip"):
        numels = _numels(case)
        total = sum(k for k, _ in numels)
        b = sum(k * size[dt] for k, dt in numels) + 4 * (len(numels) + 1)
        if case["kind"] == "clip":
            b += sum(k * size[_out_type(case, dt)] for k, dt in numels)
        return {"bytes": b, "flops": (3 if case["kind"] == "clip" else 2) * total}
    N = case["tokens"]
    if case["kind"] == "quantise":
        e = N * case["n"]
        return {"bytes": e * (size[case["dtype"]] + 17 / 32 + size[case["out"]]), "flops": 4 * e}
    b = f = 0
    for n, nb in _weights(case):
        b += n * nb * (8 if case["beta"] > 0 else 4)
        b += N * n * (17 / 32 if case["kind"] == "moment" else size[case["dtype"]])
        f += N * n * (nb + 1)
    return {"bytes": b, "flops": f}


# ---- inputs ------------------------------------------------------------------------------------
def _activations(N, n, gen):
    """Rows of tokens: normal entries, columns of log-normal size with a few far larger ones, and tokens
    of differing size, as the inputs of linear layers come."""
    col = torch.randn(n, generator=gen, device=DEV).mul_(0.8).exp_()
    col = torch.where(torch.rand(n, generator=gen, device=DEV) < 0.01, 20 * col, col)
    tok = torch.randn(N, 1, generator=gen, device=DEV).mul_(0.3).exp_()
    return torch.randn(N, n, generator=gen, device=DEV).mul_(col).mul_(tok)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = {"case": case}
    if case["kind"] in ("norm", "clip"):
        numels = _numels(case)
        total = sum(k for k, _ in numels)
        held = {dt: sum(k for k, d in numels if d == dt) for dt in sorted({d for _, d in numels})}
        flat = {dt: torch.empty(k, dtype=DT[dt], device=DEV) for dt, k in held.items()}
        for f in flat.values():
            f.normal_(0.0, case["norm"] / math.sqrt(total), generator=gen)
        s["grads"] = _views(flat, numels)
        if len(s["grads"]) > 1:        # layers differ in size by factors
            sizes = torch.randn(len(s["grads"]), generator=gen, device=DEV).mul_(0.5).exp_().tolist()
            for g, x in zip(s["grads"], sizes):
                g.mul_(x)
        if case["kind"] == "clip":
            to = [(k, _out_type(case, dt)) for k, dt in numels]
            s["flat"] = {dt: torch.empty(sum(k for k, d in to if d == dt), dtype=DT[dt], device=DEV) for dt in sorted({d for _, d in to})}
            s["outs"] = _views(s["flat"], to)
        s["norms"] = torch.empty(len(numels), device=DEV)
        s["total"] = torch.empty((), device=DEV)
        return s
    N = case["tokens"]
    if case["kind"] == "quantise":
        x = _activations(N, case["ld"], gen).to(DT[case["dtype"]])
        s["x"] = x[:, :case["n"]]
        return s
    s["A"] = []
    for n, nb in _weights(case):
        if case["kind"] == "moment":
            s.setdefault("held", []).append(_pack(_activations(N, n, gen)))
        else:
            s["x"] = [_activations(k, n, gen).to(DT[case["dtype"]]) for k in _parts(case)]
        a = torch.randn(n // nb, nb, nb, generator=gen, device=DEV)
        s["A"].append(a + a.transpose(1, 2))
    return s


# ---- the plain forms ---------------------------------------------------------------------------
def _norms(grads):
    """Norm of every tensor and of all of them; the sums in 64 bits."""
    sq = torch.stack([g.float().square().sum(dtype=torch.float64) for g in grads])
    return sq.sqrt().float(), sq.sum().sqrt().float()


def _tiled(x):
    """Rows of tokens (N x n) in tiles of four groups of 32 tokens, zeros behind the last token."""
    N, n = x.shape
    T = (N + 127) // 128
    p = torch.zeros(T * 128, n, dtype=torch.float32, device=x.device)
    p[:N] = x
    return p.view(T, 4, 32, n)


def _pow2(e):
    """2^e for whole e from -127 to 127, exact (a library power need not be)."""
    return torch.where(e == -127, 1 << 22, (e + 127) << 23).to(torch.int32).view(torch.float32)


def _elements(x):
    """(signed e2m1 values, exponents) of x in groups: nearest values, ties to even, over the power of two
    that brings each group's largest entry into [4, 8), what is over 6 being 6."""
    t = _tiled(x)
    top = t.abs().amax(2, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(-127, 127)
    y = t * _pow2(-e)
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp(max=6.0), y), e


def _pack(x):
    """Codes (T, 4, n, 16) and scales (T, n, 4) of x."""
    v, e = _elements(x)
    a = v.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code + 8 * torch.signbit(v).to(torch.uint8)
    code = code.permute(0, 1, 3, 2).contiguous()
    codes = code[..., 0::2] + 16 * code[..., 1::2]
    return codes, (e + 127).to(torch.uint8)[:, :, 0].permute(0, 2, 1).contiguous()


def _unpack(codes, scales, N):
    """The values that codes and scales stand for, N x n."""
    T, _, n, _ = codes.shape
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    code = torch.stack([codes & 15, codes >> 4], -1).view(T, 4, n, 32)
    v = table[code.int()] * _pow2(scales.permute(0, 2, 1).unsqueeze(-1).int() - 127)
    return v.permute(0, 1, 3, 2).reshape(T * 128, n)[:N]


def _values(x):
    v, e = _elements(x)
    return (v * _pow2(e)).reshape(-1, x.shape[1])[:x.shape[0]]


def _moment(x, nb, N, beta, A):
    """A <- beta A + (1 - beta) / N X_b^T X_b over blocks of nb columns; products over 1024 tokens in 32 bits,
    those added in 64 (the diagonal's terms are all of one sign)."""
    rows, n = x.shape
    C = (rows + 1023) // 1024
    p = torch.zeros(C * 1024, n, device=x.device) if rows % 1024 else x
    if rows % 1024:
        p[:rows] = x
    xb = p.view(C, 1024, n // nb, nb).permute(2, 0, 3, 1).reshape(-1, nb, 1024)
    g = torch.bmm(xb, xb.transpose(1, 2).contiguous()).view(n // nb, C, nb, nb).sum(1, dtype=torch.float64)
    A.copy_(beta * A + (1 - beta) / N * g if beta > 0 else g / N)


# ---- one pass ----------------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["kind"] == "norm":
        norms, total = _norms(s["grads"])
        return {"norms": norms, "total": total}
    if case["kind"] == "clip":
        norms, total = _norms(s["grads"])
        coef = (case["max_norm"] / (total + 1e-6)).clamp(max=1.0)
        [o.copy_(g.float() * coef) for o, g in zip(s["outs"], s["grads"])]
        return {"norms": norms, "total": total, **s["flat"]}
    if case["kind"] == "quantise":
        return _values(s["x"].float()).to(DT[case["out"]])
    if case["kind"] == "moment":
        [_moment(_unpack(c, e, case["tokens"]), nb, case["tokens"], case["beta"], A)
         for (c, e), A, (_, nb) in zip(s["held"], s["A"], _weights(case))]
        return s["A"]
    x = torch.cat([_values(x.float()) for x in s["x"]])
    _moment(x, case["nb"], case["tokens"], case["beta"], s["A"][0])
    return s["A"]


def _run_own(s, case):
    import block_diagonal_eigenbasis_amd as dobb
    if case["kind"] == "norm":
        dobb.dobb_grad_norm_grouped(s["grads"], norms=s["norms"], total=s["total"])
        return {"norms": s["norms"], "total": s["total"]}
    if case["kind"] == "clip":
        dobb.dobb_clip_grad_norm_grouped(s["grads"], case["max_norm"], outs=s["outs"], norms=s["norms"], total=s["total"])
        return {"norms": s["norms"], "total": s["total"], **s["flat"]}
    if case["kind"] == "quantise":
        codes, scales = dobb.dobb_mx4_quantize(s["x"])
        return dobb.dobb_mx4_dequantize(codes, scales, case["tokens"], DT[case["out"]])
    if case["kind"] == "moment":
        dobb.dobb_accumulate_moment_mx4_grouped([c for c, _ in s["held"]], [e for _, e in s["held"]], s["A"],
                                                [nb for _, nb in _weights(case)], case["tokens"], case["beta"])
        return s["A"]
    held = [dobb.dobb_mx4_quantize(x) for x in s["x"]]
    codes, scales = held[0] if len(held) == 1 else (torch.cat([h[0] for h in held]), torch.cat([h[1] for h in held]))
    dobb.dobb_accumulate_moment_mx4(codes, scales, s["A"][0], case["nb"], case["tokens"], case["beta"])
    return s["A"]


# ---- the definition in 64 bits -------------------------------------------------------------------
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _two_to(k):
    """2^k in 64 bits for a tensor of whole numbers k."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _mx_exact(x):
    """x (N x n, any type) in MXFP4, in 64 bits: each entry takes the nearest of LEVELS, of two equally near
    ones that with the even index, over its group's power of two."""
    lev = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    mid = (lev[1:] + lev[:-1]) / 2
    rows = []
    for t in range(0, x.shape[0], 32):
        g = x[t:t + 32].double()
        top = g.abs().max(0).values
        e = torch.floor(torch.log2(top.clamp(min=2.0 ** -140)))
        e = e + (_two_to(e + 1) <= top).double() - (_two_to(e) > top).double()
        scale = _two_to((e - 2).clamp(-127, 127))
        y = (g / scale).abs()
        # how many midpoints lie below y; one that y equals counts where the level above it is even
        k = torch.bucketize(y, mid)
        on = torch.isin(y, mid) & (k % 2 == 1)
        rows.append(lev[k + on.long()] * torch.sign(g) * scale)
    return torch.cat(rows)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] in ("norm", "clip"):
        sq = [torch.linalg.vector_norm(g.double()) ** 2 for g in s["grads"]]
        total = torch.sqrt(sum(sq))
        got = {"norms": torch.sqrt(torch.stack(sq)), "total": total}
        if case["kind"] == "clip":
            scale = min(1.0, case["max_norm"] / (float(total) + 1e-6))
            by = {dt: [] for dt in s["flat"]}
            for g, (_, dt) in zip(s["grads"], _numels(case)):
                by[_out_type(case, dt)].append(g.double() * scale)
            got.update({dt: torch.cat(v) for dt, v in by.items()})
        return got
    if case["kind"] == "quantise":
        return _mx_exact(s["x"])
    out = []
    for i, ((n, nb), A) in enumerate(zip(_weights(case), s["A"])):
        if case["kind"] == "moment":
            codes, scales = s["held"][i]
            T = codes.shape[0]
            lev = torch.tensor(np.concatenate([LEVELS, -LEVELS]), dtype=torch.float64, device=codes.device)
            x = torch.empty(T, 4, 32, n, dtype=torch.float64, device=codes.device)
            for k in range(32):
                nibble = (codes[..., k // 2] >> (4 * (k % 2))) & 15
                x[:, :, k] = lev[nibble.long()] * _two_to(scales.permute(0, 2, 1).long() - 127)
            x = x.view(T * 128, n)[:case["tokens"]]
        else:
            x = torch.cat([_mx_exact(p) for p in s["x"]])
        a = torch.stack([x[:, b:b + nb].T @ x[:, b:b + nb] for b in range(0, n, nb)])
        out.append(case["beta"] * A.double() + (1 - case["beta"]) / case["tokens"] * a)
    return out
