"""The launches that production sizes take and small ones do not, against 64 bits on the GPU:

* moments of more blocks than the chip runs at once, whose last round alone is split over the tokens (its
  blocks, partial sums and reduction are counted from the first split block on), with several matrices in the
  launch and the border inside one of them;
* captures above 128 MB, which the narrow kernel reads past the caches;
* more matrices of one width than a launch takes, whose launches share the workspace;
* more gradients than a table of the norm's second kernel takes;
* captures whose sums fp32 holds exactly, where the result has one rounding and no more.

Tolerances of the moments: a wave runs S matrix instructions in a row, at most 64 (blocks of up to 128 columns)
or 256; twice u = 2^-24 of the magnitudes' sum is allowed for each (one rounding of the running sum, and the
instruction's own sum of 64 products, measured below u), three additions over waves, one rounding of a split's
partial sum and one of the result: (2 S + 4) u (1 - beta)/N sum_t |x_i x_j| + u |A_ij|, with the float beta.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
dobb = pytest.importorskip("block_diagonal_eigenbasis_amd")
DEV = "cuda"
U = 2.0 ** -24
F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def activations(N, n, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(N, n, generator=g, device=DEV)
    return x.mul_(torch.randn(n, generator=g, device=DEV).exp_()).mul_(torch.randn(N, 1, generator=g, device=DEV).mul_(0.5).exp_()).to(BF16)


def sym(B, nb, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    a = torch.randn(B, nb, nb, generator=g, device=DEV)
    return a + a.transpose(1, 2)


def check(A, A0, codes, scales, nb, N, beta):
    """A against the definition in 64 bits, block by block."""
    x = dobb.dobb_mx4_dequantize(codes, scales, N)
    b = float(np.float32(beta))
    S = 4 * min((codes.shape[0] + 1) // 2, 16 if nb <= 128 else 64)
    worst = torch.zeros((), dtype=F64, device=DEV)
    for k in range(A.shape[0]):
        xb = x[:, k * nb:(k + 1) * nb].to(F64)
        xt = xb.T.contiguous()
        want = (1 - b) / N * (xt @ xb)
        m = (1 - b) / N * (xt.abs() @ xb.abs())
        if beta > 0:
            want += b * A0[k].to(F64)
        tol = (2 * S + 4) * U * m + U * want.abs()
        worst = torch.maximum(worst, ((A[k].to(F64) - want).abs() / tol.clamp(min=1e-300)).max())
    assert float(worst) <= 1.0, float(worst)
    assert torch.equal(A, A.transpose(1, 2))


def al256(k):
    return -(-k // 256) * 256


# block width, blocks a matrix, matrices, tokens; the blocks that fill the chip's rounds stay whole
MIXED = [(16, 57, 9, 8192), (32, 80, 7, 16384), (100, 64, 9, 16384), (129, 26, 10, 4096), (192, 27, 10, 8192),
         (300, 20, 7, 4096), (400, 20, 7, 4096), (400, 1, 140, 2500)]


@pytest.mark.parametrize("nb,B,mats,N", MIXED)
@pytest.mark.parametrize("beta", [0.0, 0.9])
def test_moments_whose_last_round_is_split(nb, B, mats, N, beta):
    print(f"mixed plan: nb={nb} {mats} x {B} blocks N={N} beta={beta}", flush=True)
    n, tiles = nb * B, dobb.mx4_tiles(N)
    if mats <= 96:
        ws = dobb.dobb_moment_mx4_workspace_size([(1, n, nb)] * mats, tiles)
        assert 0 < ws < al256(2 * mats * B * nb * nb * 4)      # split, but not all blocks of the launch
    caps = [dobb.dobb_mx4_quantize(activations(N, n, 100 + i)) for i in range(mats)]
    As = [sym(B, nb, i) if beta else torch.full((B, nb, nb), math.nan, device=DEV) for i in range(mats)]
    A0 = [a.clone() for a in As]
    dobb.dobb_accumulate_moment_mx4_grouped([c for c, _ in caps], [s for _, s in caps], As, [nb] * mats, N, beta)
    for (c, s), a, a0 in zip(caps, As, A0):
        check(a, a0, c, s, nb, N, beta)


@pytest.mark.parametrize("nb", [16, 64, 96, 128])
def test_moment_of_a_capture_above_128_mb(nb):
    print(f"read past the caches: nb={nb}", flush=True)
    B, N = 5376 // nb, 50001
    n = nb * B
    codes, scales = dobb.dobb_mx4_quantize(activations(N, n, nb))
    assert codes.numel() + scales.numel() > 128 << 20
    A = sym(B, nb, 1)
    A0 = A.clone()
    dobb.dobb_accumulate_moment_mx4(codes, scales, A, nb, N, 0.5)
    check(A, A0, codes, scales, nb, N, 0.5)


@pytest.mark.parametrize("n,nb,N", [(96, 48, 5000), (200, 200, 5000), (64, 64, 300)])
def test_more_matrices_than_a_launch_takes(n, nb, N):
    print(f"200 matrices: n={n} nb={nb} N={N}", flush=True)
    caps = [dobb.dobb_mx4_quantize(activations(N, n, i)) for i in range(200)]
    As = [sym(n // nb, nb, i) for i in range(200)]
    A0 = [a.clone() for a in As]
    dobb.dobb_accumulate_moment_mx4_grouped([c for c, _ in caps], [s for _, s in caps], As, [nb] * 200, N, 0.9)
    for (c, s), a, a0 in zip(caps, As, A0):
        check(a, a0, c, s, nb, N, 0.9)


@pytest.mark.parametrize("count", [900, 901, 1900])
def test_norms_of_more_gradients_than_a_table_takes(count):
    print(f"norms: {count}", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(count)
    sizes = [1 + (7919 * i) % 9001 if i % 17 else 0 for i in range(count)]
    flat = torch.randn(sum(sizes), generator=g, device=DEV)
    ts = list(flat.split(sizes))
    for i in range(0, count, 3):
        ts[i] = ts[i].to(BF16)
    norms = torch.full((count,), 7.0, device=DEV)
    outs = [torch.empty_like(t) for t in ts]
    total = dobb.dobb_clip_grad_norm_grouped(ts, 1.0, outs=outs, norms=norms)
    sq = torch.stack([t.double().square().sum() for t in ts])
    want = sq.sqrt()
    assert bool(((norms.double() - want).abs() <= 1.01 * U * want).all())
    all_ = float(sq.sum().sqrt())
    assert abs(float(total) - all_) <= 1.01 * U * all_
    c = min(1.0, 1.0 / (all_ + 1e-6))
    for o, t in zip(outs, ts):
        want = c * t.double()
        tol = (6 * U + (2.0 ** -8 * (1 + 6 * U) if t.dtype == BF16 else 0.0)) * want.abs() + 2.0 ** -134
        assert bool(((o.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantise_ties_borders_and_subnormals_by_type(dtype):
    """Every multiple of 1/8 up to 8 at scales down to the subnormal ones, signed zeros, the largest values, and
    the type's neighbours of each: codes, scales and values have to be the definition's."""
    k = torch.arange(64, dtype=F64) / 8.0
    cols = []
    for e in (-136, -133, -128, -127, -126, -125, -124, -60, -3, 0, 1, 40, 122, 124, 125):
        v = (k * 2.0 ** e).to(dtype)
        bits = v.view(torch.int16 if dtype == BF16 else torch.int32)
        for w in (bits, bits + 1, (bits - 1).clamp(min=0)):
            w = w.view(dtype)
            w = torch.where(w.isfinite(), w, torch.zeros((), dtype=dtype))
            for half in (w[:32], w[32:]):
                cols += [half, -half]
    zeros = torch.zeros(32, dtype=dtype)
    top = torch.finfo(dtype).max
    cols += [zeros, -zeros, torch.full((32,), top, dtype=dtype), torch.tensor([top, -top] * 16, dtype=dtype)]
    x = torch.stack(cols, 1)
    N, n = x.shape
    xd = x.double()
    big = xd.abs().amax(0)
    # floor(log2) of a double from its exponent field: exact
    e = ((big.view(torch.int64) >> 52) & 2047) - 1023
    S = torch.where(big > 0, (e - 2).clamp(min=-127), torch.tensor(-127))
    scale = torch.ldexp(torch.ones(n, dtype=F64), S.to(torch.int32))
    y = xd.abs() / scale
    lev = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=F64)
    off = (y.unsqueeze(-1) - lev).abs()
    near = off == off.amin(-1, keepdim=True)
    even = near & (torch.arange(8) % 2 == 0)
    code = torch.where(even.any(-1), even.int().argmax(-1), near.int().argmax(-1))
    neg = xd.signbit()
    value = torch.where(neg, -1.0, 1.0) * lev[code] * scale
    codes, scales = dobb.dobb_mx4_quantize(x.to(DEV))
    nib = (code + 8 * neg).to(torch.uint8).T                     # n x 32
    want = nib[:, 0::2] | (nib[:, 1::2] << 4)
    assert torch.equal(scales.cpu()[0, :, 0], (S + 127).to(torch.uint8))
    assert torch.equal(codes.cpu()[0, 0], want)
    assert not bool(codes[0, 1:].any()) and not bool(scales[0, :, 1:].any())
    got = dobb.dobb_mx4_dequantize(codes, scales, N).cpu()
    assert torch.equal(got.double(), value) and torch.equal(got.signbit(), neg)
    got = dobb.dobb_mx4_dequantize(codes, scales, N, BF16).cpu()
    assert torch.equal(got, value.float().to(BF16))


# block width, blocks a matrix, matrices, tiles
EXACT = [(1, 40, 1, 3), (16, 57, 9, 64), (32, 5, 2, 127), (33, 7, 1, 1), (64, 9, 3, 129), (100, 64, 9, 128), (100, 16, 1, 128),
         (128, 4, 7, 32), (129, 26, 10, 32), (192, 4, 1, 32), (255, 3, 1, 5), (300, 20, 7, 32), (400, 4, 5, 400), (512, 2, 1, 128),
         (544, 1, 1, 33), (1024, 1, 2, 128)]


@pytest.mark.parametrize("nb,B,mats,tiles", EXACT)
@pytest.mark.parametrize("beta", [0.0, 0.5])
def test_sums_that_fp32_holds_are_rounded_once(nb, B, mats, tiles, beta):
    """Columns whose groups all have one scale: products are multiples of a quarter of two scales' product, at
    most 36 times it, so every partial sum over less than 2^24 / 144 = 116508 tokens is exact in fp32, in
    whatever order.  What is left is the rounding of the result to fp32, half a step."""
    print(f"exact sums: nb={nb} {mats} x {B} blocks {tiles} tiles beta={beta}", flush=True)
    n, N = nb * B, 128 * tiles - 19
    g = torch.Generator(device=DEV)
    g.manual_seed(nb + tiles)
    caps, As = [], []
    for i in range(mats):
        codes = torch.randint(0, 256, (tiles, 4, n, 16), generator=g, device=DEV, dtype=torch.uint8)
        col = torch.randint(117, 138, (n,), generator=g, device=DEV, dtype=torch.uint8)
        caps.append((codes, col.view(1, n, 1).expand(tiles, n, 4).contiguous()))
        As.append(sym(B, nb, i) if beta else torch.full((B, nb, nb), math.nan, device=DEV))
    A0 = [a.clone() for a in As]
    dobb.dobb_accumulate_moment_mx4_grouped([c for c, _ in caps], [s for _, s in caps], As, [nb] * mats, N, beta)
    for (c, s), a, a0 in zip(caps, As, A0):
        x = dobb.dobb_mx4_dequantize(c, s, 128 * tiles)          # the tiles are full: N is the divisor alone
        for k in range(B):
            xb = x[:, k * nb:(k + 1) * nb].to(F64)
            want = (1 - beta) / N * (xb.T.contiguous() @ xb)
            if beta:
                want += beta * a0[k].to(F64)
            assert bool(((a[k].to(F64) - want).abs() <= U * (1 + 2.0 ** -20) * want.abs()).all()), k
        assert torch.equal(a, a.transpose(1, 2))
