"""The ways in which the FP8 products and moments (include/dobb_layers.h) divide their work: products in parts of k, by
tiles of 64 x 64 and 128 x 128, and thin ones; moments with some blocks whole and the others split along the tokens,
and more matrices than one launch holds.  Against 64 bits; bounds as in the operators' other tests:

* products: S = 8 matrix instructions for each tile of 128 entries at most, 2 S u sum |a b| with u = 2^-24, a rounding each
  for bias, old entry, result and every part that is added (32 at most); results in bf16 2^-10 sum |a b| and their own
  rounding besides;
* moments: (2 S + 3) u (1 - beta)/N sum_t |x_i x_j| + u |A_ij|, S over the tokens of one split.
"""
import numpy as np
import pytest
import torch

from layers_reference import U

pytestmark = pytest.mark.gpu
dobb = pytest.importorskip("block_diagonal_eigenbasis_amd")
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def values(R, K, seed, dtype=F32):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(R, K, generator=g, device=DEV) * torch.exp(torch.randn(K, generator=g, device=DEV))
    x = x * torch.exp(torch.randn(R, 1, generator=g, device=DEV))
    x[torch.rand(R, K, generator=g, device=DEV) < 0.05] = 0.0
    return x.to(dtype)


def launches(fn):
    """(fn's result, {kernel: launches})"""
    dobb.dobb_profile_reset()
    dobb.dobb_profile_enable(True)
    try:
        got = fn()
    finally:
        dobb.dobb_profile_enable(False)
    names = {k: v[0] for k, v in dobb.dobb_profile_read().items()}
    dobb.dobb_profile_reset()
    return got, names


def check(a, b, dtype, kernels, bias=None, out=None, accumulate=False):
    A, B = dobb.dobb_fp8_dequantize(a).double(), dobb.dobb_fp8_dequantize(b).double()
    zero = torch.zeros((), dtype=torch.float64, device=DEV)
    add, old = zero if bias is None else bias.double(), out.double().clone() if accumulate else zero
    got, names = launches(lambda: dobb.dobb_fp8_matmul(a, b, out=out, dtype=dtype, bias=bias, accumulate=accumulate))
    assert sorted(names) == sorted(kernels), names
    want, mags = A @ B.t() + add + old, A.abs() @ B.abs().t()
    tol = (2 * 8 * a.tiles + 32) * U * mags + 2 * U * (mags + add.abs() + old.abs())
    if got.dtype == BF16:
        tol = tol + 2.0 ** -10 * mags
    tol = tol + torch.finfo(got.dtype).eps / 2 * (want.abs() + tol)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), f"{int(bad.sum())} off, the first at {bad.nonzero()[0].tolist()}"
    return got


PARTS, THIN = ("fp8_matmul", "fp8_join"), ("fp8_matmul_thin",)


@pytest.mark.parametrize("M,N,K,kernels", [(300, 300, 11008, PARTS), (130, 1001, 9000, PARTS), (40, 50, 12000, PARTS), (33, 4100, 2000, PARTS),
                                           (500, 513, 5000, PARTS), (1600, 1600, 16384, PARTS), (1000, 1103, 9000, PARTS),
                                           (1, 4096, 11008, THIN), (32, 32, 16384, THIN), (1601, 7, 6400, THIN), (31, 1601, 1600, THIN)])
@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
def test_products(M, N, K, kernels, fa, fb):
    a, b = dobb.dobb_fp8_quantize(values(M, K, 1), fmt=fa)[0], dobb.dobb_fp8_quantize(values(N, K, 2), fmt=fb, square=True)[0]
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    bias = torch.randn(N, generator=g, device=DEV)
    for dtype in (F32, BF16):
        first = check(a, b, dtype, kernels)
        for _ in range(3):
            assert torch.equal(first, dobb.dobb_fp8_matmul(a, b, dtype=dtype))
        check(a, b, dtype, kernels, bias=bias)
        check(a, b, dtype, kernels, bias=bias.to(BF16))
        old = torch.randn(M, N, generator=g, device=DEV).to(dtype)
        check(a, b, dtype, kernels, out=old.clone(), accumulate=True)
        big = torch.full((M, N + 23), 5.0, dtype=dtype, device=DEV)
        check(a, b, dtype, kernels, out=big[:, 11:11 + N], accumulate=True, bias=bias)
        assert bool((big[:, :11] == 5.0).all()) and bool((big[:, 11 + N:] == 5.0).all())


def check_moments(ops, As, nbs, N, beta):
    old = [A.clone() for A in As]
    _, names = launches(lambda: dobb.dobb_accumulate_moment_fp8_grouped(ops, As, nbs, N, beta))
    b32 = float(np.float32(beta))
    for op, A, was, nb in zip(ops, As, old, nbs):
        S = 8 * min(op.tiles, 128)
        X = dobb.dobb_fp8_dequantize(op).double().view(A.shape[0], nb, -1)
        for i in range(A.shape[0]):
            g, mags = X[i] @ X[i].t(), X[i].abs() @ X[i].abs().t()
            want = (b32 * was[i].double() if beta > 0 else 0.0) + (1 - b32) / N * g
            tol = (2 * S + 3) * U * (1 - b32) / N * mags + U * want.abs() + 1e-44
            assert bool(((A[i].double() - want).abs() <= tol).all()), f"block {i} of width {nb}"
        assert torch.equal(A, A.transpose(1, 2))
    return names


def symmetric(B, nb, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    a = torch.randn(B, nb, nb, generator=g, device=DEV)
    return a + a.transpose(1, 2)


# 256 or 512 blocks whole and the rest in splits (100 x 260, 97 x 260, 128 x 300, 96 x 513); all split; all whole
@pytest.mark.parametrize("nb,B,N", [(100, 260, 16384), (97, 260, 5000), (128, 300, 16384), (96, 513, 9000), (32, 520, 16384), (400, 16, 16384),
                                    (200, 30, 3000), (16, 1000, 2000)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_moments(nb, B, N, fmt):
    x = values(N, nb * B, nb + N, BF16)
    op = dobb.dobb_fp8_quantize(x, rows=False, cols=True, fmt=fmt)[1]
    names = check_moments([op], [symmetric(B, nb, 1)], [nb], N, 0.9)
    if nb * B in (26000, 38400, 49248, 6400):
        assert len(names) == 2, names                             # the sums, and the splits' sums
    A = torch.full((B, nb, nb), float("nan"), device=DEV)         # not read where beta = 0
    check_moments([op], [A], [nb], N, 0.0)
    again = torch.empty_like(A)
    dobb.dobb_accumulate_moment_fp8(op, again, nb, N, 0.0)
    assert torch.equal(A, again)


def test_moments_of_more_matrices_than_a_launch_holds():
    N, count = 300, 200
    nbs = [(16, 24, 130)[i % 3] for i in range(count)]
    ops = [dobb.dobb_fp8_quantize(values(N, 2 * nb, i), rows=False, cols=True)[1] for i, nb in enumerate(nbs)]
    names = check_moments(ops, [symmetric(2, nb, i) for i, nb in enumerate(nbs)], nbs, N, 0.5)
    assert sum(names.values()) >= 3


def test_the_default_divisor_of_joined_captures():
    """Micro-batches of 100 and 77 tokens: the moment is that of the 177 tokens."""
    x = values(177, 60, 3)
    joined = dobb.Fp8Capture.cat([dobb.Fp8Capture.quantize(x[:100]), dobb.Fp8Capture.quantize(x[100:])])
    got = dobb.dobb_accumulate_moment_fp8(joined.operand, torch.empty(3, 20, 20, device=DEV), 20)
    assert torch.equal(got, dobb.dobb_accumulate_moment_fp8(joined.operand, torch.empty(3, 20, 20, device=DEV), 20, N=177))
    v = joined.dequantize().double().view(177, 3, 20).permute(1, 2, 0).contiguous()
    want, mags = v @ v.transpose(1, 2).contiguous() / 177, v.abs() @ v.abs().transpose(1, 2).contiguous() / 177
    assert bool(((got.double() - want).abs() <= (2 * 16 + 3) * U * mags + U * want.abs()).all())
