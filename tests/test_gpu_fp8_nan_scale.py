"""A scale byte of 255 stands for NaN, whatever codes the block holds: an operand may come from elsewhere, and its entries
read back as NaN.  Every product and moment of such a block is NaN, by each kernel and for either type of result."""
import pytest
import torch

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


def operand(R, K, seed, fmt, cols=False):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(R, K, generator=g, device=DEV)
    return dobb.dobb_fp8_quantize(x.t().contiguous() if cols else x, rows=not cols, cols=cols, fmt=fmt)[cols]


# thin either way, 64 x 64 tiles whole and in parts, 128 x 128 whole and in parts, 256 x 256
@pytest.mark.parametrize("M,N,K", [(5, 70, 300), (70, 5, 300), (90, 77, 300), (300, 300, 11008), (2050, 2060, 300), (1000, 1103, 9000),
                                   (4352, 8448, 300)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_products(M, N, K, fmt, dtype):
    a, b = operand(M, K, 1, fmt), operand(N, K, 2, "e4m3")
    want = dobb.dobb_fp8_matmul(a, b, dtype=dtype)
    a.codes[1, :, M - 1] = 0                                      # zeros, and ordinary values
    a.scales[1, M - 1] = 255
    a.scales[0, 0] = 255
    assert bool(dobb.dobb_fp8_dequantize(a)[M - 1, 128:256].isnan().all())
    got, turned = dobb.dobb_fp8_matmul(a, b, dtype=dtype), dobb.dobb_fp8_matmul(b, a, dtype=dtype)
    assert bool(got[[0, M - 1]].isnan().all()) and bool(turned[:, [0, M - 1]].isnan().all())
    assert torch.equal(got[1:M - 1], want[1:M - 1]) and bool(turned[:, 1:M - 1].isfinite().all())


@pytest.mark.parametrize("nb", [32, 120, 200])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_moments(nb, fmt):
    op = operand(3 * nb, 300, 1, fmt, cols=True)
    want = dobb.dobb_accumulate_moment_fp8(op, torch.empty(3, nb, nb, device=DEV), nb)
    op.codes[2, :, nb + 8] = 0
    op.scales[2, nb + 8] = 255
    op.scales[0, 2 * nb] = 255
    A = dobb.dobb_accumulate_moment_fp8(op, torch.empty(3, nb, nb, device=DEV), nb)
    for blk, i in ((1, 8), (2, 0)):
        assert bool(A[blk, i].isnan().all()) and bool(A[blk, :, i].isnan().all())
        A[blk, i], A[blk, :, i] = want[blk, i], want[blk, :, i]
    assert torch.equal(A, want)
