"""Operands and results of the layer operators (include/dobb_layers.h) larger than 4 GB: what lies past 2^32 bytes, or 2^31
entries, against 64 bits.  Rows are picked at the start, in the middle and at the end; the bounds are those of the
operators' own tests."""
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
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("80 GB of memory")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def matrix(R, K, seed, dtype=BF16):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(R, K, generator=g, device=DEV, dtype=dtype)


def picked(R):
    return [0, 1, R // 2, R // 2 + 1, R - 130, R - 2, R - 1]


def rows_of(op, rows):
    """The values of some rows, from the layout: codes [tile][16-entry group][row], scales [tile][row]."""
    types = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
    out = []
    for r in rows:
        v = op.codes[:, :, r].contiguous().view(types[op.fmt]).double().reshape(op.tiles, 128)
        two_to = (op.scales[:, r].long() - 127 + 1023 << 52).view(torch.float64)      # (a library power need not be exact)
        out.append((v * two_to[:, None]).reshape(-1)[:op.K])
    return torch.stack(out)


def check(got, want, mags, terms, exact):
    tol = (2 * 8 * -(-terms // 128) + 34) * U * mags + (0 if exact else 2.0 ** -10 * mags)
    tol = tol + torch.finfo(got.dtype).eps / 2 * (want.abs() + tol)
    assert bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_an_operand_of_more_than_4_gb(fmt):
    R, K = 140000, 33000
    x = matrix(R, K, 1)
    rows, cols = dobb.dobb_fp8_quantize(x, cols=True, fmt=fmt)
    assert rows.codes.numel() > 1 << 32 and cols.codes.numel() > 1 << 32
    at = picked(R)
    want = dobb.dobb_fp8_quantize(x[at].contiguous(), fmt=fmt)[0]
    assert torch.equal(rows.codes[:, :, at], want.codes) and torch.equal(rows.scales[:, at], want.scales[:, :len(at)])
    # the operand along the columns: its last tiles are those of the last tokens alone
    t0 = (cols.tiles - 2) * 128
    tail = dobb.dobb_fp8_quantize(x[t0:], rows=False, cols=True, fmt=fmt)[1]
    assert torch.equal(cols.codes[-2:], tail.codes) and torch.equal(cols.scales[-2:], tail.scales)
    del x
    back = dobb.dobb_fp8_dequantize(rows, BF16)
    A = rows_of(rows, at)
    assert torch.equal(back[at].double(), A)
    del back
    back = dobb.dobb_fp8_dequantize(cols, BF16, transpose=True)
    assert torch.equal(back[t0:], dobb.dobb_fp8_dequantize(tail, BF16, transpose=True))
    del back
    # thin, by tiles, and large; to both types
    for N in (20, 130, 1000):
        b = dobb.dobb_fp8_quantize(matrix(N, K, 2), fmt="e4m3")[0]
        B = dobb.dobb_fp8_dequantize(b).double()
        for dtype in (F32, BF16):
            got = dobb.dobb_fp8_matmul(rows, b, dtype=dtype)
            check(got[at], A @ B.t(), A.abs() @ B.abs().t(), K, dtype == F32)
    # contracted over the tokens, past the last of 2^32 bytes of codes
    N = 200
    b = dobb.dobb_fp8_quantize(matrix(R, N, 3), rows=False, cols=True)[1]
    B, at = dobb.dobb_fp8_dequantize(b).double(), picked(K)
    A = rows_of(cols, at)
    for dtype in (F32, BF16):
        got = dobb.dobb_fp8_matmul(cols, b, dtype=dtype)
        check(got[at], A @ B.t(), A.abs() @ B.abs().t(), R, dtype == F32)
    for nb in (100, 330):
        M = dobb.dobb_accumulate_moment_fp8(cols, torch.empty(K // nb, nb, nb, device=DEV), nb)
        for blk in (0, K // nb // 2, K // nb - 1):
            X = rows_of(cols, range(blk * nb, (blk + 1) * nb))
            check(M[blk], X @ X.t() / R, X.abs() @ X.abs().t() / R, R, True)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_result_of_more_than_2_31_entries(dtype):
    M, N, K = 70000, 33000, 200
    a, b = dobb.dobb_fp8_quantize(matrix(M, K, 1))[0], dobb.dobb_fp8_quantize(matrix(N, K, 2))[0]
    A, B = dobb.dobb_fp8_dequantize(a).double(), dobb.dobb_fp8_dequantize(b).double()
    at = picked(M)
    got = dobb.dobb_fp8_matmul(a, b, dtype=dtype)
    want, mags = A[at] @ B.t(), A[at].abs() @ B.abs().t()
    check(got[at], want, mags, K, dtype == F32)
    once = got[at].double()
    dobb.dobb_fp8_matmul(a, b, out=got, accumulate=True)
    check(got[at], want + once, mags + once.abs(), K, dtype == F32)


def test_a_norm_of_rows_that_lie_far_apart():
    """A slice of rows 2^30 entries apart, and a matrix of more than 2^31 entries."""
    far = matrix(3, 1, 1, F32).new_zeros(3, 1 << 30)
    far[:, 5:805] = matrix(3, 800, 1, F32)
    x = far[:, 5:805]
    w, b = matrix(1, 800, 2, F32)[0], matrix(1, 800, 3, F32)[0]
    dy = matrix(3, 800, 4, F32)
    y, mean, rstd = dobb.dobb_layer_norm(x, w, b)
    want = dobb.dobb_layer_norm(x.contiguous(), w, b)
    assert torch.equal(y, want[0]) and torch.equal(mean, want[1]) and torch.equal(rstd, want[2])
    for got, ref in zip(dobb.dobb_layer_norm_backward(dy, x, mean, rstd, w), dobb.dobb_layer_norm_backward(dy, x.contiguous(), mean, rstd, w)):
        assert torch.equal(got, ref)
    assert torch.equal(dobb.dobb_fp8_quantize(x)[0].codes, dobb.dobb_fp8_quantize(x.contiguous())[0].codes)
    out = torch.zeros(3, 1 << 30, device=DEV)[:, 7:807]
    dobb.dobb_layer_norm(x, w, b, out=out)
    assert torch.equal(out, y)
    del far, x, out
    for n in (1600, 9000, 20000):
        N = (1 << 31) // n + 1000
        x = matrix(N, n, 1)
        at = picked(N)
        y, mean, rstd = dobb.dobb_layer_norm(x)
        assert torch.equal(y[at], dobb.dobb_layer_norm(x[at].contiguous())[0])
        dx, _, db = dobb.dobb_layer_norm_backward(y, x, mean, rstd)
        assert torch.equal(dx[at], dobb.dobb_layer_norm_backward(y[at].contiguous(), x[at].contiguous(), mean[at], rstd[at])[0])
        # columns' sums: fp32 over at most 1024 rows, 1024 u of their magnitudes at most, and a rounding
        cols = slice(n - 64, n)
        s, mag = y[:, cols].double().sum(0), y[:, cols].double().abs().sum(0)
        assert bool(((db[cols].double() - s).abs() <= 1024 * U * mag + U * s.abs()).all())
        del x, y, dx
