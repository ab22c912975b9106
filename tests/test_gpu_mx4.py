"""Captures in MXFP4 and the second moments from them (include/dobb_ops.h) against the definitions in
64 bits.

* Codes and scales have to be the definition's exactly (ties go to the even element), and reading back is
  exact in fp32, and in bf16 for values in its normal range.
* Moments: a wave runs S matrix instructions in a row, four for each pair of token tiles, over at most 16
  pairs (blocks of up to 128 columns: four waves share a split of 16384 tokens) or 64 (wider blocks: every
  wave runs over the whole split).  Each adds an fp32
  rounding of a partial sum that is at most sum_t |x_i x_j|; twice u = 2^-24 of that is allowed for an
  instruction (its own sum of 64 products was measured below u of their magnitudes), then three additions
  over waves and one rounding of the result: (2 S + 3) u (1 - beta)/N sum_t |x_i x_j| + u |A_ij|.
  beta is a float in the C ABI (0.9f is 2.4e-8 below 0.9, and 1 - beta 2.4e-7 relative above 0.1), so the
  reference takes the float's value.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
dobb = pytest.importorskip("block_diagonal_eigenbasis_amd")
DEV = "cuda"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def ref_quantize(x):
    """(codes T x 4 x n x 16, scales T x n x 4, values N x n) of a float64 array, from the definition."""
    N, n = x.shape
    T = -(-N // 128)
    p = np.zeros((T * 128, n))
    p[:N] = x
    p = p.reshape(T, 4, 32, n)
    top = np.abs(p).max(2)
    bad = ~np.isfinite(top)
    _, e = np.frexp(np.where(bad | (top == 0), 1.0, top))        # top = m 2^e with m in [0.5, 1)
    S = np.where(top == 0, -127, np.maximum(e - 1 - 2, -127))
    y = np.abs(np.where(bad[:, :, None], 0.0, p)) / (2.0 ** S)[:, :, None]
    d = np.abs(y[..., None] - LEVELS)                             # nearest level, ties to the even index
    best = d.min(-1, keepdims=True)
    near = d == best
    even = near & (np.arange(8) % 2 == 0)
    k = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    neg = np.signbit(np.where(bad[:, :, None], 0.0, p))
    code = (k + 8 * neg).astype(np.uint8)
    val = LEVELS[k] * np.where(neg, -1, 1) * (2.0 ** S)[:, :, None]
    val = np.where(bad[:, :, None], np.nan, val)
    c = code.transpose(0, 1, 3, 2)
    codes = c[..., 0::2] | (c[..., 1::2] << 4)
    scales = np.where(bad, 255, S + 127).astype(np.uint8).transpose(0, 2, 1)
    return codes, scales, val.reshape(T * 128, n)[:N]


def activations(N, n, seed, dtype=F32):
    g = torch.Generator()
    g.manual_seed(seed)
    x = torch.randn(N, n, generator=g) * torch.exp(torch.randn(n, generator=g)) * torch.exp(0.5 * torch.randn(N, 1, generator=g))
    x[torch.rand(N, n, generator=g) < 0.05] = 0.0
    return x.to(dtype).to(DEV)


def host(t):
    return t.detach().to("cpu", torch.float64).numpy()


def check_quantize(x):
    codes, scales = dobb.dobb_mx4_quantize(x)
    rc, rs, rv = ref_quantize(host(x))
    np.testing.assert_array_equal(scales.cpu().numpy(), rs)
    np.testing.assert_array_equal(codes.cpu().numpy(), rc)
    return codes, scales, rv


SIZES = [(1, 1), (300, 1), (1, 400), (31, 3), (32, 128), (33, 129), (127, 2), (128, 127), (129, 5), (257, 130), (1000, 400), (4096, 192)]


@pytest.mark.parametrize("N,n", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_and_read_back(N, n, dtype):
    print(f"quantize: {N} x {n} {dtype}", flush=True)
    x = activations(N, n, 1000 * N + n, dtype)
    codes, scales, rv = check_quantize(x)
    for out in (F32, BF16):
        got = dobb.dobb_mx4_dequantize(codes, scales, N, out)
        assert got.dtype == out
        np.testing.assert_array_equal(host(got), rv)
    if N > 1:      # fewer tokens than are held
        np.testing.assert_array_equal(host(dobb.dobb_mx4_dequantize(codes, scales, N - 1)), rv[:-1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,n,ld,off", [(130, 100, 101, 1), (64, 33, 100, 3), (200, 256, 777, 5)])
def test_rows_of_a_wider_unaligned_buffer(dtype, N, n, ld, off):
    buf = activations(N + 1, ld, 5, dtype).reshape(-1)
    x = buf[off:off + N * ld].view(N, ld)[:, :n]
    assert not x.is_contiguous()
    codes, scales, rv = check_quantize(x)
    held = torch.full((N * ld + off,), 7.0, dtype=dtype, device=DEV)
    out = held[off:].view(N, ld)[:, :n]
    dobb.dobb_mx4_dequantize(codes, scales, N, out=out)
    np.testing.assert_array_equal(host(out), rv)
    out.fill_(7.0)
    assert bool((held == 7.0).all())      # what lies between and behind the rows is as it was


def test_every_tie_and_border():
    """All multiples of 1/8 up to 8 at several scales, and their fp32 neighbours."""
    k = np.arange(64) / 8.0
    cols = []
    for e in (-126, -125, -60, -3, 0, 1, 40, 122, 125):
        v = np.float32(k * 2.0 ** e)
        for w in (v, -v, np.nextafter(v, np.float32(np.inf)), np.nextafter(v, np.float32(0))):
            for half in (w[:32], w[32:]):
                cols.append(np.where(np.isfinite(half), half, 0.0))
    x = torch.tensor(np.stack(cols, 1), dtype=F32, device=DEV)
    x[31, ::2] = torch.sign(x[31, ::2]) * 2.0 ** 3          # another largest entry for half of the columns
    codes, scales, rv = check_quantize(x)
    np.testing.assert_array_equal(host(dobb.dobb_mx4_dequantize(codes, scales, 32)), rv)


def test_zeros_subnormals_and_largest():
    x = torch.zeros(64, 8, device=DEV)
    x[:, 1] = -0.0
    x[5, 2] = 2.0 ** -149
    x[:32, 3] = torch.tensor([2.0 ** -127 * i / 8 for i in range(32)], device=DEV)
    x[40, 4] = 3.4028234663852886e38
    x[41, 4] = -3.4028234663852886e38
    x[:, 5] = 2.0 ** -126
    x[63, 6] = -2.0 ** -130
    codes, scales, rv = check_quantize(x)
    got = host(dobb.dobb_mx4_dequantize(codes, scales, 64))
    np.testing.assert_array_equal(got, rv)
    assert np.signbit(got[:, 1]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_groups_that_are_not_finite_read_back_as_nan(dtype, bad):
    x = activations(100, 6, 3, dtype)
    x[40, 2] = bad
    x[99, 5] = bad
    codes, scales, rv = check_quantize(x)
    got = host(dobb.dobb_mx4_dequantize(codes, scales, 100))
    np.testing.assert_array_equal(got, rv)
    assert np.isnan(got[32:64, 2]).all() and np.isnan(got[96:, 5]).all() and np.isnan(got).sum() == 36


def test_quantize_into_the_tiles_of_a_larger_capture():
    xs = [activations(k, 70, 60 + k, BF16) for k in (100, 128, 300)]
    T = [dobb.mx4_tiles(x.shape[0]) for x in xs]
    codes = torch.full((sum(T), 4, 70, 16), 0xAA, dtype=torch.uint8, device=DEV)
    scales = torch.full((sum(T), 70, 4), 0xAA, dtype=torch.uint8, device=DEV)
    at = 0
    for x, t in zip(xs, T):
        dobb.dobb_mx4_quantize(x, codes[at:at + t], scales[at:at + t])
        at += t
    want = [dobb.dobb_mx4_quantize(x) for x in xs]
    assert torch.equal(codes, torch.cat([c for c, _ in want])) and torch.equal(scales, torch.cat([s for _, s in want]))


# ---- moments -------------------------------------------------------------------------------------
def ref_moment(x, nb, N, beta, A):
    """(the blocks, the magnitudes their roundings are of)."""
    n = x.shape[1]
    beta = float(np.float32(beta))
    xb = x.reshape(-1, n // nb, nb)
    g = np.einsum("tbi,tbj->bij", xb, xb, optimize=True)
    m = np.einsum("tbi,tbj->bij", np.abs(xb), np.abs(xb), optimize=True)
    return beta * A + (1 - beta) / N * g, (1 - beta) / N * m


def check_moment(got, x, nb, N, beta, A, tiles):
    want, m = ref_moment(x, nb, N, beta, A)
    S = 4 * min(-(-tiles // 2), 16 if nb <= 128 else 64)
    got = host(got)
    tol = (2 * S + 3) * U * m + U * np.abs(want)
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / np.maximum(tol, 1e-300)).max())
    np.testing.assert_array_equal(got, got.transpose(0, 2, 1))


def sym(n, nb, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    a = torch.randn(n // nb, nb, nb, generator=g)
    return (a + a.transpose(1, 2)).to(DEV)


@pytest.mark.parametrize("nb,B", [(1, 3), (2, 17), (5, 4), (16, 3), (31, 2), (32, 4), (33, 3), (48, 16), (64, 2), (65, 1), (96, 2),
                                  (100, 5), (127, 1), (128, 3), (129, 2), (192, 4), (200, 1), (255, 1), (257, 1), (400, 2),
                                  (768, 1), (1024, 1)])
@pytest.mark.parametrize("N,beta", [(1, 0.0), (37, 0.9), (128, 0.0), (300, 0.5), (2100, 0.9)])
def test_moment(nb, B, N, beta):
    print(f"moment: nb={nb} B={B} N={N} beta={beta}", flush=True)
    n = nb * B
    codes, scales = dobb.dobb_mx4_quantize(activations(N, n, 7 * nb + N, BF16))
    x = host(dobb.dobb_mx4_dequantize(codes, scales, N))
    A0 = sym(n, nb, nb)
    A = A0.clone() if beta > 0 else torch.full_like(A0, float("nan"))     # not read when beta is 0
    out = dobb.dobb_accumulate_moment_mx4(codes, scales, A, nb, N, beta)
    assert out is A
    check_moment(A, x, nb, N, beta, host(A0) if beta > 0 else 0.0, codes.shape[0])
    again = A0.clone()
    dobb.dobb_accumulate_moment_mx4(codes, scales, again, nb, N, beta)
    assert torch.equal(again, A)


@pytest.mark.parametrize("nb,n,N", [(64, 128, 16385), (200, 200, 40000), (8, 64, 70000), (128, 256, 130 * 128)])
def test_moment_of_long_captures(nb, n, N):
    """More tokens than one split may hold, and token tiles that do not divide evenly into splits."""
    print(f"long moment: nb={nb} n={n} N={N}", flush=True)
    codes, scales = dobb.dobb_mx4_quantize(activations(N, n, 9, BF16))
    x = host(dobb.dobb_mx4_dequantize(codes, scales, N))
    A = sym(n, nb, 2)
    A0 = host(A)
    dobb.dobb_accumulate_moment_mx4(codes, scales, A, nb, N, 0.25)
    check_moment(A, x, nb, N, 0.25, A0, codes.shape[0])


def test_moment_of_all_negative_and_of_one_sided_sums():
    """Products of one sign, where sums grow and roundings do not cancel."""
    x = -activations(16384, 32, 4, F32).abs() - 0.1
    codes, scales = dobb.dobb_mx4_quantize(x)
    xq = host(dobb.dobb_mx4_dequantize(codes, scales, 16384))
    A = torch.empty(1, 32, 32, device=DEV)
    dobb.dobb_accumulate_moment_mx4(codes, scales, A, 32, 16384)
    check_moment(A, xq, 32, 16384, 0.0, 0.0, 128)


def test_moment_of_wide_ranging_scales():
    """Columns from 2^-60 to 2^55 in one block: every product is exact, whatever its neighbours."""
    x = activations(500, 116, 8, F32) * 2.0 ** torch.arange(-60, 56, device=DEV, dtype=F32)
    codes, scales = dobb.dobb_mx4_quantize(x)
    xq = host(dobb.dobb_mx4_dequantize(codes, scales, 500))
    A = torch.empty(1, 116, 116, device=DEV)
    dobb.dobb_accumulate_moment_mx4(codes, scales, A, 116, 500)
    check_moment(A, xq, 116, 500, 0.0, 0.0, 4)


@pytest.mark.parametrize("nb,bad", [(100, 37), (192, 150), (192, 191)])
def test_moment_of_a_nan_column(nb, bad):
    x = activations(300, 2 * nb, 6, F32)
    x[290, bad] = float("nan")
    codes, scales = dobb.dobb_mx4_quantize(x)
    A = torch.empty(2, nb, nb, device=DEV)
    dobb.dobb_accumulate_moment_mx4(codes, scales, A, nb, 300)
    nan = A.isnan().cpu().numpy()
    want = np.zeros((2, nb, nb), bool)
    want[0, bad, :] = want[0, :, bad] = True
    np.testing.assert_array_equal(nan, want)


@pytest.mark.parametrize("N", [200, 3000])
def test_moment_grouped_over_mixed_shapes(N):
    print(f"grouped moment: N={N}", flush=True)
    dims = [(256, 64), (400, 100), (256, 64), (400, 200), (256, 64)] + [(96, 48)] * 50
    caps = [dobb.dobb_mx4_quantize(activations(N, n, 30 + i, BF16)) for i, (n, _) in enumerate(dims)]
    As = [sym(n, nb, i) for i, (n, nb) in enumerate(dims)]
    A0 = [host(a) for a in As]
    dobb.dobb_accumulate_moment_mx4_grouped([c for c, _ in caps], [s for _, s in caps], As, [nb for _, nb in dims], N, 0.9)
    for (c, s), A, a0, (n, nb) in zip(caps, As, A0, dims):
        check_moment(A, host(dobb.dobb_mx4_dequantize(c, s, N)), nb, N, 0.9, a0, c.shape[0])


def test_micro_batches_joined_by_their_tiles():
    """Captures of 100, 128 and 77 tokens one behind the other: the zeros that fill a tile add nothing."""
    xs = [activations(k, 200, 70 + k, BF16) for k in (100, 128, 77)]
    caps = [dobb.dobb_mx4_quantize(x) for x in xs]
    codes, scales = torch.cat([c for c, _ in caps]), torch.cat([s for _, s in caps])
    xq = np.concatenate([host(dobb.dobb_mx4_dequantize(c, s, x.shape[0])) for (c, s), x in zip(caps, xs)])
    A = sym(200, 100, 3)
    A0 = host(A)
    dobb.dobb_accumulate_moment_mx4(codes, scales, A, 100, 305, 0.5)
    check_moment(A, xq, 100, 305, 0.5, A0, 3)


def test_capture_on_a_stream_of_its_own():
    x = activations(1500, 400, 12, BF16)
    A = torch.empty(4, 100, 100, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    codes, scales = dobb.dobb_mx4_quantize(x, stream=s)
    dobb.dobb_accumulate_moment_mx4(codes, scales, A, 100, 1500, stream=s)
    out = dobb.dobb_mx4_dequantize(codes, scales, 1500, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    check_moment(A, host(out), 100, 1500, 0.0, 0.0, 12)
    np.testing.assert_array_equal(host(out), ref_quantize(host(x))[2])


def test_graph_replays():
    x = activations(2000, 384, 13, BF16)
    A = sym(384, 192, 1)
    codes, scales = dobb.dobb_mx4_quantize(x)
    ws = torch.empty(max(256, dobb.dobb_moment_mx4_workspace_size([(1, 384, 192)], codes.shape[0])), dtype=torch.uint8, device=DEV)
    out = torch.empty(2000, 384, device=DEV)

    def go(A):
        dobb.dobb_mx4_quantize(x, codes, scales)
        dobb.dobb_accumulate_moment_mx4(codes, scales, A, 192, 2000, 0.5, ws=ws)
        dobb.dobb_mx4_dequantize(codes, scales, 2000, out=out)
    go(A.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(A)
    for it in range(4):
        x.copy_(activations(2000, 384, 40 + it, BF16))
        eager = A.clone()
        go(eager)
        values = out.clone()
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(A, eager) and torch.equal(out, values)


def test_refusals():
    x = activations(200, 64, 1, F32)
    codes, scales = dobb.dobb_mx4_quantize(x)
    A = torch.zeros(1, 64, 64, device=DEV)
    with pytest.raises(ValueError, match="column stride"):
        dobb.dobb_mx4_quantize(x.T)
    with pytest.raises(ValueError, match="rows that do not overlap"):
        dobb.dobb_mx4_quantize(x[:1].expand(5, 64))
    with pytest.raises(ValueError, match="at least one"):
        dobb.dobb_mx4_quantize(x[:0])
    with pytest.raises(TypeError, match="dtype"):
        dobb.dobb_mx4_quantize(x.half())
    with pytest.raises(ValueError, match="tokens x columns"):
        dobb.dobb_mx4_quantize(x.view(2, 100, 64))
    with pytest.raises(ValueError, match="codes must have shape"):
        dobb.dobb_mx4_quantize(x, codes[:1], scales)
    with pytest.raises(ValueError, match="N must be"):
        dobb.dobb_mx4_dequantize(codes, scales, 257)
    with pytest.raises(ValueError, match="scales must have shape"):
        dobb.dobb_mx4_dequantize(codes, scales[:1], 200)
    with pytest.raises(ValueError, match="out must have shape"):
        dobb.dobb_mx4_dequantize(codes, scales, 200, out=torch.empty(199, 64, device=DEV))
    with pytest.raises(ValueError, match="does not divide"):
        dobb.dobb_accumulate_moment_mx4(codes, scales, A, 60, 200)
    with pytest.raises(ValueError, match="A must have shape"):
        dobb.dobb_accumulate_moment_mx4(codes, scales, A, 32, 200)
    with pytest.raises(dobb.DobbError):
        dobb.dobb_accumulate_moment_mx4(codes, scales, A, 64, 257)
    with pytest.raises(dobb.DobbError):
        dobb.dobb_accumulate_moment_mx4(codes, scales, A, 64, 200, 1.0)
    with pytest.raises(ValueError, match="number of tiles"):
        dobb.dobb_accumulate_moment_mx4_grouped([codes, codes[:1]], [scales, scales[:1]], [A, A.clone()], [64, 64], 100)


def test_shared_captures_and_repeated_moments():
    """One capture for several weights (q, k and v see the same activations) is in order; one moment listed
    twice would be written by two workgroups and is refused."""
    codes, scales = dobb.dobb_mx4_quantize(activations(300, 128, 2, BF16))
    As = [torch.empty(2, 64, 64, device=DEV) for _ in range(3)]
    dobb.dobb_accumulate_moment_mx4_grouped([codes] * 3, [scales] * 3, As, [64] * 3, 300)
    assert torch.equal(As[0], As[1]) and torch.equal(As[0], As[2])
    check_moment(As[0], host(dobb.dobb_mx4_dequantize(codes, scales, 300)), 64, 300, 0.0, 0.0, 3)
    with pytest.raises(dobb.DobbError):
        dobb.dobb_accumulate_moment_mx4_grouped([codes] * 2, [scales] * 2, [As[0], As[0]], [64] * 2, 300)


def test_two_captures_at_once_on_two_streams():
    xs = [activations(3000, 400, 80 + i, BF16) for i in range(2)]
    want = []
    for x in xs:
        c, s = dobb.dobb_mx4_quantize(x)
        want.append(dobb.dobb_accumulate_moment_mx4(c, s, torch.empty(1, 400, 400, device=DEV), 400, 3000))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [torch.empty(1, 400, 400, device=DEV) for _ in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        for x, st, A in zip(xs, streams, got):
            c, s = dobb.dobb_mx4_quantize(x, stream=st)
            dobb.dobb_accumulate_moment_mx4(c, s, A, 400, 3000, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_negated_views_are_refused():
    x = torch.randn(40, 8, dtype=torch.complex64, device=DEV).conj().imag
    assert x.is_neg()
    with pytest.raises(ValueError, match="negated view"):
        dobb.dobb_mx4_quantize(x)
