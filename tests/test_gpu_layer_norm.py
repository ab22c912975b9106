"""Layer norm forward and backward (include/dobb_layers.h) against the definition in 64 bits; the bounds
are derived beside the reference (layers_reference.py)."""
import numpy as np
import pytest
import torch

import layers_reference as ref
from layers_reference import U, host

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


def rand(*shape, seed=0, dtype=F32, scale=1.0, shift=0.0):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype).to(DEV)


def within(got, want, bound, what):
    got, want = host(got), np.asarray(want)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} off, worst {np.max(np.abs(got - want) / np.maximum(bound, 1e-300)):.3g} of the bound"


def half(dtype):
    return torch.finfo(dtype).eps


def check_forward(x, w, b, eps=1e-5, out=None, dtype=None):
    y, mean, rstd = dobb.dobb_layer_norm(x, w, b, eps, out=out, dtype=dtype)
    X, W, B = host(x), None if w is None else host(w), None if b is None else host(b)
    ry, rm, rr, _ = ref.norm(X, W, B, eps)
    by, bm, br = ref.norm_bounds(X, W, B, eps, half(y.dtype))
    within(mean, rm, bm, "mean")
    within(rstd, rr, br, "rstd")
    within(y, ry, by, "y")
    return y, mean, rstd


# widths at the edges of every kernel: 64 threads a row up to 1024 entries, then 128, 256, 512, 1024, then rows read again
WIDTHS = [1, 2, 7, 8, 9, 511, 512, 513, 768, 1024, 1025, 1600, 1601, 2048, 2049, 4096, 4097, 8192, 8193, 11008, 16384, 16385, 40001]


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward_widths(n, dtype):
    x = rand(5, n, seed=n, dtype=dtype, shift=0.3)
    w, b = rand(n, seed=n + 1, shift=1.0), rand(n, seed=n + 2)
    check_forward(x, w, b)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 63, 997, 4097])
def test_forward_rows(rows):
    check_forward(rand(rows, 200, seed=rows), None, None)
    check_forward(rand(rows, 1100, seed=rows, dtype=BF16), rand(1100, seed=1, dtype=BF16), rand(1100, seed=2, dtype=BF16))


@pytest.mark.parametrize("dtype,out", [(F32, BF16), (BF16, F32), (F32, F32), (BF16, BF16)])
@pytest.mark.parametrize("wt", [F32, BF16])
def test_forward_types(dtype, out, wt):
    x = rand(33, 130, seed=3, dtype=dtype)
    check_forward(x, rand(130, seed=4, dtype=wt), rand(130, seed=5, dtype=wt), dtype=out)
    check_forward(x, rand(130, seed=4, dtype=wt), None, dtype=out)
    check_forward(x, None, rand(130, seed=5, dtype=wt), dtype=out)


def test_forward_strided_unaligned_and_in_place():
    big = rand(9, 700, seed=1, dtype=BF16)
    x = big[:, 3:3 + 601]                                        # rows at odd offsets, not aligned to 16 bytes
    out = torch.full((9, 650), 7.0, device=DEV)
    y, _, _ = check_forward(x, None, None, out=out[:, 1:602])
    assert y.data_ptr() == out[:, 1:].data_ptr()
    rest = out.clone()
    rest[:, 1:602] = 7.0
    assert bool((rest == 7.0).all())                             # nothing beside it written
    for dtype in (F32, BF16):
        z = rand(6, 333, seed=2, dtype=dtype)
        want = dobb.dobb_layer_norm(z)[0]
        got = dobb.dobb_layer_norm(z, out=z)[0]
        assert got.data_ptr() == z.data_ptr() and torch.equal(got, want)


def test_forward_far_from_zero_constant_and_masked_rows():
    """Rows around 1000 with a spread of 1; equal entries (rstd = eps^-1/2, y = bias); and the entries that masked
    places hold: infinities and NaN stay in their row."""
    x = rand(4, 1600, seed=7, shift=1000.0)
    check_forward(x, rand(1600, seed=8), None)
    c = torch.full((3, 768), 0.37, device=DEV)
    b = rand(768, seed=9)
    y, mean, rstd = dobb.dobb_layer_norm(c, None, b)
    # the mean of equal entries is off by a rounding of theirs at most, which rstd (316) then multiplies
    assert float((mean - c[:, 0]).abs().max()) <= 3e-8
    within(rstd, np.full(3, 1e-5 ** -0.5), 1e-5 ** -0.5 * 4 * U + 1e-9, "rstd")
    within(y, host(b)[None, :].repeat(3, 0), 317 * 3e-8 + U * np.abs(host(b)), "y")
    z = rand(6, 1000, seed=10)
    want = dobb.dobb_layer_norm(z)[0]
    z[1, 17], z[3, 999], z[4, 0] = float("nan"), float("inf"), torch.finfo(F32).min
    y, mean, rstd = dobb.dobb_layer_norm(z)
    for r in (0, 2, 5):
        assert torch.equal(y[r], want[r])
    assert bool(y[1].isnan().all()) and bool(y[3].isnan().all())
    assert bool(rstd[1].isnan()) and bool(mean[1].isnan())


def test_eps_zero():
    x = rand(3, 64, seed=1)
    check_forward(x, None, None, eps=0.0)
    x[1] = 2.0
    y, _, rstd = dobb.dobb_layer_norm(x, eps=0.0)
    assert bool(y[1].isnan().all()) and not bool(rstd[1].isfinite()) and bool(y[[0, 2]].isfinite().all())


def check_backward(dy, x, w, eps=1e-5, **kw):
    _, mean, rstd = dobb.dobb_layer_norm(x, eps=eps)
    dx, dw, db = dobb.dobb_layer_norm_backward(dy, x, mean, rstd, w, **kw)
    (rx, rw, rb), (bx, bw, bb) = ref.norm_grad(host(dy), host(x), host(mean), host(rstd), None if w is None else host(w))
    within(dx, rx, bx + (U + half(dx.dtype) / 2) * np.abs(rx) + 1e-44, "dx")
    if dw is not None:
        within(dw, rw, bw + half(dw.dtype) / 2 * (np.abs(rw) + bw) + 1e-44, "dweight")
    if db is not None:
        within(db, rb, bb + half(db.dtype) / 2 * (np.abs(rb) + bb) + 1e-44, "dbias")
    return dx, dw, db


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_backward_widths(n, dtype):
    check_backward(rand(5, n, seed=n + 3, dtype=dtype), rand(5, n, seed=n, dtype=dtype, shift=0.3), rand(n, seed=n + 1, shift=1.0))


@pytest.mark.parametrize("rows", [1, 3, 4, 5, 511, 513, 2047, 2049, 5000])
@pytest.mark.parametrize("n", [24, 1030])
def test_backward_rows(rows, n):
    check_backward(rand(rows, n, seed=rows), rand(rows, n, seed=rows + 1), rand(n, seed=2))


@pytest.mark.parametrize("dyt,xt,dxt,wt", [(F32, BF16, F32, BF16), (BF16, F32, BF16, F32), (BF16, BF16, F32, BF16), (F32, F32, BF16, None)])
@pytest.mark.parametrize("n", [300, 17000])
def test_backward_types(dyt, xt, dxt, wt, n):
    w = None if wt is None else rand(n, seed=1, dtype=wt)
    _, dw, db = check_backward(rand(37, n, seed=2, dtype=dyt), rand(37, n, seed=3, dtype=xt), w, dtype=dxt)
    assert dw.dtype == db.dtype == (wt or F32)


def test_backward_targets_and_in_place():
    x, dy, w = rand(50, 513, seed=1), rand(50, 513, seed=2), rand(513, seed=3)
    dx, dw, db = check_backward(dy, x, w)
    assert check_backward(dy, x, w, dweight=False)[1] is None
    assert check_backward(dy, x, w, dbias=False)[2] is None
    dx2, dw2, db2 = check_backward(dy, x, w, dweight=False, dbias=False)
    assert dw2 is None and db2 is None and torch.equal(dx, dx2)
    tw, tb = torch.empty(513, dtype=BF16, device=DEV), torch.empty(513, dtype=BF16, device=DEV)
    check_backward(dy, x, w, dweight=tw, dbias=tb)
    _, mean, rstd = dobb.dobb_layer_norm(x)
    z = dy.clone()
    got = dobb.dobb_layer_norm_backward(z, x, mean, rstd, w, dX=z)
    assert got[0].data_ptr() == z.data_ptr() and torch.equal(got[0], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)
    big = torch.full((50, 700), 3.0, device=DEV)
    dobb.dobb_layer_norm_backward(dy, x, mean, rstd, w, dX=big[:, 5:518])
    assert torch.equal(big[:, 5:518], dx) and bool((big[:, :5] == 3.0).all()) and bool((big[:, 518:] == 3.0).all())


@pytest.mark.parametrize("n", [100, 600, 1600, 3000, 8000, 8193, 17000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_backward_in_place_at_every_width(n, dtype):
    """dX written over dY, rows read once or twice: the sums are those of the gradient as it was."""
    x, dy, w = rand(131, n, seed=1, dtype=dtype), rand(131, n, seed=2, dtype=dtype), rand(n, seed=3)
    _, mean, rstd = dobb.dobb_layer_norm(x, w)
    want = dobb.dobb_layer_norm_backward(dy, x, mean, rstd, w)
    got = dobb.dobb_layer_norm_backward(dy, x, mean, rstd, w, dX=dy)
    assert got[0].data_ptr() == dy.data_ptr() and all(torch.equal(p, q) for p, q in zip(got, want))
    y = dobb.dobb_layer_norm(x, w)[0]
    assert torch.equal(dobb.dobb_layer_norm(x, w, out=x)[0], y)


def test_backward_against_differences():
    """The gradient of sum(c y) for fixed c, by central differences of the forward pass in 64 bits."""
    x, w, b, c = rand(3, 40, seed=1), rand(40, seed=2, shift=1.0), rand(40, seed=3), rand(3, 40, seed=4)
    _, mean, rstd = dobb.dobb_layer_norm(x, w, b)
    got = dobb.dobb_layer_norm_backward(c, x, mean, rstd, w)
    X, W, B, C = host(x), host(w), host(b), host(c)
    loss = lambda X, W, B: (C * ref.norm(X, W, B, 1e-5)[0]).sum()  # noqa: E731
    h = 1e-6
    for k, (t, g) in enumerate(zip((X, W, B), got)):
        want = np.empty_like(t)
        for i in np.ndindex(t.shape):
            args = [[v.copy() for v in (X, W, B)] for _ in range(2)]
            args[0][k][i] += h
            args[1][k][i] -= h
            want[i] = (loss(*args[0]) - loss(*args[1])) / (2 * h)
        # differences: h^2 of a third derivative and 1e-16 / h of the loss, both below 1e-8; fp32 sums of 40 terms
        np.testing.assert_allclose(host(g), want, atol=1e-5, rtol=1e-5)


def test_repeats_bit_for_bit():
    x, dy, w = rand(3000, 1600, seed=1, dtype=BF16), rand(3000, 1600, seed=2, dtype=BF16), rand(1600, seed=3)
    a = dobb.dobb_layer_norm(x, w)
    first = (*a, *dobb.dobb_layer_norm_backward(dy, x, a[1], a[2], w))
    for _ in range(3):
        a = dobb.dobb_layer_norm(x, w)
        again = (*a, *dobb.dobb_layer_norm_backward(dy, x, a[1], a[2], w))
        assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_empty_refused():
    for shape in ((0, 8), (3, 0)):
        with pytest.raises(ValueError):
            dobb.dobb_layer_norm(torch.empty(*shape, device=DEV))
    x = rand(4, 8)
    m = torch.empty(4, device=DEV)
    with pytest.raises(ValueError):
        dobb.dobb_layer_norm(x.t())
    with pytest.raises(TypeError):
        dobb.dobb_layer_norm(x.half())
    with pytest.raises(TypeError):
        dobb.dobb_layer_norm(x, rand(8), rand(8, dtype=BF16))
    with pytest.raises(ValueError):
        dobb.dobb_layer_norm(x, rand(7))
    with pytest.raises(dobb.DobbError):
        dobb.dobb_layer_norm(x, eps=-1.0)
    with pytest.raises(dobb.DobbError):
        dobb.dobb_layer_norm(x, eps=float("nan"))
    with pytest.raises(dobb.DobbError):                           # mean written over x
        dobb.dobb_layer_norm(x, mean=x.view(-1)[:4])
    with pytest.raises(ValueError):
        dobb.dobb_layer_norm_backward(x[:2], x, m, m)
    with pytest.raises(dobb.DobbError):                           # dX written over X
        dobb.dobb_layer_norm_backward(rand(4, 8, seed=1), x, m, m, dX=x)
