"""The layer operators (include/dobb_layers.h) as a training step runs them: layer norm, FP8 operands, products,
gradients, captures and the optimizer's step in a row; replayed from a HIP graph; on a stream of the caller's.
"""
import numpy as np
import pytest
import torch

import layers_reference as ref
from layers_reference import U, host

pytestmark = pytest.mark.gpu
dobb = pytest.importorskip("block_diagonal_eigenbasis_amd")
from block_diagonal_eigenbasis_amd.optimizer import Dobb, DobbGroup  # noqa: E402

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


class Layer:
    """A layer norm and a linear map behind it, forward and backward, in FP8."""

    def __init__(self, n, m, seed=0):
        self.g, self.b = rand(n, seed=seed, scale=0.2, shift=1.0), rand(n, seed=seed + 1, scale=0.1)
        self.W, self.c = rand(m, n, seed=seed + 2, scale=n ** -0.5), rand(m, seed=seed + 3, scale=0.1)

    def step(self, x, dy):
        xr, xc, mean, rstd = dobb.dobb_layer_norm_fp8(x, self.g, self.b, rows=True, cols=True)
        wr, wc = dobb.dobb_fp8_quantize(self.W, cols=True, square=True)
        y = dobb.dobb_fp8_matmul(xr, wr, bias=self.c)
        dr, dc = dobb.dobb_fp8_quantize(dy, cols=True, fmt="e5m2")
        dh = dobb.dobb_fp8_matmul(dr, wc)
        dW = dobb.dobb_fp8_matmul(dc, xc, dtype=F32)
        dx, dg, db = dobb.dobb_layer_norm_backward(dh, x, mean, rstd, self.g)
        return dict(y=y, dh=dh, dW=dW, dx=dx, dg=dg, db=db, xr=xr, xc=xc, wr=wr, wc=wc, dr=dr, dc=dc, mean=mean, rstd=rstd)


def check_layer(layer, x, dy, got):
    """Every output against 64 bits, each from the operator's inputs as the step had them (bounds: as in the
    operators' own tests)."""
    v = {k: host(dobb.dobb_fp8_dequantize(got[k])) for k in ("xr", "xc", "wr", "wc", "dr", "dc")}
    assert np.array_equal(v["wr"], v["wc"].T)

    def product(out, a, b, add=0.0):
        want, mags = a @ b.T + add, np.abs(a) @ np.abs(b).T + np.abs(add)
        S = 8 * -(-a.shape[1] // 128)
        tol = (2 * S + 3) * U * mags + (2.0 ** -10 * mags if out.dtype == BF16 else 0.0)
        tol = tol + torch.finfo(out.dtype).eps / 2 * (np.abs(want) + tol)
        assert (np.abs(host(out) - want) <= tol).all()
    product(got["y"], v["xr"], v["wr"], host(layer.c))
    product(got["dh"], v["dr"], v["wc"])
    product(got["dW"], v["dc"], v["xc"])
    want, bounds = ref.norm_grad(host(got["dh"]), host(x), host(got["mean"]), host(got["rstd"]), host(layer.g))
    for k, w, b in zip(("dx", "dg", "db"), want, bounds):
        eps = torch.finfo(got[k].dtype).eps / 2
        assert (np.abs(host(got[k]) - w) <= b + eps * (np.abs(w) + b) + U * np.abs(w)).all(), k


@pytest.mark.parametrize("N,n,m", [(1, 48, 40), (333, 400, 520), (640, 768, 2304)])
def test_training_step(N, n, m):
    layer = Layer(n, m)
    x, dy = rand(N, n, seed=8, dtype=BF16, shift=0.1), rand(N, m, seed=9, dtype=BF16, scale=1e-3)
    got = layer.step(x, dy)
    check_layer(layer, x, dy, got)
    # near the step without rounding, by as much as FP8 allows: e4m3 is off by 2^-4 of a value at most, e5m2 by 2^-3
    h = ref.norm(host(x), host(layer.g), host(layer.b), 1e-5)[0]
    mags = np.abs(h) @ np.abs(host(layer.W)).T + np.abs(host(layer.c))
    assert (np.abs(host(got["y"]) - (h @ host(layer.W).T + host(layer.c))) <= 0.16 * mags).all()
    mags = np.abs(host(dy)).T @ np.abs(h)
    assert (np.abs(host(got["dW"]) - host(dy).T @ h) <= 0.22 * mags + 1e-12).all()


def test_captures_from_the_gradients_operand_in_the_optimizer():
    """Two micro-batches of a layer's step whose operands along the tokens are the optimizer's captures: the step is
    that of a group which is given the same values as fp32 tensors, up to the moments' rounding."""
    n, m, nb, sizes = 96, 64, 32, (300, 180)
    layer = Layer(n, m)
    p = torch.nn.Parameter(layer.W.clone())
    opt = Dobb([p], lr=0.01, block_size=nb, capture="all", refresh_period=2)
    twin = DobbGroup([layer.W.clone()], [nb], lr=0.01, momentum=0.9)
    for it in range(4):
        dW, kept = torch.zeros(m, n, device=DEV), []
        for k, N in enumerate(sizes):
            x, dy = rand(N, n, seed=10 * it + k, dtype=BF16), rand(N, m, seed=100 + 10 * it + k, dtype=BF16, scale=1e-2)
            _, xc, _, _ = dobb.dobb_layer_norm_fp8(x, layer.g, layer.b, rows=True, cols=True)
            dc = dobb.dobb_fp8_quantize(dy, rows=False, cols=True, fmt="e5m2")[1]
            dobb.dobb_fp8_matmul(dc, xc, out=dW, accumulate=True)
            kept.append(dobb.Fp8Capture(xc))
            if opt.wants_capture():
                opt.capture(p, kept[-1])
        p.grad = dW.clone()
        refresh = opt.wants_capture()
        opt.step()
        vals = dobb.Fp8Capture.cat(kept).dequantize()
        if it == 0:
            twin.refresh_step([vals], 0.0, dobb.DOBB_REFRESH_EXACT, 0, [dW], warm_start=False)
        elif refresh:
            twin.refresh_step([vals], 0.9, dobb.DOBB_REFRESH_ORTH_ITER, 1, [dW])
        else:
            twin.step([dW])
        A, B = opt._group.A[0], twin.A[0]
        # products exact on both sides; sums of 480 tokens in fp32 on one, fp32 and fp64 on the other
        assert float((A - B).abs().max()) <= 2e-6 * float(B.abs().max())
    assert float((p.data - twin.W[0]).abs().max()) <= 0.02 * 4 * 0.2 * 3 and bool(p.data.isfinite().all())


@pytest.mark.parametrize("fmt", ["native", "mx4", "fp8"])
def test_optimizer_with_every_capture_format(fmt):
    """What the optimizer keeps in FP8 through its hooks is what it would be given: the quantised values."""
    torch.manual_seed(0)
    lin = torch.nn.Linear(64, 48, bias=False, device=DEV)
    opt = Dobb([lin.weight], lr=0.01, block_size=16, capture_format=fmt)
    opt.attach_capture_hooks([lin])
    x = rand(200, 64, seed=1)
    lin(x).square().mean().backward()
    opt.step()
    vals = x if fmt == "native" else None
    if fmt == "fp8":
        vals = dobb.Fp8Capture.quantize(x).dequantize()
    if vals is not None:
        want = dobb.dobb_accumulate_moment(vals.contiguous(), torch.empty(4, 16, 16, device=DEV), 16)
        want = want if isinstance(want, torch.Tensor) else opt._group.A[0]
        assert float((opt._group.A[0] - want).abs().max()) <= 2e-6 * float(want.abs().max())


def test_group_of_mixed_captures_on_two_streams():
    dims = [(64, 400, 200), (48, 400, 200), (32, 384, 64), (16, 320, 32)]
    mk = lambda streams: DobbGroup([0.02 * rand(m, n, seed=i) for i, (m, n, _) in enumerate(dims)], [nb for _, _, nb in dims],  # noqa: E731
                                   streams=streams)
    xs = [rand(1500, n, seed=20 + i, dtype=BF16) for i, (_, n, _) in enumerate(dims)]
    caps = [dobb.Fp8Capture.quantize(xs[0]), xs[1], dobb.Fp8Capture.quantize(xs[2], "e5m2"), dobb.Fp8Capture.quantize(xs[3])]
    a, b = mk(1), mk(2)
    grads = [rand(m, n, seed=40 + i) for i, (m, n, _) in enumerate(dims)]
    for g in (a, b):
        g.refresh_step(caps, 0.0, dobb.DOBB_REFRESH_EXACT, 0, grads, warm_start=False)
        g.refresh_step(caps, 0.9, dobb.DOBB_REFRESH_ORTH_ITER, 1, grads)
    torch.cuda.synchronize()
    for i, c in enumerate(caps):
        vals = c.dequantize() if isinstance(c, dobb.Fp8Capture) else c.float()
        nb = dims[i][2]
        X = host(vals)
        for k in range(X.shape[1] // nb):
            want = X[:, k * nb:(k + 1) * nb].T @ X[:, k * nb:(k + 1) * nb] / 1500
            assert np.abs(host(a.A[i][k]) - want).max() <= 2e-6 * np.abs(want).max()
    # (another partition of the set may split the tokens otherwise)
    assert all(float((p - q).abs().max()) <= 2e-6 * float(q.abs().max()) for p, q in zip(a.A, b.A))


def test_graph_replays_with_new_inputs():
    """A step captured once and replayed with other inputs in the same buffers, between eager calls: every replay
    is the eager result bit for bit."""
    N, n, m, nb = 515, 400, 520, 100
    layer = Layer(n, m)
    x, dy = rand(N, n, seed=1, dtype=BF16), rand(N, m, seed=2, dtype=BF16)
    A = torch.zeros(n // nb, nb, nb, device=DEV)

    def step():
        r = layer.step(x, dy)
        dobb.dobb_accumulate_moment_fp8(r["xc"], A, nb, N, 0.5)
        return [r[k] for k in ("y", "dh", "dW", "dx", "dg", "db")] + [A]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in range(4):
        x.copy_(rand(N, n, seed=50 + k, dtype=BF16))
        dy.copy_(rand(N, m, seed=60 + k, dtype=BF16))
        A.copy_(torch.zeros_like(A) + k)
        want = [t.clone() for t in step()]
        A.copy_(torch.zeros_like(A) + k)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, want))


def test_group_graph_holds_fp8_captures():
    g = DobbGroup([0.02 * rand(64, 400, seed=1)], [100])
    cap = dobb.Fp8Capture.quantize(rand(2000, 400, seed=2))
    grads = [rand(64, 400, seed=3)]
    g.refresh_step([cap], 0.0, dobb.DOBB_REFRESH_EXACT, 0, grads, warm_start=False)
    twin = DobbGroup([0.02 * rand(64, 400, seed=1)], [100])
    twin.refresh_step([cap], 0.0, dobb.DOBB_REFRESH_EXACT, 0, grads, warm_start=False)
    graph = g.capture_refresh_step([cap], 0.9, dobb.DOBB_REFRESH_ORTH_ITER, 1, grads)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        twin.refresh_step([cap], 0.9, dobb.DOBB_REFRESH_ORTH_ITER, 1, grads)
    torch.cuda.synchronize()
    for name in ("W", "M", "A", "Q"):
        assert torch.equal(getattr(g, name)[0], getattr(twin, name)[0]), name


def test_callers_stream():
    """Work and allocations on a stream of the caller's while another one is current: results are the current
    stream's, and what a call returns is not given away before the current stream is done with it."""
    N, n, m = 700, 1030, 300
    x, dy, w = rand(N, n, seed=1, dtype=BF16), rand(N, n, seed=2, dtype=BF16), rand(m, n, seed=3)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()

    def both(call):
        want = call(None)
        torch.cuda.synchronize()
        got = call(s)
        s.synchronize()
        flat = lambda v: [v] if isinstance(v, torch.Tensor) else [t for u in v if u is not None and not isinstance(u, (int, str)) for t in flat(u)]  # noqa: E731
        assert len(flat(got)) == len(flat(want)) and all(torch.equal(p, q) for p, q in zip(flat(got), flat(want)))
        return want
    _, mean, rstd = both(lambda s: dobb.dobb_layer_norm(x, stream=s))
    both(lambda s: dobb.dobb_layer_norm_backward(dy, x, mean, rstd, stream=s))
    both(lambda s: dobb.dobb_layer_norm_fp8(x, rows=True, cols=True, stream=s))
    xr, xc = both(lambda s: dobb.dobb_fp8_quantize(x, cols=True, stream=s))
    wr, _ = both(lambda s: dobb.dobb_fp8_quantize(w, square=True, stream=s))
    both(lambda s: dobb.dobb_fp8_dequantize(xc, transpose=True, stream=s))
    both(lambda s: dobb.dobb_fp8_matmul(xr, wr, stream=s))
    both(lambda s: dobb.dobb_accumulate_moment_fp8(xc, torch.zeros(10, 103, 103, device=DEV), 103, stream=s))
    As = [torch.zeros(10, 103, 103, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    dobb.dobb_accumulate_moment_fp8_grouped([xc, xc], As, [103, 103], N, stream=s)
    s.synchronize()
    assert torch.equal(As[0], As[1])
