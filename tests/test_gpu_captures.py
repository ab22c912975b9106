"""Captures as the hooks of the torch.optim wrapper meet them, in both formats: gradients that a broadcast loss
gives with strides of zero, transposed inputs, micro-batches without tokens.  A capture in MXFP4 has to be, bit
for bit, that of the dense copy.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
dobb = pytest.importorskip("block_diagonal_eigenbasis_amd")
from block_diagonal_eigenbasis_amd.optimizer import Dobb, Mx4Capture  # noqa: E402

DEV = "cuda"


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def randn(*shape, seed=0):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g).to(DEV)


def linear(n, m, fmt, basis, **kw):
    lin = torch.nn.Linear(n, m, bias=False).to(DEV)
    opt = Dobb([lin.weight], blocks=2, capture_format=fmt, basis=basis, **kw)
    opt.attach_capture_hooks([lin])
    return lin, opt


def check(opt, w, want, fmt):
    (held,) = opt._captured[id(w)]
    if fmt == "native":
        assert torch.equal(held, want)
    else:
        dense = Mx4Capture.quantize(want.contiguous())
        assert torch.equal(held.codes, dense.codes) and torch.equal(held.scales, dense.scales) and held.parts == dense.parts
    opt.step()
    assert opt._group.refreshes == 1 and bool(w.isfinite().all())
    x = want.double() if fmt == "native" else dense.dequantize().double()
    nb = x.shape[1] // 2
    for b in range(2):
        xb = x[:, b * nb:(b + 1) * nb]
        # up to 200 products in fp32: 200 half steps of their magnitudes, and the result's
        tol = 201 * 2.0 ** -24 * (xb.abs().T @ xb.abs()) / x.shape[0]
        assert bool(((opt._group.A[0][b].double() - xb.T @ xb / x.shape[0]).abs() <= tol).all())


@pytest.mark.parametrize("fmt", ["native", "mx4"])
@pytest.mark.parametrize("loss", ["sum", "mean", "row"])
def test_output_gradients_of_a_broadcast_loss(fmt, loss):
    print(f"broadcast loss: {fmt} {loss}", flush=True)
    lin, opt = linear(40, 24, fmt, "output_gradient")
    x = randn(4, 50, 40, seed=1).requires_grad_()
    y = lin(x)
    if loss == "row":
        c = randn(24, seed=2)
        (y.sum((0, 1)) * c).sum().backward()
        want = c.expand(200, 24)
    else:
        getattr(y, loss)().backward()
        want = torch.full((200, 24), 1.0 if loss == "sum" else 1.0 / y.numel(), device=DEV)
    check(opt, lin.weight, want, fmt)


@pytest.mark.parametrize("fmt", ["native", "mx4"])
def test_transposed_inputs(fmt):
    print(f"transposed input: {fmt}", flush=True)
    lin, opt = linear(40, 24, fmt, "activation")
    x = randn(40, 130, seed=3)
    lin(x.t()).square().sum().backward()
    check(opt, lin.weight, x.t(), fmt)


@pytest.mark.parametrize("fmt", ["native", "mx4"])
@pytest.mark.parametrize("policy", ["first", "all"])
def test_micro_batches_without_tokens(fmt, policy):
    print(f"no tokens: {fmt} {policy}", flush=True)
    lin, opt = linear(40, 24, fmt, "activation", capture=policy)
    for k in (0, 100, 0):
        lin(randn(k, 40, seed=k)).square().sum().backward()
    check(opt, lin.weight, randn(100, 40, seed=100), fmt)
