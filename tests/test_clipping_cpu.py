"""Clipping as the optimizer layer offers it, without a GPU."""
import pytest
import torch

import block_diagonal_eigenbasis_amd as dobb
from block_diagonal_eigenbasis_amd import _ops
from block_diagonal_eigenbasis_amd.optimizer import DobbGroup, clip_grad_norm_


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_the_norm_of_no_gradients_is_on_the_parameters_device(device):
    a, b = (torch.nn.Parameter(torch.zeros(3, 4, device=device, dtype=torch.bfloat16)) for _ in range(2))
    for given in (a, [a, b], iter((a, b))):
        total = clip_grad_norm_(given, 1.0)
        assert total.device.type == device and total.shape == () and total.dtype == torch.float32
    assert float(clip_grad_norm_([], 1.0)) == 0.0


@pytest.mark.parametrize("bad", ["shape", "strides", "dtype", "capture", "capture's dtype"])
def test_a_step_that_is_refused_has_clipped_nothing(monkeypatch, bad):
    """Gradients are clipped in place, so everything that a call refuses is refused before."""
    clipped = []
    monkeypatch.setattr(_ops, "dobb_clip_grad_norm_grouped", lambda Gs, *a, **k: clipped.append(Gs))
    g = DobbGroup([torch.zeros(8, 16), torch.zeros(4, 32)], [8, 16])
    grads = [torch.ones(8, 16), torch.ones(4, 32)]
    xs = [torch.ones(5, 16), torch.ones(5, 32)]
    error = ValueError
    if bad == "shape":
        grads[1] = torch.ones(32, 4)
    elif bad == "strides":
        grads[1] = torch.ones(32, 4).T
    elif bad == "dtype":
        grads[1], error = grads[1].double(), TypeError
    elif bad == "capture":
        xs[1] = torch.ones(5, 33)
    else:
        xs[1], error = xs[1].double(), TypeError
    if not bad.startswith("capture"):
        with pytest.raises(error):
            g.step(grads, max_grad_norm=1.0)
    with pytest.raises(error):
        g.refresh_step(xs, 0.9, dobb.DOBB_REFRESH_ORTH_ITER, 1, grads, max_grad_norm=1.0)
    assert not clipped
