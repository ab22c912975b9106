"""Clipping as the optimizer layer offers it, without a GPU."""
import pytest
import torch

from block_diagonal_eigenbasis_amd.optimizer import clip_grad_norm_


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_the_norm_of_no_gradients_is_on_the_parameters_device(device):
    a, b = (torch.nn.Parameter(torch.zeros(3, 4, device=device, dtype=torch.bfloat16)) for _ in range(2))
    for given in (a, [a, b], iter((a, b))):
        total = clip_grad_norm_(given, 1.0)
        assert total.device.type == device and total.shape == () and total.dtype == torch.float32
    assert float(clip_grad_norm_([], 1.0)) == 0.0
