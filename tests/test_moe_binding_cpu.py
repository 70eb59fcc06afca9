"""What the routed-experts binding makes of its arguments, without a GPU."""
from types import SimpleNamespace

import pytest
import torch

import activation_epilogue_amd as fl
from activation_epilogue_amd import moe


def test_route_options_follow_a_tensor_changed_in_place():
    """Options given as 0-dim tensors count with the value they have at the
    call, not with that of an earlier call."""
    scale, groups, renorm = torch.tensor(2.0), torch.tensor(2), torch.tensor(True)
    first = moe._route_options("softmax", groups, 1, 1, renorm, scale)._obj
    assert (first.scale, first.groups, first.raw) == (2.0, 2, 0)
    scale.fill_(3.0)
    groups.fill_(4)
    renorm.fill_(False)
    again = moe._route_options("softmax", groups, 1, 1, renorm, scale)._obj
    assert (again.scale, again.groups, again.raw) == (3.0, 4, 1)
    scale.fill_(0.0)
    with pytest.raises(ValueError, match="scale"):
        moe._route_options("softmax", groups, 1, 1, renorm, scale)


@pytest.mark.parametrize("scale", [1e-50, -1e-46, 2.0 ** -151])
def test_a_scale_that_is_zero_in_32_bits_is_refused(scale):
    """The library takes 0 for 1, so that a scale too small for a float would
    count as none at all."""
    with pytest.raises(ValueError, match="scale"):
        fl.moe_route(torch.zeros(4, 8), 2, scale=scale)
    assert moe._route_options("softmax", 1, 1, 1, True, 2.0 ** -149)._obj.scale == 2.0 ** -149


def test_a_stream_of_another_device_is_refused():
    """The call would run on the operands' device's current stream instead, in
    no order with the stream that was asked for."""
    operand = SimpleNamespace(is_cuda=True, device=torch.device("cuda", 0))
    with pytest.raises(ValueError, match="stream is on cuda:1, expected cuda:0"):
        moe._On(operand, SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0))
    assert moe._On(operand, SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=0)).index == 0
