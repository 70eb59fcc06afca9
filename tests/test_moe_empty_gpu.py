"""The routed-experts layer and operators with nothing to do: no tokens, no
choices, no columns."""
import os
import sys

import pytest
import torch

import activation_epilogue_amd as fl
from gpu_util import say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from routed_experts import RoutedExperts  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_training_step_of_no_tokens(dtype):
    say("a training step of no tokens", dtype)
    layer = RoutedExperts(64, 96, 4, 2, dtype=dtype)
    x = torch.zeros(0, 64, dtype=dtype, device="cuda")
    out, kept = layer.forward(x, keep=True)
    assert out.shape == (0, 64)
    dx, grads = layer.backward(torch.zeros_like(x), kept)
    assert dx.shape == (0, 64)
    for name, p in layer.parameters().items():
        assert grads[name].shape == p.shape and bool((grads[name] == 0).all()), name


def test_gradients_of_a_combination():
    slots = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    say("gradients of combinations of nothing")
    for T, k, S, H in ((0, 2, 0, 8), (3, 0, 4, 8), (3, 2, 0, 8), (3, 2, 6, 0)):
        rows, dout = torch.ones(S, H, device="cuda"), torch.ones(T, H, device="cuda")
        drows, dweights = fl.moe_combine_bwd(dout, rows, slots[:T, :k].contiguous())
        assert drows.shape == (S, H) and dweights.shape == (T, k) and bool((dweights == 0).all())
