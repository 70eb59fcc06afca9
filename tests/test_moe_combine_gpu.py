"""Each gradient of a combination by itself."""
import pytest
import torch

import activation_epilogue_amd as fl
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,k,H", [(5, 3, 64), (40, 2, 257), (3000, 2, 128)])
def test_one_gradient_of_a_combination(T, k, H, dtype):
    """The bits of the call that computes both; rows are not read for drows
    alone (they are NaN, and the weights' gradient untouched)."""
    g = torch.Generator(device="cuda").manual_seed(H)
    rows, dout = (torch.randn(n, H, generator=g, device="cuda").to(dtype) for n in (T * k, T))
    slot = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k)
    w = torch.rand(T, k, generator=g, device="cuda")
    say("one gradient of a combination", T, k, H, dtype)
    drows, dweights = fl.moe_combine_bwd(dout, rows, slot, w)
    only, none = fl.moe_combine_bwd(dout, torch.full_like(rows, float("nan")), slot, w, dweights=False)
    assert none is None and torch.equal(only, drows)
    none, only = fl.moe_combine_bwd(dout, rows, slot, w, drows=False)
    assert none is None and torch.equal(only, dweights)
    with pytest.raises(fl.FusedLinearError, match="both NULL"):
        fl.moe_combine_bwd(dout, rows, slot, w, drows=False, dweights=False)
