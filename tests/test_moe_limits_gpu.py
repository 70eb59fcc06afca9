"""The routed-experts operators at the ends of the sizes they accept: row
numbers next to 2^31, runs that are all empty, many experts by many columns."""
import math

import pytest
import torch

import activation_epilogue_amd as fl
from gpu_util import say

pytestmark = pytest.mark.gpu
LAST = 2 ** 31 - 1


def offsets(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("N", [1, 8])
def test_bias_gradient_of_the_last_rows(N):
    """Runs that start next to row 2^31 - 1, and an empty one that starts at
    it: sums of whole numbers below 2^8, exact in every order."""
    S = LAST if N == 1 else LAST - 8
    say("bias gradient of the last rows", S, N)
    A = torch.ones(S, 0, dtype=torch.bfloat16, device="cuda")
    G = torch.empty(S, N, dtype=torch.bfloat16, device="cuda")
    G[-400:] = math.inf  # rows of nobody
    g = torch.Generator(device="cuda").manual_seed(N)
    G[-300:] = torch.randint(-8, 9, (300, N), generator=g, device="cuda").to(torch.bfloat16)
    o = offsets(S - 300, S - 295, S - 5, S - 5, S, S)
    _, dbias = fl.grouped_weight_grad(A, G, o)
    tail = G[-300:].float()
    want = torch.stack([tail[:5].sum(0), tail[5:295].sum(0), torch.zeros(N, device="cuda"), tail[295:].sum(0),
                        torch.zeros(N, device="cuda")])
    assert torch.equal(dbias, want)
