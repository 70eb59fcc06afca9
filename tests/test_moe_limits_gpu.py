"""The routed-experts operators at the ends of the sizes they accept: row
numbers next to 2^31, runs that are all empty, many experts by many columns."""
import math

import pytest
import torch

import activation_epilogue_amd as fl
from activation_epilogue_amd import moe
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


@pytest.mark.parametrize("form", ["forward", "backward", "gradient"])
def test_a_run_of_every_row_up_to_the_last(form):
    """One run of 2^31 - 1 rows: one product a row, rounded once, or one sum
    of whole numbers below 2^8, exact in every order."""
    say("a run of 2^31 - 1 rows", form)
    g = torch.Generator(device="cuda").manual_seed(1)
    A = torch.empty(LAST, 1, dtype=torch.bfloat16, device="cuda")
    if form == "gradient":
        A.zero_()
        A[:: 2 ** 24] = 1.0
        A[-3:] = -2.0
        G = torch.full((LAST, 1), 3.0, dtype=torch.bfloat16, device="cuda")
        dW, _ = fl.grouped_weight_grad(A, G, offsets(0, LAST, LAST), dbias=None)
        assert dW.flatten().tolist() == [3.0 * (128 - 6), 0.0]
        return
    A.normal_(generator=g)
    w = torch.tensor([[[1.7]], [[math.nan]]], dtype=torch.bfloat16, device="cuda")
    out = torch.full((LAST, 1), math.nan, dtype=torch.bfloat16, device="cuda")
    o = offsets(0, LAST, LAST)
    if form == "forward":
        fl.grouped_linear(A, w, o, act="none", out=out)
    else:
        fl.grouped_linear_bwd(A, w, None, o, act="none", dX=out)
    for lo in range(0, LAST, 2 ** 28):
        a, got = A[lo:lo + 2 ** 28], out[lo:lo + 2 ** 28]
        assert torch.equal(got, (a.float() * w[0, 0].float()).to(torch.bfloat16)), lo


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("indexed", [False, True])
def test_parts_of_runs_that_are_all_empty(indexed, dtype):
    """Sums in parts where every slot was dropped: nothing is written."""
    S, K, N, E = 2, 4096, 64, 3
    assert moe.grouped_workspace_bytes(S, N, K, E, dtype) > 0
    say("parts of empty runs", indexed, dtype)
    A = torch.ones(S, K, dtype=dtype, device="cuda")
    B = torch.ones(E, K, N, dtype=dtype, device="cuda")
    index = offsets(-1, -1) if indexed else None
    for first in (0, 1, S):
        out, pre = (torch.full((S, N), math.nan, dtype=dtype, device="cuda") for _ in range(2))
        fl.grouped_linear(A, B, offsets(*[first] * (E + 1)), act="relu", out=out, pre=pre, index=index)
        assert bool(torch.isnan(out).all()) and bool(torch.isnan(pre).all())


def test_bias_gradient_of_many_experts_and_columns():
    """1024 experts by 2^19 columns: 2^22 blocks of 1024 threads."""
    S, N, E = 4, 2 ** 19, 1024
    say("bias gradient of", E, "experts,", N, "columns")
    g = torch.Generator(device="cuda").manual_seed(2)
    G = torch.randint(-8, 9, (S, N), generator=g, device="cuda").to(torch.bfloat16)
    A = torch.ones(S, 0, dtype=torch.bfloat16, device="cuda")
    o = offsets(0, *[1] * (E - 1), S)
    dbias = torch.full((E, N), math.nan, device="cuda")
    fl.grouped_weight_grad(A, G, o, dbias=dbias)
    assert torch.equal(dbias[0], G[0].float()) and torch.equal(dbias[-1], G[1:].float().sum(0))
    assert bool((dbias[1:-1] == 0).all())
