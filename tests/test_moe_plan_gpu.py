"""Plans of many slots: counts of hundreds to half a million blocks."""
import pytest
import torch

import activation_epilogue_amd as fl
from gpu_util import say

pytestmark = pytest.mark.gpu


def check_plan(e, E, plan, k):
    """offsets are the counts' sums; the rows of an expert hold its slots in
    their order; slots without an expert have no row (in pieces of 2^27)."""
    flat, rows, tokens = e.reshape(-1), plan.row_of_slot.reshape(-1), plan.token_of_row
    S, step = flat.numel(), 2 ** 27
    counts = torch.zeros(E + 1, dtype=torch.long, device="cuda")
    for lo in range(0, S, step):
        f = flat[lo:lo + step]
        f = torch.where((f >= 0) & (f < E), f, torch.full_like(f, E)).long()
        if E <= 8:
            counts += torch.stack([(f == i).sum() for i in range(E + 1)])
        else:
            counts += torch.bincount(f, minlength=E + 1)
    first = torch.cat([counts.new_zeros(1), counts[:E].cumsum(0)])
    assert torch.equal(plan.offsets.long(), first)
    n = int(first[-1])
    assert bool((tokens[n:] == -1).all())
    last = torch.full((E + 1,), -1, dtype=torch.long, device="cuda")  # the last row given to an expert so far
    for lo in range(0, S, step):
        f, r = flat[lo:lo + step], rows[lo:lo + step]
        live = (f >= 0) & (f < E)
        assert bool((r[~live] == -1).all())
        at = r[live].long()
        slot = (lo + torch.arange(f.numel(), device="cuda"))[live]
        assert int(at.min()) >= 0 and int(at.max()) < n
        assert torch.equal(tokens[at].long(), slot // k)
        for i in range(E) if E <= 8 else (0, 1, E // 2, E - 1):
            mine = r[f == i].long()  # this expert's rows, in the order of the slots: each the next
            if mine.numel():
                start = int(last[i]) + 1 if int(last[i]) >= 0 else int(first[i])
                assert torch.equal(mine, start + torch.arange(mine.numel(), device="cuda"))
                last[i] = mine[-1]


@pytest.mark.parametrize("T,k,E", [
    (4096 * 256, 1, 8), (4096 * 256 + 1, 1, 8), (4096 * 512, 1, 8), (4096 * 512 + 1, 1, 8), (1_048_577, 2, 3), (700_001, 7, 256), (600_000, 5, 1024),
    (3_000_000, 1, 65), (9_000_001, 2, 1), (2_500_000, 8, 200)])
def test_plan_of_many_blocks(T, k, E):
    g = torch.Generator(device="cuda").manual_seed(E)
    e = torch.randint(-1, E + 1, (T, k), generator=g, device="cuda", dtype=torch.int32)
    say("plan of many blocks", T, k, E)
    # (the workspace as it comes: nothing in it is taken for zero)
    need = fl.moe_plan_workspace_bytes(T, k, E)
    ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    plan = fl.moe_plan(e, E, workspace=ws[:need])
    check_plan(e, E, plan, k)
    assert bool((ws[need:] == 0x5A).all())


def test_plan_of_as_many_slots_as_it_takes():
    """2^31 - 1 slots, in 524288 blocks."""
    S, E = 2 ** 31 - 1, 5
    g = torch.Generator(device="cuda").manual_seed(7)
    e = torch.empty(S, 1, dtype=torch.int32, device="cuda")
    for lo in range(0, S, 2 ** 28):
        e[lo:lo + 2 ** 28].random_(-1, E, generator=g)
    say("plan of", S, "slots")
    check_plan(e, E, fl.moe_plan(e, E), 1)
