"""The experts' products at seeded random sizes, runs, types, activations and
alignments, forward, indexed, backward and weight gradients, against the 64-bit
definitions; guard bands behind every output."""
import math
import random

import pytest
import torch

import activation_epilogue_amd as fl
from gpu_util import say
from moe_util import DT, grouped64, grouped_bwd64, weight_grad64, worst
from test_moe_gpu import check_rows, guarded, normal

pytestmark = pytest.mark.gpu


def size(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def shifted(t, by):
    """t on the GPU, `by` elements past a 16-byte boundary."""
    buf = torch.zeros(t.numel() + by, dtype=t.dtype, device="cuda")
    buf[by:].copy_(t.reshape(-1))
    return buf[by:].view(t.shape)


@pytest.mark.parametrize("seed", range(80))
def test_products_of_random_sizes(seed):
    rng, g = random.Random(seed), torch.Generator().manual_seed(seed)
    dtype, act = rng.choice(list(DT)), rng.choice(["none", "relu", "gelu_tanh", "glu"])
    dt, E = DT[dtype], size(rng, 1, 40)
    K, N = size(rng, 1, 3000), size(rng, 1, 900)
    most = max(1, 150_000_000 // (K * N * 12))
    counts = [0 if rng.random() < 0.3 else size(rng, 1, max(1, min(700, 2 * most // E))) for _ in range(E)]
    first, spare = rng.choice([0, 0, 3]), rng.choice([0, 1, 6])
    o = [first]
    for c in counts:
        o.append(o[-1] + c)
    S, offsets = o[-1] + spare, torch.tensor(o, dtype=torch.int32)
    by = [rng.choice([0, 0, 1, 3, 8]) for _ in range(8)]
    say("random products", seed, dtype, act, "rows", counts[:8], "first", first, "S", S, "K", K, "N", N, "shifts", by)
    A, G, D = normal(g, S, K).to(dt), normal(g, S, K).to(dt), normal(g, S, N).to(dt)
    for t in (A, G, D):  # rows of nobody
        t[:first], t[o[-1]:] = math.nan, math.inf
    B, W = normal(g, E, K, N, std=K ** -0.5).to(dt), normal(g, E, N, K, std=K ** -0.5).to(dt)
    bias, X = normal(g, E, N).to(dt), normal(g, S, N).to(dt)
    Y = normal(g, S, N).to(dt) if act == "glu" else None
    dY = None if Y is None else shifted(Y, by[0])
    do, dB = offsets.cuda(), shifted(B, by[1])
    rows = size(rng, 1, S + 1)
    index = torch.randint(-1, rows + 1, (S,), generator=g, dtype=torch.int32)
    few = normal(g, rows, K).to(dt)

    for ix, src in ((None, A), (index, few)):
        (out, ok), (pre, pok) = guarded((S, N), dt), guarded((S, N), dt)
        fl.grouped_linear(shifted(src, by[2]), dB, do, shifted(bias, by[3]), dY, act=act, out=out, pre=pre,
                          index=None if ix is None else ix.cuda())
        r, rb, p, pb = grouped64(src, ix, offsets, B, bias, Y, act)
        check_rows(out, r, rb, dt)
        check_rows(pre, p, pb, dt)
        assert ok() and pok()

    (dX, ok), (gate, gok) = guarded((S, N), dt), guarded((S, N), dt)
    fl.grouped_linear_bwd(shifted(G, by[4]), shifted(W, by[5]), None if act == "none" else X.cuda(), do, dY, act=act, dX=dX,
                          dY=gate if act == "glu" else None)
    r, rb, y, yb = grouped_bwd64(G, W, X, offsets, Y, act)
    check_rows(dX, r, rb, dt)
    if act == "glu":
        check_rows(gate, y, yb, dt)
    assert ok() and gok()

    dwt = rng.choice([dt, torch.float32])
    (dW, ok), (db, dok) = guarded((E, K, N), dwt), guarded((E, N), torch.float32)
    fl.grouped_weight_grad(shifted(A, by[6]), shifted(D, by[7]), do, dW=dW, dbias=db)
    r, rb, b, bb = weight_grad64(A, D, offsets)
    assert worst(dW.cpu(), r, rb, dwt) <= 1.0 and worst(db.cpu(), b, bb, torch.float32) <= 1.0
    assert ok() and dok()
