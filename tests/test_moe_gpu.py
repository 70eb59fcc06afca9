"""The routed-experts operators on the GPU against the 64-bit definitions of
moe_util: routing and its gradient, the plan, the movement of rows, the
experts' products, their backward epilogue and weight gradients; odd and empty
sizes, masks that leave nothing, infinities and NaN in masked places, row
numbers outside their arrays, guard bands behind every output."""
import math
import random

import pytest
import torch

import activation_epilogue_amd as fl
from gpu_util import say
from moe_util import (DT, U32, act64, grouped64, grouped_bwd64, plan64, route64, route_bwd64, scores64, unit,
                      weight_grad64, weight_rel, worst)

pytestmark = pytest.mark.gpu
GUARD = 512
DTYPES = ["f32", "f16", "bf16"]
ACTS = ["none", "relu", "gelu_tanh", "glu"]


def guarded(shape, dtype, fill=float("nan")):
    """(tensor, check): a tensor with a guard band before and behind it."""
    n = math.prod(shape)
    fill = fill if dtype.is_floating_point else -77
    buf = torch.full((n + 2 * GUARD,), fill, dtype=dtype, device="cuda")
    t = buf[GUARD:GUARD + n].view(shape)

    def intact():
        rest = torch.cat([buf[:GUARD], buf[GUARD + n:]])
        return bool((torch.isnan(rest) if dtype.is_floating_point else rest == fill).all())
    return t, intact


def normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g) * std


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


# ------------------------------------------------------------------ router

def route_logits(g, T, E, dtype, kind):
    x = normal(g, T, E, std=2.0)
    if kind == "masked":
        x[torch.rand(T, E, generator=g) < 0.4] = -math.inf
        x[0] = -math.inf                                   # nothing left
        if T > 3:
            x[1] = torch.finfo(dtype).min                  # the type's lowest value is not a mask
            x[2] = -math.inf
            x[2, E // 2] = -3.0                            # one left
            x[3, : E // 2] = math.nan                      # NaN counts as masked
    elif kind == "ties":
        x = torch.randint(-2, 3, (T, E), generator=g).float()
    elif kind == "extreme":
        x = x * 40
        if T > 2:
            x[1, E // 3] = math.inf
            x[2, :: 2] = math.inf
    return x.to(dtype)


ROUTES = [
    # T, E, k, options
    (5, 8, 2, {}),
    (33, 64, 6, dict(renorm=False)),
    (7, 1, 1, {}),
    (9, 3, 3, dict(score="sigmoid")),
    (65, 65, 7, dict(score="sigmoid", renorm=False, scale=2.5)),
    (17, 128, 8, dict(bias=True)),
    (40, 256, 8, dict(score="sigmoid", bias=True, groups=8, top_groups=4, group_top=2, scale=2.5)),
    (19, 96, 5, dict(groups=4, top_groups=2)),
    (21, 60, 4, dict(groups=6, top_groups=3, group_top=2)),
    (11, 64, 3, dict(groups=64, top_groups=2, group_top=2, bias=True)),
    (6, 1000, 64, dict(score="sigmoid", bias=True)),
    (4, 1024, 10, dict(renorm=False, bias=True)),
    (3, 500, 9, {}),
    (301, 16, 4, dict(bias=True, groups=2, top_groups=1)),
]


@pytest.mark.parametrize("kind", ["plain", "masked", "ties", "extreme"])
@pytest.mark.parametrize("case", range(len(ROUTES)))
def test_route(case, kind):
    T, E, k, o = ROUTES[case]
    o = dict(o)
    dtype = DT[DTYPES[case % 3]]
    g = torch.Generator().manual_seed(100 * case + len(kind))
    x = route_logits(g, T, E, dtype, kind)
    bias = normal(g, E, std=0.2) if o.pop("bias", False) else None
    if bias is not None and kind == "masked" and E > 4:
        bias[1], bias[3] = math.nan, -math.inf  # experts that a key of their own rules out
    say("route", T, E, k, o, kind, dtype)
    (w, wok), (e, eok) = guarded((T, k), torch.float32), guarded((T, k), torch.int32)
    fl.moe_route(x.cuda(), k, bias=None if bias is None else bias.cuda(), weights=w, experts=e, **o)
    rw, re = route64(x, k, bias=bias, **o)
    assert wok() and eok()
    assert torch.equal(e.cpu().long(), re)
    n = k if o.get("renorm", True) else E
    assert float(((w.cpu().double() - rw).abs() - weight_rel(x, n) * rw.abs()).max()) <= 2.0 ** -125

    # the gradient, for the choice made
    dw = normal(g, T, k)
    how = {n: o[n] for n in ("score", "renorm", "scale") if n in o}
    d, dok = guarded((T, E), dtype)
    fl.moe_route_bwd(x.cuda(), e.contiguous(), dw.cuda(), dlogits=d, **how)
    rd, mag = route_bwd64(x, re, dw, **how)
    assert dok()
    bound = 4 * weight_rel(x, n) * mag + 2.0 ** -120
    assert worst(d.cpu(), rd, bound, dtype) <= 1.0


def test_route_gradient_against_differences():
    """fp32 logits, the loss sum(dw * w) with the choice held: central
    differences of the 64-bit weights."""
    T, E, k = 6, 24, 4
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            g = torch.Generator().manual_seed(9)
            x, dw = normal(g, T, E), normal(g, T, k)
            w, e = fl.moe_route(x.cuda(), k, score=score, renorm=renorm)
            d = fl.moe_route_bwd(x.cuda(), e, dw.cuda(), score=score, renorm=renorm).cpu().double()

            def loss(t, row):
                s = torch.tensor(scores64(row.tolist(), score), dtype=torch.float64)[e[t].cpu().long()]
                return float((dw[t].double() * (s / s.sum() if renorm else s)).sum())
            h = 1e-4
            for t in range(T):
                for i in range(E):
                    up, down = x[t].double().clone(), x[t].double().clone()
                    up[i] += h
                    down[i] -= h
                    # the third derivative of a score is below 1, the loss has k of them: h^2 k |dw| / 6
                    assert abs((loss(t, up) - loss(t, down)) / (2 * h) - float(d[t, i])) < 1e-5


def test_route_close_keys():
    """Keys that fp32 cannot tell apart: sigmoid scores near 1 and biases that
    nearly cancel a difference of scores."""
    g = torch.Generator().manual_seed(3)
    T, E, k = 64, 128, 8
    x = 9.0 + 1e-3 * normal(g, T, E)
    bias = -1e-7 * torch.arange(E).float()
    w, e = fl.moe_route(x.cuda(), k, bias=bias.cuda(), score="sigmoid")
    assert torch.equal(e.cpu().long(), route64(x, k, bias=bias, score="sigmoid")[1])
    x = 1e-3 * normal(g, T, E)
    opt = dict(groups=8, top_groups=3, group_top=2)
    w, e = fl.moe_route(x.cuda(), k, bias=bias.cuda(), **opt)
    assert torch.equal(e.cpu().long(), route64(x, k, bias=bias, **opt)[1])


# -------------------------------------------------------------------- plan

@pytest.mark.parametrize("T,k,E,kind", [
    (1, 1, 1, "all"), (1, 2, 8, "all"), (32, 6, 64, "some"), (7, 3, 5, "none"), (1000, 2, 8, "one"),
    (1365, 3, 17, "some"), (2048, 2, 4, "all"), (2049, 2, 4, "wild"), (5000, 8, 256, "some"), (3000, 4, 1024, "wild"),
    (16384, 1, 1000, "one"), (0, 3, 6, "all"), (5, 0, 6, "all")])
def test_plan(T, k, E, kind):
    g = torch.Generator().manual_seed(T + k + E)
    e = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    if kind == "some":
        e[torch.rand(T, k, generator=g) < 0.3] = -1
    elif kind == "none":
        e[:] = -1
    elif kind == "one":
        e[:] = E // 2
    elif kind == "wild":  # values that are no expert
        bad = torch.tensor([-1, -5, E, E + 9, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
        pick = torch.rand(T, k, generator=g) < 0.2
        e[pick] = bad[torch.randint(0, 6, (int(pick.sum()),), generator=g)]
    say("plan", T, k, E, kind)
    (o, ook), (tr, tok), (rs, rok) = (guarded((E + 1,), torch.int32), guarded((T * k,), torch.int32),
                                      guarded((T, k), torch.int32))
    fl.moe_plan(e.cuda(), E, out=(o, tr, rs))
    ro, rt, rr = plan64(e, E)
    assert torch.equal(o.cpu(), ro) and torch.equal(tr.cpu(), rt) and torch.equal(rs.cpu(), rr)
    assert ook() and tok() and rok()


# ---------------------------------------------------------------- movement

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,S,H,shift", [(1, 1, 1, 1, 0), (5, 3, 15, 64, 0), (33, 6, 198, 257, 0), (64, 2, 128, 2048, 0),
                                           (40, 8, 100, 1000, 0), (9, 2, 18, 128, 1), (3, 64, 192, 24, 0),
                                           (130, 1, 130, 4096, 0)])
def test_movement(T, k, S, H, shift, dtype):
    """Gather, combine and their gradients; some slots without a row, some row
    numbers outside the arrays; `shift` moves every operand one element off a
    16-byte boundary."""
    dt = DT[dtype]
    g = torch.Generator().manual_seed(T * 7 + H)

    def dev(t):
        buf = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
        buf[shift:].copy_(t.reshape(-1))
        return buf[shift:].view(t.shape)
    slot = torch.randperm(max(S, T * k), generator=g)[: T * k].to(torch.int32).view(T, k)
    slot[slot >= S] = -1
    wild = slot.clone()
    wild[torch.rand(T, k, generator=g) < 0.1] = S + 5
    if T > 2:
        wild[1] = -7  # a token without rows
    index = torch.randint(0, T, (S,), generator=g, dtype=torch.int32)
    index[torch.rand(S, generator=g) < 0.1] = -1
    if S > 3:
        index[2] = T
    X, rows, R, dout = (normal(g, *s).to(dt) for s in ((T, H), (S, H), (T, H), (T, H)))
    weights = torch.rand(T, k, generator=g)
    weights[wild < 0] = math.nan  # never used
    say("movement", T, k, S, H, shift, dtype)

    got, ok = guarded((S, H), dt)
    fl.moe_gather(dev(X), index.cuda(), rows=got)
    inside = (index >= 0) & (index < T)
    ref = torch.where(inside[:, None], X[index.clamp(0, T - 1).long()], torch.zeros((), dtype=dt))
    assert torch.equal(got.cpu(), ref) and ok()

    used = (wild >= 0) & (wild < S)
    picked = rows.double()[wild.clamp(0, S - 1).long()] * used[..., None]
    for w, res in ((weights, R), (weights, None), (None, None), (None, R)):
        got, ok = guarded((T, H), dt)
        fl.moe_combine(dev(rows), wild.cuda(), None if w is None else w.cuda(), R=None if res is None else dev(res), out=got)
        terms = picked if w is None else picked * torch.where(used, w, torch.zeros(()))[..., None].double()
        ref = terms.sum(1) + (res.double() if res is not None else 0.0)
        bound = (k + 1) * U32 * (terms.abs().sum(1) + (res.double().abs() if res is not None else 0.0))
        assert worst(got.cpu(), ref, bound, dt) <= 1.0 and ok()
    same = dev(R)
    fl.moe_combine(dev(rows), wild.cuda(), weights.cuda(), R=same, out=same)
    terms = picked * torch.where(used, weights, torch.zeros(()))[..., None].double()
    assert worst(same.cpu(), terms.sum(1) + R.double(), (k + 1) * U32 * (terms.abs().sum(1) + R.double().abs()), dt) <= 1.0

    for w in (weights, None):
        (dr, drok), (dw, dwok) = guarded((S, H), dt), guarded((T, k), torch.float32)
        fl.moe_combine_bwd(dev(dout), dev(rows), wild.cuda(), None if w is None else w.cuda(), drows=dr, dweights=dw)
        d = dout.double()
        ref = (picked * d[:, None, :]).sum(2)
        bound = H * U32 * (picked.abs() * d.abs()[:, None, :]).sum(2)
        assert worst(dw.cpu(), ref, bound, torch.float32) <= 1.0 and dwok() and drok()
        want = torch.full((S, H), math.nan, dtype=torch.float64)
        for t in range(T):
            for j in range(k):
                if used[t, j]:
                    want[wild[t, j]] = d[t] if w is None else d[t] * float(w[t, j])
        left = torch.isnan(want[:, 0])
        assert bool(torch.isnan(dr.cpu()[left]).all())
        if bool((~left).any()):
            assert worst(dr.cpu()[~left], want[~left], U32 * want[~left].abs(), dt) <= 1.0
    # in place, and each gradient alone
    inplace = dev(rows)
    dw2 = torch.empty(T, k, device="cuda")
    fl.moe_combine_bwd(dev(dout), inplace, wild.cuda(), None, drows=inplace, dweights=dw2)
    assert torch.equal(dw2, dw) and torch.equal(inplace.cpu()[~left], dr.cpu()[~left])
    assert torch.equal(inplace.cpu()[left], rows[left])


# ------------------------------------------------------- experts' products

def offsets_of(counts):
    return torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32)


# rows of every expert (empty runs first, last and between), K, N, rows left over past the last run
PRODUCTS = [
    ([1], 8, 8, 0),
    ([0, 3, 0, 0, 2, 0], 64, 64, 0),
    ([1, 1, 1, 1, 0, 1], 256, 128, 3),
    ([17, 0, 31, 33], 96, 200, 1),
    ([5, 64, 65, 0, 130], 72, 130, 2),
    ([300, 257, 0, 3], 130, 264, 0),
    ([40, 1, 90], 31, 33, 5),
    ([3, 9], 1, 1, 0),
    ([7, 2], 5, 3, 1),
    ([12, 20], 0, 16, 0),
    ([513, 0, 260], 640, 520, 0),
    ([2] * 70, 40, 24, 0),
]


def product(case, dtype, act, seed=0):
    counts, K, N, spare = PRODUCTS[case]
    g = torch.Generator().manual_seed(1000 * case + seed)
    dt = DT[dtype]
    E, S = len(counts), sum(counts) + spare
    std = max(K, 1) ** -0.5
    B = normal(g, E, K, N, std=std).to(dt)
    bias = normal(g, E, N).to(dt)
    Y = normal(g, S, N).to(dt) if act == "glu" else None
    return g, dt, E, S, K, N, offsets_of(counts), B, bias, Y


def check_rows(got, ref, bound, dt):
    """got against ref where ref is a number; NaN (untouched) elsewhere."""
    got, live = got.cpu(), ~torch.isnan(ref)
    if got.numel() == 0:
        return
    assert bool(torch.isnan(got[~live]).all()), "a row outside every run was written"
    assert worst(got[live], ref[live], bound[live], dt) <= 1.0


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(PRODUCTS)))
def test_grouped_linear(case, dtype, act):
    g, dt, E, S, K, N, offsets, B, bias, Y = product(case, dtype, act)
    A = normal(g, S, K).to(dt)
    A[int(offsets[-1]):] = math.nan  # rows of nobody
    say("grouped_linear", PRODUCTS[case][:1], K, N, dtype, act)
    dA, dB, db, dY, do = cuda(A, B, bias, Y, offsets)
    for b, pre in ((bias, True), (None, False)):
        (out, ok), (x, xok) = guarded((S, N), dt), guarded((S, N), dt)
        fl.grouped_linear(dA, dB, do, None if b is None else db, dY, act=act, out=out, pre=x if pre else None)
        r, rb, p, pb = grouped64(A, None, offsets, B, b, Y, act)
        check_rows(out, r, rb, dt)
        if pre:
            check_rows(x, p, pb, dt)
        assert ok() and xok()
    if act == "glu":  # out in the gate operand's place
        fl.grouped_linear(dA, dB, do, None, dY, act=act, out=dY)
        live = int(offsets[-1])
        assert torch.equal(dY[:live].view(torch.uint8), out[:live].view(torch.uint8))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(PRODUCTS)))
def test_grouped_linear_indexed(case, dtype):
    g, dt, E, S, K, N, offsets, B, bias, _ = product(case, dtype, "relu", seed=1)
    T = max(1, S // 3)
    A = normal(g, T, K).to(dt)
    index = torch.randint(0, T, (S,), generator=g, dtype=torch.int32)
    if S > 4:  # row numbers outside A read zeros
        index[0], index[1], index[S // 2], index[-1] = T, -1, 2 ** 31 - 1, -2 ** 31
    say("grouped_linear indexed", PRODUCTS[case][:1], K, N, dtype)
    out, ok = guarded((S, N), dt)
    fl.grouped_linear(A.cuda(), B.cuda(), offsets.cuda(), bias.cuda(), act="relu", out=out, index=index.cuda())
    r, rb, _, _ = grouped64(A, index, offsets, B, bias, None, "relu")
    check_rows(out, r, rb, dt)
    assert ok()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(PRODUCTS)))
def test_grouped_linear_bwd(case, dtype, act):
    g, dt, E, S, K, N, offsets, B, bias, Y = product(case, dtype, act, seed=2)
    W = normal(g, E, N, K, std=max(N, 1) ** -0.5).to(dt)
    G, X = normal(g, S, K).to(dt), normal(g, S, N).to(dt)
    G[int(offsets[-1]):] = math.nan
    X[: S // 3, : N // 2] = 0.0  # the corner of relu
    say("grouped_linear_bwd", PRODUCTS[case][:1], K, N, dtype, act)
    dG, dW, dXs, dY, do = cuda(G, W, X, Y, offsets)
    (out, ok), (out2, ok2) = guarded((S, N), dt), guarded((S, N), dt)
    fl.grouped_linear_bwd(dG, dW, None if act == "none" else dXs, do, dY, act=act, dX=out,
                          dY=out2 if act == "glu" else None)
    r, rb, y, yb = grouped_bwd64(G, W, X, offsets, Y, act)
    check_rows(out, r, rb, dt)
    if act == "glu":
        check_rows(out2, y, yb, dt)
    assert ok() and ok2()
    if act != "none":  # in place of X, and of Y
        fl.grouped_linear_bwd(dG, dW, dXs, do, dY, act=act, dX=dXs, dY=dY)
        live = int(offsets[-1])
        assert torch.equal(dXs[:live].view(torch.uint8), out[:live].view(torch.uint8))
        assert act != "glu" or torch.equal(dY[:live].view(torch.uint8), out2[:live].view(torch.uint8))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(PRODUCTS)))
def test_grouped_weight_grad(case, dtype):
    g, dt, E, S, K, N, offsets, _, _, _ = product(case, dtype, "relu", seed=3)
    A, G = normal(g, S, K).to(dt), normal(g, S, N).to(dt)
    A[int(offsets[-1]):] = math.nan
    G[int(offsets[-1]):] = math.inf
    say("grouped_weight_grad", PRODUCTS[case][:1], K, N, dtype)
    r, rb, d, db = weight_grad64(A, G, offsets)
    for dwt in {dt, torch.float32}:
        (dW, ok), (bias, bok) = guarded((E, K, N), dwt), guarded((E, N), torch.float32)
        fl.grouped_weight_grad(A.cuda(), G.cuda(), offsets.cuda(), dW=dW, dbias=bias)
        assert worst(dW.cpu(), r, rb, dwt) <= 1.0 and worst(bias.cpu(), d, db, torch.float32) <= 1.0
        assert ok() and bok()
    again, none = fl.grouped_weight_grad(A.cuda(), G.cuda(), offsets.cuda(), dbias=None, dw_dtype=torch.float32)
    assert none is None and worst(again.cpu(), r, rb, torch.float32) <= 1.0


def test_neighbours_do_not_leak():
    """NaN and infinities in the rows, weights and biases of one expert reach
    that expert's rows only, at sizes where tiles and chunks straddle them."""
    for dtype in DTYPES:
        for case in (4, 6, 8):
            g, dt, E, S, K, N, offsets, B, bias, _ = product(case, dtype, "none", seed=5)
            A = normal(g, S, K).to(dt)
            lo, hi = int(offsets[1]), int(offsets[2])
            A[lo:hi] = math.nan
            B[1] = math.inf
            bias[1] = math.nan
            out = torch.zeros(S, N, dtype=dt, device="cuda")
            fl.grouped_linear(A.cuda(), B.cuda(), offsets.cuda(), bias.cuda(), act="none", out=out)
            r, rb, _, _ = grouped64(A, None, offsets, B, bias, None, "none")
            keep = torch.ones(S, dtype=torch.bool)
            keep[lo:hi] = False
            keep[int(offsets[-1]):] = False
            assert worst(out.cpu()[keep], r[keep], rb[keep], dt) <= 1.0, (dtype, case)
            assert bool(torch.isnan(out[lo:hi]).all())
            dW, db = fl.grouped_weight_grad(A.cuda(), torch.ones(S, N, dtype=dt, device="cuda"), offsets.cuda())
            keep = [e for e in range(E) if e != 1]
            rw, rwb, _, _ = weight_grad64(A, torch.ones(S, N, dtype=dt), offsets)
            assert worst(dW.cpu()[keep], rw[keep], rwb[keep], dt) <= 1.0, (dtype, case)


def test_wild_offsets_stay_inside():
    """Offsets outside [0,S], falling or repeated: limited before any access;
    runs that are sane still compute."""
    S, K, N = 100, 64, 48
    for dtype in DTYPES:
        dt = DT[dtype]
        g = torch.Generator().manual_seed(8)
        A, B = normal(g, S, K).to(dt), normal(g, 5, K, N, std=0.1).to(dt)
        offsets = torch.tensor([-50, 20, 60, 10, 2 ** 31 - 1, -9], dtype=torch.int32)
        limited = [(0, 0, 20), (1, 20, 60), (3, 10, 100)]  # clamped; run 2 and 4 fall, so they are empty
        out, ok = guarded((S, N), dt)
        fl.grouped_linear(A.cuda(), B.cuda(), offsets.cuda(), act="none", out=out)
        assert ok()
        got = out.cpu().double()
        for e, lo, hi in limited[:1]:
            ref = A[lo:hi].double() @ B[e].double()
            # run 3 overlaps rows 10 .. 100: only the rows below are one run's alone
            assert worst(got[:10], ref[:10], K * U32 * (A[:10].double().abs() @ B[e].double().abs()), dt) <= 1.0
        dX, ok = guarded((S, K), dt)
        fl.grouped_linear_bwd(torch.zeros(S, N, dtype=dt, device="cuda"), B.cuda(), None, offsets.cuda(), act="none", dX=dX)
        dW, ok2 = guarded((5, K, N), dt)
        fl.grouped_weight_grad(A.cuda(), torch.zeros(S, N, dtype=dt, device="cuda"), offsets.cuda(), dW=dW)
        assert ok() and ok2() and bool((dW == 0).all())


def test_gradients_against_differences():
    """dX, dW and dbias of a small fp32 layer against central differences of
    its 64-bit loss."""
    g = torch.Generator().manual_seed(4)
    offsets = offsets_of([3, 0, 4])
    E, K, N, S = 3, 5, 6, 7
    A, B, bias = normal(g, S, K), normal(g, E, K, N, std=0.5), normal(g, E, N)
    D = normal(g, S, N)
    for act in ("gelu_tanh", "glu"):
        Y = normal(g, S, N) if act == "glu" else None
        _, pre = fl.grouped_linear(*cuda(A, B, offsets, bias, Y), act=act, pre=True)
        # the loss sum(D * out): an identity as the next product makes D the gradient at out
        eye = torch.eye(N).expand(E, N, N).contiguous()
        dX, dY = fl.grouped_linear_bwd(D.cuda(), eye.cuda(), pre, offsets.cuda(), None if Y is None else Y.cuda(), act=act)
        dW, db = fl.grouped_weight_grad(A.cuda(), dX, offsets.cuda())
        dA, _ = fl.grouped_linear_bwd(dX, B.cuda(), None, offsets.cuda(), act="none")

        def loss(A, B, bias, Y):
            total = 0.0
            for e in range(E):
                lo, hi = int(offsets[e]), int(offsets[e + 1])
                x = A[lo:hi] @ B[e] + bias[e]
                total += float((D[lo:hi].double() * act64(x, None if Y is None else Y[lo:hi], act)).sum())
            return total
        args = [A.double(), B.double(), bias.double(), None if Y is None else Y.double()]
        for i, grad in enumerate((dA, dW, db, dY)):
            if grad is None:
                continue
            flat = args[i].view(-1)
            for p in range(flat.numel()):
                keep, h = float(flat[p]), 1e-4
                flat[p] = keep + h
                up = loss(*args)
                flat[p] = keep - h
                down = loss(*args)
                flat[p] = keep
                # differences: h^2 times a third derivative of order 10, and fp32 gradients of order 10
                assert abs((up - down) / (2 * h) - float(grad.reshape(-1)[p])) < 2e-5, (act, i, p)
