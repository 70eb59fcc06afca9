"""The routed-experts operators together (examples/routed_experts.py) against
64-bit autograd, in a graph, on streams; sums in parts; tiles at sizes where a
workgroup takes several of them; arrays beyond 2^31 elements."""
import math
import os
import sys

import pytest
import torch

import activation_epilogue_amd as fl
from activation_epilogue_amd import moe
from gpu_util import say
from moe_util import U32, act64, act_bound, act_grad64, act_grad_bound, unit

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from routed_experts import RoutedExperts, every_row  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def offsets_of(counts):
    return torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32, device="cuda")


def normal(g, *shape, std=1.0, dt=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def check(got, ref, bound, dt):
    """One rounding to dt of a value off by at most `bound`."""
    u = unit(dt)
    allow = bound * (1 + u) + u * ref.abs() + (2.0 ** -25 if dt == torch.float16 else 2.0 ** -134)
    off = (got.double() - ref).abs()
    assert bool(torch.isfinite(got).all())
    assert bool((off <= allow).all()), float((off / allow).max())


# --------------------------------------------------------- the products

def forward64(A, index, offsets, B, bias, Y, act):
    """(out, bound, pre, bound) of every run's rows, in 64 bits on the GPU."""
    o = offsets.tolist()
    rows = A if index is None else A[index.long()]
    res = [[], [], [], []]
    for e in range(len(o) - 1):
        a, b, c = rows[o[e]:o[e + 1]].double(), B[e].double(), bias[e].double()
        x = a @ b + c
        ex = (B.shape[1] + 20) * U32 * (a.abs() @ b.abs() + c.abs())
        y = Y[o[e]:o[e + 1]].double() if Y is not None else torch.zeros_like(x)
        for r, v in zip(res, (act64(x, y, act), act_bound(x, y, act, ex), x, ex)):
            r.append(v)
    return [torch.cat(r) for r in res]


# counts, K, N: workgroups with several tiles, tiles with idle waves (half of their rows or columns missing), runs
# that end inside a tile, K and N that end inside a stage or chunk
LARGE = [
    ([1100, 0, 700, 1, 385], 200, 1290),
    ([600] * 8, 130, 1408),
    ([129, 130, 0, 127, 260, 385, 3, 500], 777, 1033),
    ([2500], 64, 3333),
    ([4] * 64, 512, 1408),
    ([30, 64, 65, 0, 17, 1] * 11, 201, 1403),
    ([16] * 32 + [70, 0], 328, 3000),
    ([2300, 2200, 0, 2500], 1291, 4001),
]


@pytest.mark.parametrize("act", ["gelu_tanh", "glu"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", range(len(LARGE)))
def test_large_runs(case, dtype, act):
    counts, K, N = LARGE[case]
    dt, g, offsets = DT[dtype], gen(case), offsets_of(LARGE[case][0])
    E, S = len(counts), sum(counts)
    A, B, bias = normal(g, S, K, dt=dt), normal(g, E, K, N, std=K ** -0.5, dt=dt), normal(g, E, N, dt=dt)
    Y = normal(g, S, N, dt=dt) if act == "glu" else None
    say("large runs", counts[:8], K, N, dtype, act)
    index = torch.randperm(S, generator=g, device="cuda").to(torch.int32)
    for ix in (None, index):
        out, pre = fl.grouped_linear(A, B, offsets, bias, Y, act=act, index=ix, pre=True)
        r, rb, x, xb = forward64(A, ix, offsets, B, bias, Y, act)
        check(out, r, rb, dt)
        check(pre, x, xb, dt)
    G, W, X = normal(g, S, K, dt=dt), normal(g, E, N, K, std=N ** -0.5, dt=dt), normal(g, S, N, dt=dt)
    dX, dY = fl.grouped_linear_bwd(G, W, X, offsets, Y, act=act)
    D = normal(g, S, N, dt=dt)
    dW, db = fl.grouped_weight_grad(A, D, offsets)
    o = offsets.tolist()
    for e in range(E):
        s = slice(o[e], o[e + 1])
        gd, w = G[s].double(), W[e].double().t().contiguous()
        d, ed = gd @ w, K * U32 * (gd.abs() @ w.abs())
        x, y = X[s].double(), Y[s].double() if Y is not None else torch.zeros_like(d)
        slope, es = act_grad64(x, y, act), act_grad_bound(x, y, act)
        check(dX[s], d * slope, ed * (slope.abs() + es) + d.abs() * es + U32 * (d * slope).abs(), dt)
        if act == "glu":
            check(dY[s], d * x, ed * x.abs() + U32 * (d * x).abs(), dt)
        a, dd = A[s].double(), D[s].double()
        n = counts[e] + 20
        check(dW[e], a.t().contiguous() @ dd, n * U32 * (a.abs().t().contiguous() @ dd.abs()), dt)
        check(db[e], dd.sum(0), n * U32 * dd.abs().sum(0), torch.float32)


# counts, K, N of few tiles and long sums: the parts of K
PARTS = [([1, 0, 1], 4096, 256), ([3], 4096, 64), ([0, 2, 5, 1], 2111, 131), ([1], 5000, 1)]


@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh", "glu"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", range(len(PARTS)))
def test_parts_forward(case, dtype, act):
    counts, K, N = PARTS[case]
    dt, g, offsets = DT[dtype], gen(50 + case), offsets_of(counts)
    E, S = len(counts), sum(counts)
    need = moe.grouped_workspace_bytes(S + 2, N, K, E, dt)
    assert need > 0 and need % ((S + 2) * N * 4) == 0
    A, B, bias = normal(g, S + 2, K, dt=dt), normal(g, E, K, N, std=K ** -0.5, dt=dt), normal(g, E, N, dt=dt)
    Y = normal(g, S + 2, N, dt=dt) if act == "glu" else None
    A[S:] = math.nan  # rows of nobody
    say("parts forward", counts, K, N, dtype, act)
    ws = torch.full((need // 4 + 64,), math.nan, device="cuda")
    out, pre = (torch.full((S + 2, N), math.nan, dtype=dt, device="cuda") for _ in range(2))
    fl.grouped_linear(A, B, offsets, bias, Y, act=act, out=out, pre=pre, workspace=ws[:need // 4])
    r, rb, x, xb = forward64(A, None, offsets, B, bias, Y, act)
    check(out[:S], r, rb, dt)
    check(pre[:S], x, xb, dt)
    assert bool(torch.isnan(out[S:]).all()) and bool(torch.isnan(pre[S:]).all()) and bool(torch.isnan(ws[need // 4:]).all())
    again = torch.empty_like(out)
    fl.grouped_linear(A, B, offsets, bias, Y, act=act, out=again)
    assert torch.equal(again[:S].view(torch.uint8), out[:S].view(torch.uint8))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("counts,K,N", [([5000, 0, 3000], 100, 100), ([4097], 70, 33), ([1, 8000], 256, 130)])
def test_parts_weight_grad(counts, K, N, dtype):
    dt, g, offsets = DT[dtype], gen(70), offsets_of(counts)
    E, S = len(counts), sum(counts)
    need = moe.grouped_grad_workspace_bytes(S + 3, N, K, E, dt)
    assert need > 0 and need % (E * K * N * 4) == 0
    A, D = normal(g, S + 3, K, dt=dt), normal(g, S + 3, N, dt=dt)
    A[S:], D[S:] = math.nan, math.inf
    say("parts weight_grad", counts, K, N, dtype)
    ws = torch.full((need // 4 + 64,), math.nan, device="cuda")
    for dwt in {dt, torch.float32}:
        dW, db = fl.grouped_weight_grad(A, D, offsets, dw_dtype=dwt, workspace=ws[:need // 4])
        assert bool(torch.isnan(ws[need // 4:]).all())
        whole = torch.empty_like(dW)
        moe._ok(moe._lib().fl_grouped_weight_grad(A.data_ptr(), D.data_ptr(), offsets.data_ptr(), whole.data_ptr(), None,
                                                  S + 3, N, K, E, fl._dtype_code(dt), fl._dtype_code(dwt),
                                                  torch.cuda.current_stream().cuda_stream))
        o = offsets.tolist()
        for e in range(E):
            a, d = A[o[e]:o[e + 1]].double(), D[o[e]:o[e + 1]].double()
            bound = (counts[e] + 20) * U32 * (a.abs().t().contiguous() @ d.abs())
            check(dW[e], a.t().contiguous() @ d, bound, dwt)
            check(whole[e], a.t().contiguous() @ d, bound, dwt)
            check(db[e], d.sum(0), (counts[e] + 20) * U32 * d.abs().sum(0), torch.float32)


def test_same_bits_every_time():
    g = gen(5)
    offsets = offsets_of([300, 20, 0, 700])
    A, B, D = normal(g, 1020, 1000, dt=torch.bfloat16), normal(g, 4, 1000, 520, dt=torch.bfloat16), normal(g, 1020, 520, dt=torch.bfloat16)
    first = [fl.grouped_linear(A, B, offsets, act="none"), *fl.grouped_weight_grad(A, D, offsets)]
    for _ in range(5):
        for a, b in zip(first, [fl.grouped_linear(A, B, offsets, act="none"), *fl.grouped_weight_grad(A, D, offsets)]):
            assert torch.equal(a, b)


# ------------------------------------------------------------- the layer

def layer64(layer, x, experts):
    """The layer by its definition on 64-bit leaves, the choice of experts given."""
    p = {n: v.double().cpu().requires_grad_() for n, v in layer.parameters().items()}
    x = x.double().cpu().requires_grad_()
    logits = x @ p["Wr"]
    s = torch.softmax(logits, 1) if layer.weighting["score"] == "softmax" else torch.sigmoid(logits)
    s = s.gather(1, experts.cpu().long())
    w = layer.weighting["scale"] * (s / s.sum(1, keepdim=True) if layer.weighting["renorm"] else s)
    rows = []
    for t in range(x.shape[0]):
        row = x[t]
        for j in range(layer.k):
            e = int(experts[t, j])
            h = x[t] @ p["W1"][e] + p["b1"][e]
            h = 0.5 * h * (1 + torch.tanh(math.sqrt(2 / math.pi) * (h + 0.044715 * h ** 3)))
            row = row + w[t, j] * (h @ p["W2"][e] + p["b2"][e])
        rows.append(row)
    return torch.stack(rows), x, p


@pytest.mark.parametrize("options", [{}, {"score": "sigmoid", "scale": 2.5, "groups": 2, "top_groups": 1},
                                     {"renorm": False}])
def test_layer_against_autograd(options):
    """fp32, where the layer's own rounding stays below 1e-4 of the largest
    entry: sums of at most 96 terms through four products in a row."""
    layer = RoutedExperts(48, 96, 6, 2, dtype=torch.float32, seed=3, **options)
    x = normal(gen(4), 37, 48)
    out, kept = layer.forward(x, keep=True)
    ref, leaf, params = layer64(layer, x, kept[3])
    dout = normal(gen(6), 37, 48)
    (ref * dout.double().cpu()).sum().backward()
    dx, grads = layer.backward(dout, kept)
    say("layer", options)

    def near(got, want):
        assert float((got.double().cpu() - want).abs().max()) <= 1e-4 * float(want.abs().max())
    near(out, ref.detach())
    near(dx, leaf.grad)
    for name, g in grads.items():
        near(g, params[name].grad)
    # one token at a time, and without what backward needs
    assert float((torch.cat([layer.forward(x[t:t + 1].contiguous()) for t in range(37)]) - out).abs().max()) <= 1e-4
    assert torch.equal(layer.forward(x), out)


def test_layer_in_a_graph():
    """Forward and backward captured once; every replay, on new inputs and with
    eager work between, equals the eager results to the bit."""
    layer = RoutedExperts(256, 512, 8, 2, seed=1)
    x, dout = normal(gen(1), 300, 256, dt=torch.bfloat16), normal(gen(2), 300, 256, dt=torch.bfloat16)

    def work():
        out, kept = layer.forward(x, keep=True)
        dx, grads = layer.backward(dout, kept)
        return [out, dx, kept[2], kept[3], *grads.values()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    say("layer: capture")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for seed in range(4):
        x.copy_(normal(gen(10 + seed), 300, 256, dt=torch.bfloat16))
        dout.copy_(normal(gen(20 + seed), 300, 256, dt=torch.bfloat16))
        eager = [t.clone() for t in work()]
        for t in held:
            t.fill_(-1 if not t.dtype.is_floating_point else math.nan)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, eager):
            assert torch.equal(a, b), seed


def test_layer_on_another_stream():
    layer = RoutedExperts(256, 512, 8, 2, seed=1)
    x = normal(gen(1), 100, 256, dt=torch.bfloat16)
    want = layer.forward(x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = layer.forward(x)
    s.synchronize()
    assert torch.equal(got, want)
    logits = fl.grouped_linear(x, layer.Wr[None], every_row(x), act="none")
    s.wait_stream(torch.cuda.current_stream())
    w, e = fl.moe_route(logits, 2, stream=s)  # the stream as an argument
    plan = fl.moe_plan(e, 8, stream=s)
    h = fl.grouped_linear(x, layer.W1, plan.offsets, layer.b1, act="gelu_tanh", index=plan.token_of_row, stream=s)
    y = fl.grouped_linear(h, layer.W2, plan.offsets, layer.b2, act="none", stream=s)
    out = fl.moe_combine(y, plan.row_of_slot, w, R=x, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


# ------------------------------------------- beyond 2^31 elements

def test_rows_beyond_31_bits():
    """S*N and S*H above 2^31: products, gradients and movement at the end of
    their arrays."""
    S, K, N = 150_000, 64, 14_336 + 8
    g = gen(9)
    counts = [S - 300, 0, 300]
    offsets = offsets_of(counts)
    A, B = normal(g, S, K, dt=torch.bfloat16), normal(g, 3, K, N, std=0.1, dt=torch.bfloat16)
    say("S*N beyond 2^31")
    out = fl.grouped_linear(A, B, offsets, act="none")
    tail = A[-300:].double()
    check(out[-300:], tail @ B[2].double(), K * U32 * (tail.abs() @ B[2].double().abs()), torch.bfloat16)
    head = A[:70].double()
    check(out[:70], head @ B[0].double(), K * U32 * (head.abs() @ B[0].double().abs()), torch.bfloat16)
    dW, db = fl.grouped_weight_grad(A, out, offsets)
    d = out[-300:].double()
    check(dW[2], tail.t().contiguous() @ d, 320 * U32 * (tail.abs().t().contiguous() @ d.abs()), torch.bfloat16)
    check(db[2], d.sum(0), 320 * U32 * d.abs().sum(0), torch.float32)
    assert bool((dW[1] == 0).all()) and bool((db[1] == 0).all())
    back, _ = fl.grouped_linear_bwd(out, B, None, offsets, act="none")
    check(back[-300:], d @ B[2].double().t().contiguous(), N * U32 * (d.abs() @ B[2].double().abs().t().contiguous()),
          torch.bfloat16)
    index = torch.arange(S - 1, -1, -1, dtype=torch.int32, device="cuda")
    rows = fl.moe_gather(out, index)
    assert torch.equal(rows[-50:], out[:50].flip(0)) and torch.equal(rows[:50], out[-50:].flip(0))
    comb = fl.moe_combine(out, index[:, None].contiguous(), None, out=rows)
    assert torch.equal(comb[-50:], out[:50].flip(0))
    _, dw = fl.moe_combine_bwd(out, out, torch.arange(S, dtype=torch.int32, device="cuda")[:, None], None, drows=rows)
    assert torch.equal(rows[-50:], out[-50:])
    sq = (d * d).sum(1)
    check(dw[-300:, 0], sq, N * U32 * sq, torch.float32)


def test_weights_beyond_31_bits():
    """E*K*N above 2^31: the last expert's weights."""
    E, K, N = 40, 4096, 14_336
    g = gen(11)
    B = torch.zeros(E, K, N, dtype=torch.bfloat16, device="cuda")
    B[E - 1] = normal(g, K, N, std=K ** -0.5, dt=torch.bfloat16)
    A = normal(g, 20, K, dt=torch.bfloat16)
    counts = [3] + [0] * (E - 2) + [17]
    say("E*K*N beyond 2^31")
    out = fl.grouped_linear(A, B, offsets_of(counts), act="none")
    a, b = A[3:].double(), B[E - 1].double()
    check(out[3:], a @ b, (K + 20) * U32 * (a.abs() @ b.abs()), torch.bfloat16)
    assert bool((out[:3] == 0).all())
    D = normal(g, 20, N, dt=torch.bfloat16)
    dA, _ = fl.grouped_linear_bwd(D, B, None, offsets_of(counts), act="none")
    d = D[3:].double()
    bt = b.t().contiguous()
    check(dA[3:], d @ bt, N * U32 * (d.abs() @ bt.abs()), torch.bfloat16)
    dW, _ = fl.grouped_weight_grad(A, D, offsets_of(counts), dbias=None, dW=B)
    ref = A[3:].double().t().contiguous() @ d
    check(dW[E - 1], ref, 40 * U32 * (A[3:].double().abs().t().contiguous() @ d.abs()), torch.bfloat16)
    assert bool((dW[E - 2] == 0).all())


# ------------------------------------------- routing and plans of many tokens

@pytest.mark.parametrize("E,k,options", [
    (200, 8, {}), (256, 8, dict(score="sigmoid", bias=True, groups=8, top_groups=4, group_top=2)),
    (144, 16, dict(renorm=False, groups=16, top_groups=5, group_top=2)), (256, 3, dict(bias=True)), (64, 6, {}),
    (20, 5, dict(score="sigmoid", renorm=False, bias=True))])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_route_many_tokens(E, k, options, dtype):
    """Long batches take other lane arrangements than short ones: the choices
    are the same, the weights up to the order of fp32 sums over at most E."""
    T, options = 5003, dict(options)
    g = gen(E + k)
    x = normal(g, T, E, std=2.0, dt=DT[dtype])
    x[torch.rand(T, E, generator=g, device="cuda") < 0.1] = -math.inf
    x[7], x[4096] = -math.inf, math.nan
    bias = normal(g, E, std=0.1) if options.pop("bias", False) else None
    say("route many", E, k, options, dtype)
    w, e = fl.moe_route(x, k, bias=bias, **options)
    dw = normal(g, T, k)
    how = {n: options[n] for n in ("score", "renorm") if n in options}
    d = fl.moe_route_bwd(x, e, dw, **how)
    parts = [fl.moe_route(x[i:i + 100].contiguous(), k, bias=bias, **options) for i in range(0, T, 100)]
    assert torch.equal(e, torch.cat([p[1] for p in parts]))
    other = torch.cat([p[0] for p in parts])
    assert float((w - other).abs().max()) <= 2 * (E + 8) * U32
    assert int((e[7] >= 0).sum()) == 0 and float(w[7].abs().max()) == 0.0 and float(w[4096].abs().max()) == 0.0
    back = torch.cat([fl.moe_route_bwd(x[i:i + 100].contiguous(), e[i:i + 100].contiguous(), dw[i:i + 100].contiguous(), **how)
                      for i in range(0, T, 100)])
    # sums of terms below 5 (weights at most 1, |dw| below 5) in another order, one rounding each
    assert float((d.double() - back.double()).abs().max()) <= 10 * (E + 8) * U32 + 2 * unit(DT[dtype]) * float(back.abs().max())


def test_plan_of_many_slots():
    for T, k, E in ((70001, 7, 256), (30000, 3, 1000), (100000, 8, 5)):
        g = gen(T)
        e = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
        say("plan many", T, k, E)
        plan = fl.moe_plan(e, E)
        flat = e.reshape(-1).long()
        key = torch.where(flat < 0, E, flat)
        order = torch.sort(key, stable=True).indices
        n = int((flat >= 0).sum())
        counts = torch.bincount(key, minlength=E + 1)[:E]
        assert torch.equal(plan.offsets[1:].long(), counts.cumsum(0)) and int(plan.offsets[0]) == 0
        assert torch.equal(plan.token_of_row[:n].long(), order[:n] // k) and bool((plan.token_of_row[n:] == -1).all())
        rows = torch.full_like(flat, -1)
        rows[order[:n]] = torch.arange(n, device="cuda")
        assert torch.equal(plan.row_of_slot.reshape(-1).long(), rows)


# ------------------------------------------------ operands off 16 bytes

@pytest.mark.parametrize("dtype", list(DT))
def test_unaligned_operands(dtype):
    """Every operand one element past a 16-byte boundary gives the bits of the
    aligned call."""
    dt, g = DT[dtype], gen(31)
    counts, K, N = [70, 0, 130, 3], 136, 264
    offsets, S, E = offsets_of(counts), 203, 4

    def off(t):
        buf = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:].copy_(t.reshape(-1))
        return buf[1:].view(t.shape)
    A, B, bias, Y = normal(g, S, K, dt=dt), normal(g, E, K, N, dt=dt), normal(g, E, N, dt=dt), normal(g, S, N, dt=dt)
    G, W, X, D = normal(g, S, K, dt=dt), normal(g, E, N, K, dt=dt), normal(g, S, N, dt=dt), normal(g, S, N, dt=dt)
    index = torch.randperm(S, generator=g, device="cuda").to(torch.int32)
    say("unaligned", dtype)
    want = fl.grouped_linear(A, B, offsets, bias, Y, act="glu", index=index, pre=True)
    got = fl.grouped_linear(off(A), off(B), off(offsets), off(bias), off(Y), act="glu", index=off(index),
                            out=off(torch.zeros_like(Y)), pre=off(torch.zeros_like(Y)))
    want += fl.grouped_linear_bwd(G, W, X, offsets, Y, act="glu")
    got += fl.grouped_linear_bwd(off(G), off(W), off(X), offsets, off(Y), act="glu", dX=off(torch.zeros_like(Y)),
                                 dY=off(torch.zeros_like(Y)))
    want += fl.grouped_weight_grad(A, D, offsets)
    got += fl.grouped_weight_grad(off(A), off(D), offsets, dW=off(torch.zeros_like(B)))
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_no_tokens():
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    layer = RoutedExperts(64, 96, 4, 2)
    w, e = fl.moe_route(torch.zeros(0, 4, device="cuda"), 2)
    plan = fl.moe_plan(e, 4)
    assert w.shape == e.shape == (0, 2) and plan.offsets.tolist() == [0] * 5
    h = fl.grouped_linear(x, layer.W1, plan.offsets, layer.b1, act="gelu_tanh", index=plan.token_of_row)
    assert h.shape == (0, 96)
    assert fl.moe_combine(h, plan.row_of_slot, w).shape == (0, 96)
    dW, db = fl.grouped_weight_grad(x, h, plan.offsets)
    assert bool((dW == 0).all()) and bool((db == 0).all())
    assert fl.moe_gather(x, plan.token_of_row).shape == (0, 64)
