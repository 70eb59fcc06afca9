"""Plain 64-bit implementations of the routed-experts operators, written from
their definitions one token, slot or expert at a time, and the error bounds
their results are held to.  torch on the CPU throughout.

Bounds.  A rounding to a type with unit roundoff u = eps/2 is off by at most
u * |value| (plus half the smallest step, which only fp16 meets).  A sum of n
products in fp32 is off by at most n * 2^-23 * sum |terms|: 2^-24 for each
addition, doubled because a matrix instruction may truncate where the
definition rounds.
"""
import math

import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U32 = 2.0 ** -23


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def floor_of(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134


# ------------------------------------------------------------------ router

def scores64(x, kind):
    """Scores of one token's logits (a list of floats, -inf or NaN: masked)."""
    x = [v if v > -math.inf else -math.inf for v in x]
    if kind == "sigmoid":
        return [1.0 / (1.0 + math.exp(-v)) if v > -700 else (math.exp(v) if v > -math.inf else 0.0) for v in x]
    m = max(x)
    if m == -math.inf:
        return [0.0] * len(x)
    e = [1.0 if v == m else math.exp(v - m) if v > -math.inf else 0.0 for v in x]
    return [v / sum(e) for v in e]


def route64(logits, k, bias=None, score="softmax", groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0):
    """(weights (T,k) float64, experts (T,k) int64) by the definition."""
    T, E = logits.shape
    weights, experts = torch.zeros(T, k, dtype=torch.float64), torch.full((T, k), -1)
    per = E // groups
    for t in range(T):
        x = [float(v) if float(v) > -math.inf else -math.inf for v in logits[t].double()]
        s = scores64(x, score)
        key = [x[e] if bias is None else s[e] + float(bias[e]) for e in range(E)]
        live = [e for e in range(E) if x[e] > -math.inf and key[e] > -math.inf]
        if groups > 1:
            rank = []
            for g in range(groups):
                by = s if bias is None and group_top == 2 else key
                top = sorted((by[e] for e in live if e // per == g), reverse=True)[:group_top]
                if top:
                    rank.append((-sum(top), g))
            kept = [g for _, g in sorted(rank)[:top_groups]]
            live = [e for e in live if e // per in kept]
        chosen = sorted(live, key=lambda e: (-key[e], e))[:k]
        logs = [x[e] if score == "softmax" else min(x[e], 0.0) - math.log1p(math.exp(-abs(x[e]))) for e in chosen]
        for j, e in enumerate(chosen):
            experts[t, j] = e
            if renorm:  # s_j / sum s from the logs, which cannot underflow together
                m = max(logs)
                z = [1.0 if v == m else math.exp(v - m) for v in logs]
                weights[t, j] = scale * z[j] / sum(z)
            else:
                weights[t, j] = scale * s[e]
    return weights, experts


def weight_rel(logits, n):
    """Relative error of a weight in fp32: the exponent (a difference, or the
    log of a sigmoid, rounded at the size of the largest logit, twice), n
    additions, and a few units for the exponential, logarithm and quotient."""
    x = logits.double()
    x = x[torch.isfinite(x)]
    return (2 * float(x.abs().max()) if x.numel() else 0.0) * U32 + (n + 8) * U32


def route_bwd64(logits, experts, dweights, score="softmax", renorm=True, scale=1.0):
    """(dlogits (T,E) float64 from the Jacobian of the weights, entry by entry;
    the sum of the absolute values of each entry's terms)."""
    T, E = logits.shape
    out, mag = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        x = [float(v) if float(v) > -math.inf else -math.inf for v in logits[t].double()]
        s = scores64(x, score)
        chosen = [(j, int(e)) for j, e in enumerate(experts[t]) if 0 <= int(e) < E and x[int(e)] > -math.inf]
        d = {j: scale * float(dweights[t, j]) for j, _ in chosen}
        rest = scores64([-v if v > -math.inf else v for v in x], "sigmoid")  # 1 - s of the sigmoid, without cancellation
        if renorm and chosen:
            logs = [x[e] if score == "softmax" else min(x[e], 0.0) - math.log1p(math.exp(-abs(x[e]))) for _, e in chosen]
            m = max(logs)
            z = [1.0 if v == m else math.exp(v - m) for v in logs]
            p = [v / sum(z) for v in z]
            for i, (j, e) in enumerate(chosen):
                slope = rest[e] if score == "sigmoid" else 1.0
                for l, (j2, _) in enumerate(chosen):
                    term = slope * d[j2] * p[l] * ((1.0 if l == i else 0.0) - p[i])
                    out[t, e] += term
                    mag[t, e] += slope * abs(d[j2]) * p[l] * ((1.0 if l == i else 0.0) + p[i])
        elif not renorm:
            for j, e in chosen:
                if score == "sigmoid":
                    out[t, e] += d[j] * s[e] * rest[e]
                    mag[t, e] += abs(d[j]) * s[e]
                else:
                    for i in range(E):
                        out[t, i] += d[j] * s[e] * ((1.0 if i == e else 0.0) - s[i])
                        mag[t, i] += abs(d[j]) * s[e] * ((1.0 if i == e else 0.0) + s[i])
    return out, mag


# -------------------------------------------------------------------- plan

def plan64(experts, E):
    """(offsets, token_of_row, row_of_slot) as lists of lists would sort them."""
    T, k = experts.shape
    runs = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            e = int(experts[t, j])
            if 0 <= e < E:
                runs[e].append((t, j))
    offsets, tokens = [0], []
    row_of_slot = torch.full((T, k), -1, dtype=torch.int32)
    for run in runs:
        for t, j in run:
            row_of_slot[t, j] = len(tokens)
            tokens.append(t)
        offsets.append(len(tokens))
    tokens += [-1] * (T * k - len(tokens))
    return torch.tensor(offsets, dtype=torch.int32), torch.tensor(tokens, dtype=torch.int32), row_of_slot


# ------------------------------------------------------- experts' products

def act64(x, y, act):
    if act == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
    return x + x * y if act == "glu" else x


def act_grad64(x, y, act):
    if act == "relu":
        return (x > 0).double()
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (x + 0.044715 * x ** 3))
        return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)
    return 1 + y if act == "glu" else torch.ones_like(x)


def act_bound(x, y, act, ex):
    """How far the fp32 activation of x may be off where x itself is off by ex.
    GELU's slope is below 1.13 and its exponential, quotient and products add
    at most 8 units of fp32 (the exponent's error, a few units of 2|u|, meets
    the sigmoid's slope, below 0.45 / 2|u|)."""
    if act == "glu":
        return ex * (1 + y.abs()) + U32 * (x.abs() + (x * y).abs())
    if act == "gelu_tanh":
        return 1.13 * ex + 8 * U32 * x.abs()
    return ex


def act_grad_bound(x, y, act):
    """How far the fp32 derivative may be off: GELU's has a few products of
    values below 1.13 and x * s * (1 - s) * du, below 0.6, each with the
    exponential's error."""
    if act == "gelu_tanh":
        return 16 * U32 * torch.ones_like(x)
    return U32 * (1 + y.abs()) if act == "glu" else torch.zeros_like(x)


def runs_of(offsets):
    o = [int(v) for v in offsets]
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1) if o[e + 1] > o[e]]


def grouped64(A, index, offsets, B, bias, Y, act):
    """(out, its bound, pre, its bound), rows outside every run NaN."""
    E, K, N = B.shape
    S = A.shape[0] if index is None else index.numel()
    A64 = A.double()
    if index is not None:
        at = index.long()
        ok = (at >= 0) & (at < A.shape[0])
        A64 = torch.where(ok[:, None], A64[at.clamp(0, max(0, A.shape[0] - 1))], torch.zeros(1, dtype=torch.float64))
    res = [torch.full((S, N), math.nan, dtype=torch.float64) for _ in range(4)]
    for e, lo, hi in runs_of(offsets):
        a, b = A64[lo:hi], B[e].double()
        c = bias[e].double() if bias is not None else torch.zeros(N, dtype=torch.float64)
        x = a @ b + c
        ex = (K + 1) * U32 * (a.abs() @ b.abs() + c.abs())
        y = Y[lo:hi].double() if Y is not None else torch.zeros_like(x)
        res[2][lo:hi], res[3][lo:hi] = x, ex
        res[0][lo:hi], res[1][lo:hi] = act64(x, y, act), act_bound(x, y, act, ex)
    return res


def grouped_bwd64(G, W, X, offsets, Y, act):
    """(dX, its bound, dY, its bound), rows outside every run NaN."""
    E, N, K = W.shape
    S = G.shape[0]
    res = [torch.full((S, N), math.nan, dtype=torch.float64) for _ in range(4)]
    for e, lo, hi in runs_of(offsets):
        g, w = G[lo:hi].double(), W[e].double().t()
        d = g @ w
        ed = K * U32 * (g.abs() @ w.abs())
        x = X[lo:hi].double() if X is not None else torch.zeros_like(d)
        y = Y[lo:hi].double() if Y is not None else torch.zeros_like(d)
        slope, es = act_grad64(x, y, act), act_grad_bound(x, y, act)
        res[0][lo:hi] = d * slope
        res[1][lo:hi] = ed * (slope.abs() + es) + d.abs() * es + U32 * (d * slope).abs()
        res[2][lo:hi] = d * x
        res[3][lo:hi] = ed * x.abs() + U32 * (d * x).abs()
    return res


def weight_grad64(A, G, offsets):
    """(dW, its bound, dbias, its bound)."""
    E, K, N = len(offsets) - 1, A.shape[1], G.shape[1]
    dW, bW = (torch.zeros(E, K, N, dtype=torch.float64) for _ in range(2))
    db, bb = (torch.zeros(E, N, dtype=torch.float64) for _ in range(2))
    for e, lo, hi in runs_of(offsets):
        a, g = A[lo:hi].double(), G[lo:hi].double()
        dW[e], bW[e] = a.t() @ g, (hi - lo) * U32 * (a.abs().t() @ g.abs())
        db[e], bb[e] = g.sum(0), (hi - lo) * U32 * g.abs().sum(0)
    return dW, bW, db, bb


def worst(got, ref, bound, dtype):
    """The largest |got - ref| over its allowance: the bound and one rounding
    to dtype (of a value that is itself off by the bound)."""
    u = unit(dtype) if dtype is not None else 0.0
    allow = bound * (1 + u) + u * ref.abs() + (floor_of(dtype) if dtype is not None else 0.0)
    off = (got.double() - ref).abs()
    if not bool(torch.isfinite(got.double()).all()):
        return math.inf
    return float(torch.where(off == 0, torch.zeros_like(off), off / allow).max()) if off.numel() else 0.0
