"""Error bounds of the router's weights and of its logits' gradient, for each
token by itself, and 64-bit results to hold them to.

u = 2^-24 is half a step of fp32, U32 = 2u.  The exponential and the logarithm
are taken to be off by 2 steps (2 U32), the quotient and products by u.

Renormalised softmax weights: p_j = exp(d_j), d_j = x_j - max x rounded once, so
off by u |d_j|, relatively; the sum of n of them weighs these errors with p_j, and
p |d| is at most 1/e.  With the additions, the quotient and the scale a weight is
off by less than (|d_j| + n + 8) U32, relatively.  Raw softmax weights: the same
with all E logits.
Renormalised sigmoid weights: of the logarithms l = min(x,0) - q, q =
log1p(exp(-|x|)), q is off by 4 U32 q and the difference by u |l|, unless q is 0
in fp32 (|x| above 104) and l is x: e(l).  A difference from the largest, m, is off
by e(l_j) + e(m) + u |d_j|, the sum's by less than 3 e(m) + (n/e + 3) U32: a weight
by less than e(l_j) + 4 e(m) + (|d_j| + 2 n + 12) U32.
Raw sigmoid weights: 1 / (1 + exp(-x)), 8 U32.
What underflows is off by the smallest normal number at most: 2^-125 in all.

Gradients.  Renormalised: p_j (d_j - sum_l d_l p_l), every p off by the token's
largest relative error r, k additions and a few products: (2 r + (k + 12) U32)
times the sum of the terms' absolute values.  Raw softmax: s_i (d_i - sum_j d_j s_j)
likewise, with the errors of s_i and of the chosen s_j.  Raw sigmoid:
d s (1 - s), the factors computed apart: 20 U32 of the value.
"""
import math

import torch

from moe_util import U32, floor_of, unit

TINY = 2.0 ** -125


def log_sigmoid(x):
    """(the logarithm of the sigmoid, how far the fp32 one may be off)"""
    q = math.log1p(math.exp(-abs(x)))
    l = min(x, 0.0) - q
    return l, (4 * U32 * q + U32 / 2 * abs(l) if abs(x) < 104 else 0.0)


def weight_rel(x, experts, score, renorm):
    """Relative error of each weight of one token: x its logits (a list, -inf
    or NaN masked), experts its choice (-1: none)."""
    x = [v if v > -math.inf else -math.inf for v in x]
    if score == "sigmoid" and not renorm:
        return [8 * U32 for _ in experts]
    over = [x[e] for e in experts if e >= 0] if renorm else [v for v in x if v > -math.inf]
    if not over:
        return [0.0 for _ in experts]
    n = len(over)
    if score == "sigmoid":
        m, em = max(log_sigmoid(v) for v in over)
        of = [log_sigmoid(x[e]) if e >= 0 else (m, 0.0) for e in experts]
        return [err + 4 * em + (abs(l - m) + 2 * n + 12) * U32 for l, err in of]
    m = max(over)  # (below an infinite one a weight is 0, without an error)
    return [0.0 if e < 0 or (x[e] != m and math.isinf(m - x[e])) else ((0.0 if x[e] == m else m - x[e]) + n + 8) * U32
            for e in experts]


def weight_bound(logits, experts, weights64, score="softmax", renorm=True, scale=1.0):
    """How far each weight may be off (T,k)."""
    rel = torch.tensor([weight_rel(x.tolist(), e.tolist(), score, renorm) for x, e in zip(logits.double(), experts)],
                       dtype=torch.float64).reshape(experts.shape)
    return rel * weights64.abs() + TINY * max(1.0, abs(scale))


def gradient_rel(logits, experts, score="softmax", renorm=True):
    """Relative error of an entry's terms (T,E)."""
    T, E = logits.shape
    out = torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        x = [v if v > -math.inf else -math.inf for v in logits[t].double().tolist()]
        e = [int(v) for v in experts[t]]
        r = max(weight_rel(x, e, score, renorm), default=0.0)
        if score == "sigmoid" and not renorm:
            out[t] = 20 * U32
        elif renorm:
            out[t] = 2 * r + (len(e) + 12) * U32
        else:
            every = weight_rel(x, list(range(E)), score, renorm)
            out[t] = torch.tensor([r + (w if x[i] > -math.inf else 0.0) + (len(e) + 12) * U32
                                   for i, w in enumerate(every)])
    return out


def gradient_allowance(logits, experts, grad64, mag, dtype, score="softmax", renorm=True):
    """How far each entry of the gradient, rounded to dtype, may be off (T,E)."""
    size = grad64.abs() if score == "sigmoid" and not renorm else mag
    bound = gradient_rel(logits, experts, score, renorm) * size + 2.0 ** -120
    u = unit(dtype)
    return bound * (1 + u) + u * grad64.abs() + floor_of(dtype)

