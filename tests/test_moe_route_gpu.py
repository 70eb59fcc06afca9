"""The router's weights and its logits' gradient, each token held to its own
bounds (moe_route_bounds): masked experts, the type's lowest value, NaN, ties,
infinities, fewer experts left than choices; short and long batches."""
import math

import pytest
import torch

import activation_epilogue_amd as fl
from gpu_util import say
from moe_route_bounds import gradient_allowance, weight_bound
from moe_util import DT, route64, route_bwd64
from test_moe_gpu import ROUTES, guarded, normal, route_logits

pytestmark = pytest.mark.gpu


def check_tokens(x, w, e, d, dw, bias, o):
    """Every token of x against the definition (all on the CPU)."""
    rw, re = route64(x, e.shape[1], bias=bias, **o)
    assert torch.equal(e.long(), re)
    how = {n: o[n] for n in ("score", "renorm") if n in o}
    bound = weight_bound(x, re, rw, scale=o.get("scale", 1.0), **how)
    off = (w.double() - rw).abs()
    assert bool((off <= bound).all()), float((off / bound).max())
    rd, mag = route_bwd64(x, re, dw, scale=o.get("scale", 1.0), **how)
    allow = gradient_allowance(x, re, rd, mag, x.dtype, **how)
    off = (d.double() - rd).abs()
    assert bool((off <= allow).all()), float((off / allow).max())


@pytest.mark.parametrize("kind", ["plain", "masked", "ties", "extreme", "few"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", range(len(ROUTES)))
def test_route_of_each_token(case, dtype, kind):
    T, E, k, o = ROUTES[case]
    o, dt = dict(o), DT[dtype]
    g = torch.Generator().manual_seed(1000 * case + len(kind))
    x = route_logits(g, T, E, dt, kind)
    if kind == "few":  # 0 to k + 1 experts left for a token
        for t in range(T):
            left = torch.randperm(E, generator=g)[: t % (k + 2)]
            rest = torch.ones(E, dtype=torch.bool)
            rest[left] = False
            x[t, rest] = math.nan if t % 3 == 0 else -math.inf
    bias = normal(g, E, std=0.2) if o.pop("bias", False) else None
    say("route of each token", T, E, k, o, kind, dtype)
    (w, wok), (e, eok), (d, dok) = guarded((T, k), torch.float32), guarded((T, k), torch.int32), guarded((T, E), dt)
    fl.moe_route(x.cuda(), k, bias=None if bias is None else bias.cuda(), weights=w, experts=e, **o)
    dw = normal(g, T, k)
    how = {n: o[n] for n in ("score", "renorm", "scale") if n in o}
    fl.moe_route_bwd(x.cuda(), e.contiguous(), dw.cuda(), dlogits=d, **how)
    assert wok() and eok() and dok()
    check_tokens(x, w.cpu(), e.cpu(), d.cpu(), dw, bias, o)


@pytest.mark.parametrize("E,k,options", [
    (200, 8, {}), (256, 8, dict(score="sigmoid", bias=True, groups=8, top_groups=4, group_top=2, scale=2.5)),
    (144, 16, dict(renorm=False, groups=16, top_groups=5, group_top=2)), (256, 3, dict(bias=True)), (64, 6, {}),
    (20, 5, dict(score="sigmoid", renorm=False, bias=True)), (64, 6, dict(renorm=False)), (600, 20, {})])
@pytest.mark.parametrize("dtype", list(DT))
def test_tokens_of_a_long_batch(E, k, options, dtype):
    """Tokens at the ends of a long batch and within it, those with masks that
    leave nothing, one or a few experts among them, against the definition."""
    T, o, dt = 5003, dict(options), DT[dtype]
    g = torch.Generator().manual_seed(E * k)
    x = normal(g, T, E, std=2.0)
    x[torch.rand(T, E, generator=g) < 0.1] = -math.inf
    x[7], x[4096] = -math.inf, math.nan
    x[8], x[4097] = torch.finfo(dt).min, torch.finfo(dt).max
    for i, t in enumerate((5, 6, 9, 10, 2048, 4095, 4098, 5000)):
        x[t, torch.randperm(E, generator=g)[i:]] = math.nan if i % 2 else -math.inf
    x = x.to(dt)
    bias = normal(g, E, std=0.1) if o.pop("bias", False) else None
    say("tokens of a long batch", E, k, o, dtype)
    w, e = fl.moe_route(x.cuda(), k, bias=None if bias is None else bias.cuda(), **o)
    dw = normal(g, T, k)
    d = fl.moe_route_bwd(x.cuda(), e, dw.cuda(), **{n: o[n] for n in ("score", "renorm", "scale") if n in o})
    at = sorted({*range(16), *range(2040, 2056), *range(4088, 4104), *range(T - 16, T), *range(0, T, 97)})
    check_tokens(*(v.cpu()[at] for v in (x, w, e, d, dw)), bias, o)
