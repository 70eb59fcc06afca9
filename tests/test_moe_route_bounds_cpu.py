"""The bounds that the router's results are held to tell right from wrong, for
every kind of input: a weight off by a thousandth, weights shared evenly and a
gradient of the other sign lie outside them."""
import pytest
import torch

from moe_route_bounds import gradient_allowance, weight_bound
from moe_util import DT, route64, route_bwd64
from test_moe_gpu import DTYPES, ROUTES, normal, route_logits

CASES = [c for c in range(len(ROUTES)) if ROUTES[c][1] <= 256]


@pytest.mark.parametrize("kind", ["plain", "masked", "ties", "extreme"])
@pytest.mark.parametrize("case", CASES)
def test_wrong_results_are_outside_the_bounds(case, kind):
    T, E, k, o = ROUTES[case]
    o, dtype = dict(o), DT[DTYPES[case % 3]]
    g = torch.Generator().manual_seed(100 * case + len(kind))
    x = route_logits(g, T, E, dtype, kind)
    bias = normal(g, E, std=0.2) if o.pop("bias", False) else None
    w, e = route64(x, k, bias=bias, **o)
    how = {n: o[n] for n in ("score", "renorm", "scale") if n in o}
    bound = weight_bound(x, e, w, **how)
    live = w.abs() > 1e-30
    assert bool((((w * (1 + 2.0 ** -10)) - w).abs() > bound)[live].all())
    assert bool((w.float().double() - w).abs().le(bound).all())
    if how.get("renorm", True):
        share = torch.where(e >= 0, how.get("scale", 1.0) / (e >= 0).sum(1, keepdim=True).clamp(min=1), 0.0)
        uneven = ((w - share).abs().amax(1) > 1e-3)
        assert bool(((share - w).abs() > bound).any(1)[uneven].all())
    dw = normal(g, T, k)
    d, mag = route_bwd64(x, e, dw, **how)
    allow = gradient_allowance(x, e, d, mag, dtype, **{n: v for n, v in how.items() if n != "scale"})
    # no cancellation, nothing next to zero (a raw sigmoid's is one product)
    alone = how.get("score") == "sigmoid" and not how.get("renorm", True)
    clear = d.abs() > (1e-30 if alone else 1e-2 * mag.amax(1, keepdim=True).clamp(min=1e-28))
    assert bool((2 * d.abs() > allow)[clear].all())
    assert bool(((d.to(dtype).double() - d).abs() <= allow).all())
    # (one renormalised choice has the weight 1 and no gradient; sigmoids of the largest of such logits are flat)
    if (k > 1 or not how.get("renorm", True)) and not (alone and kind == "extreme"):
        assert int(clear.any(1).sum()) > 0
