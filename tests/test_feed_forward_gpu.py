"""A feed-forward block of layer norm, linear layers and a path around them:
served with weights in 4 bits, and trained in one type.

Served: every operator's output is held to the 64-bit result for what it was
given on the device (quantising jumps at its borders, so errors in front of it
have no bound behind it).  Trained: the gradients are held to 64-bit autograd
of the whole block, with the bounds of each step carried through the next.
"""
import pytest
import torch

import activation_epilogue_amd as fl
from gpu_util import say
from moe_util import DT, U32, act64, act_grad64, worst
from mx4_util import linear64, quantize64, values64
from norm_util import backward64, forward64, inside

pytestmark = pytest.mark.gpu


def served(x, weight, bias, W1, b1, W2, b2, Y=None, ws=None, outs=(None,) * 4):
    act = "gelu_tanh" if Y is None else "glu"
    h = fl.layer_norm(x, weight, bias, out=outs[0])
    u = fl.fused_linear_mx4(h, W1, b1, Y, act=act, out=outs[1], workspace=ws)
    y = fl.fused_linear_mx4(u, W2, b2, act="none", R=x, out=outs[2], workspace=ws)
    return h, u, y, fl.layer_norm(y, weight, bias, out=outs[3])


def block(M, H, F, dt, seed, gate=False):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(dt)  # noqa: E731
    x, weight, bias = n(M, H), 1 + n(H, std=0.2), n(H, std=0.2)
    W1, b1, W2, b2 = n(H, F, std=H ** -0.5), n(F, std=0.3), n(F, H, std=F ** -0.5), n(H, std=0.3)
    Y = n(M, F) if gate else None
    return x, weight, bias, W1, b1, W2, b2, Y


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,H,F", [(1, 200, 520), (4, 256, 1024), (37, 333, 129), (600, 160, 555)])
def test_served(M, H, F, dtype, gate):
    dt = DT[dtype]
    x, weight, bias, W1, b1, W2, b2, Y = block(M, H, F, dt, M + H, gate)
    q1, q2 = fl.quantize_mx4(W1.cuda(), transposed=True), fl.quantize_mx4(W2.cuda(), transposed=True)
    say("feed-forward block served", M, H, F, dtype, gate)
    dev = [None if t is None else t.cuda() for t in (x, weight, bias, b1, b2, Y)]
    h, u, y, z = (t.cpu() for t in served(dev[0], dev[1], dev[2], q1, dev[3], q2, dev[4], dev[5]))
    for got, given in ((h, x), (z, y)):
        want, _, _, (bound, _, _) = forward64(given, weight, bias, 1e-5)
        inside(got, want, bound)
    for got, a, q, b, gates, r, act in ((u, h, q1, b1, Y, None, "glu" if gate else "gelu_tanh"),
                                        (y, u, q2, b2, None, x, "none")):
        K = a.shape[1]
        want, bound = linear64(values64(*quantize64(a), K), values64(q.codes.cpu(), q.scales.cpu(), K), b, gates, r, act)
        assert worst(got, want, bound, dt) <= 1.0


@pytest.mark.parametrize("M", [1, 16, 300])
def test_served_from_a_graph(M):
    """A whole block captured once; every replay gives what the calls give, with other work between."""
    H, F, dt = 256, 1030, torch.bfloat16
    x, weight, bias, W1, b1, W2, b2, _ = (None if t is None else t.cuda() for t in block(M, H, F, dt, 5))
    q1, q2 = fl.quantize_mx4(W1, transposed=True), fl.quantize_mx4(W2, transposed=True)
    need = max(fl.mx4_workspace_bytes(M, n, k, True, dt) for n, k in ((F, H), (H, F)))
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    outs = [torch.empty(M, n, dtype=dt, device="cuda") for n in (H, F, H, H)]
    args = (x, weight, bias, q1, b1, q2, b2)
    served(*args)  # loads what is to be loaded
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    say("feed-forward block captured", M)
    with torch.cuda.graph(graph):
        served(*args, ws=ws, outs=outs)
    for _ in range(4):
        x.normal_()
        want = served(*args)
        for t in outs:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("act", ["relu", "gelu_tanh"])
@pytest.mark.parametrize("M,H,F", [(5, 40, 72), (130, 96, 257)])
def test_trained(M, H, F, act):
    """sum(c * (x + act(norm(x) @ W + b) @ V)): the gradients of x, and of the norm's weight and bias."""
    dt = torch.float32
    x, weight, bias, W, b, V, _, _ = block(M, H, F, dt, 3 * M)
    c = torch.randn(M, H, generator=torch.Generator().manual_seed(9))
    say("feed-forward block trained", M, H, F, act)
    d = lambda t: t.cuda()  # noqa: E731
    h, mean, rstd = fl.layer_norm(d(x), d(weight), d(bias), stats=True)
    pre = fl.fused_linear(h, d(W), d(b), act="none")
    # (the activation's own backward pass is there for 16-bit types)
    dpre = (fl.gemm(d(c), d(V.t().contiguous())).double() * act_grad64(pre.double(), None, act)).float()
    dh = fl.gemm(dpre, d(W.t().contiguous()))
    dx, dw, db = fl.layer_norm_bwd(dh, d(x), mean, rstd, d(weight), R=d(c))

    leaves = [t.double().requires_grad_() for t in (x, weight, bias)]
    h64 = torch.nn.functional.layer_norm(leaves[0], (H,), leaves[1], leaves[2], 1e-5)
    pre64 = h64 @ W.double() + b.double()
    loss = (c.double() * (leaves[0] + act64(pre64, None, act) @ V.double())).sum()
    want = torch.autograd.grad(loss, leaves)

    # the steps' bounds, each over the errors it is given
    _, _, rstd64, (e_h, e_mean, e_rstd) = forward64(x, weight, bias, 1e-5)
    mean64 = x.double().mean(1, keepdim=True)
    h64, pre64 = h64.detach(), pre64.detach()
    e_pre = e_h @ W.double().abs() + (H + 2) * U32 * (h64.abs() @ W.double().abs() + b.double().abs())
    up, e_up = c.double() @ V.double().t(), (H + 1) * U32 * (c.double().abs() @ V.double().abs().t())
    slope = act_grad64(pre64, None, act)
    # GELU's second derivative is below 1.2; the rectifier's slope is 0 or 1, and either where its
    # argument is within its error of 0
    e_slope = 1.2 * e_pre if act == "gelu_tanh" else (pre64.abs() <= e_pre).double()
    dpre64 = up * slope
    e_dpre = e_up * (slope.abs() + e_slope) + up.abs() * e_slope + U32 * dpre64.abs()
    dh64 = dpre64 @ W.double().t()
    e_dh = e_dpre @ W.double().abs().t() + (F + 1) * U32 * (dpre64.abs() @ W.double().abs().t())
    dx64, _, _, (e_dx, e_w, e_b) = backward64(dh64.float(), x, mean64[:, 0], rstd64, weight, c)
    w, r = weight.double().abs(), rstd64[:, None]
    hat = (x.double() - mean64) * r
    rel = (e_rstd / rstd64)[:, None]  # of the statistics; hat's own error from them
    e_hat = e_mean[:, None] * r + rel * hat.abs()
    g, e_g = dh64.abs() * w, e_dh * w + 2.0 ** -24 * dh64.abs() * w  # dh64 was rounded to fp32 above
    mu = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    e_dx = e_dx + 2 * r * (e_g + mu(e_g) + hat.abs() * mu(e_g * hat.abs()) + e_hat * mu(g * hat.abs())
                           + hat.abs() * mu(g * e_hat) + rel * (g + mu(g) + hat.abs() * mu(g * hat.abs())))
    inside(dx, want[0], e_dx)
    inside(dw, want[1], e_w + 2 * (e_dh * hat.abs() + dh64.abs() * e_hat).sum(0) + 2.0 ** -24 * (dh64 * hat).abs().sum(0))
    inside(db, want[2], e_b + 2 * e_dh.sum(0) + 2.0 ** -24 * dh64.abs().sum(0))
    # the same bits again
    again = fl.layer_norm_bwd(dh, d(x), mean, rstd, d(weight), R=d(c))
    assert all(torch.equal(s, t) for s, t in zip((dx, dw, db), again))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_trained_in_16_bits(dtype):
    """The same steps with the fused backward layer: the norm's gradients for what they were given."""
    dt, M, H, F = DT[dtype], 130, 96, 264
    x, weight, bias, W, b, V, _, _ = block(M, H, F, dt, 11)
    c = torch.randn(M, H, generator=torch.Generator().manual_seed(9)).to(dt)
    say("feed-forward block trained", M, H, F, dtype)
    d = lambda t: t.cuda()  # noqa: E731
    h, mean, rstd = fl.layer_norm(d(x), d(weight), d(bias), stats=True)
    pre = fl.fused_linear(h, d(W), d(b), act="none")
    dpre, _, _ = fl.fused_linear_bwd(d(c), d(V), pre, act="gelu_tanh", dbias=False)
    dh = fl.gemm_nt(dpre, d(W))
    got = fl.layer_norm_bwd(dh, d(x), mean, rstd, d(weight), R=d(c))
    *want, bounds = backward64(dh.cpu(), x, mean.cpu(), rstd.cpu(), weight, c)
    for g, w, e in zip(got, want, bounds):
        inside(g, w, e)
