"""Plain 64-bit layer norm, written from its formulas, and the error bounds the
kernels' results are held to.  torch on the CPU throughout.

Bounds.  u = 2^-24 is a rounding in fp32, unit(dtype) one to the output's
type.  A sum of n terms whose longest chain of additions is c long is off by at
most c * u * sum |terms|; chains here are a lane's own elements (at most 64, or
H / 1024 * 8 of a row too long for registers), a tree of 6 steps, 16 waves.
Products and quotients add a rounding each.  First orders are summed and
doubled, for what they leave out.
"""
import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def smallest(dtype):
    """Half the smallest step of the type."""
    return 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134


def chain(H):
    return 64 + H / 128 + 24


def forward64(x, weight, bias, eps):
    """(y, mean, rstd, bounds of the three) of x (M,H) in its own type."""
    dt, H = x.dtype, x.shape[1]
    x = x.double()
    mean = x.mean(1)
    d = x - mean[:, None]
    var = (d * d).mean(1)
    rstd = (var + eps) ** -0.5
    w = torch.ones(H, dtype=torch.float64) if weight is None else weight.double()
    b = torch.zeros(H, dtype=torch.float64) if bias is None else bias.double()
    hat = d * rstd[:, None]
    y = hat * w + b
    c = chain(H)
    e_mean = (c + 2) * U * x.abs().mean(1)
    e_d = e_mean[:, None] + U * d.abs()
    e_var = (2 * d.abs() * e_d + e_d * e_d).mean(1) + (c + 3) * U * var
    least = (var + eps - e_var).clamp(min=1e-300)
    rel = ((var + eps) / least).sqrt() - 1 + 4 * U
    e_rstd = rel * rstd
    e_hat = e_d * rstd[:, None] * (1 + rel[:, None]) + hat.abs() * (rel[:, None] + 2 * U)
    e_y = 2 * (w.abs() * e_hat + 2 * U * ((hat * w).abs() + b.abs()))
    e_y = e_y + unit(dt) * (y.abs() + e_y) + smallest(dt)
    return y, mean, rstd, (e_y, 2 * e_mean + U * mean.abs(), 2 * e_rstd)


def backward64(dy, x, mean, rstd, weight, residual):
    """(dx, dweight, dbias, their bounds) with the statistics as they are given."""
    dt, (M, H) = x.dtype, x.shape
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    w = torch.ones(H, dtype=torch.float64) if weight is None else weight.double()
    hat, g = (x - mean) * rstd, dy * w
    c1, c2 = g.mean(1, keepdim=True), (g * hat).mean(1, keepdim=True)
    dx = rstd * (g - c1 - hat * c2)
    c = chain(H)
    e_c1 = (c + 3) * U * g.abs().mean(1, keepdim=True)
    e_c2 = (c + 6) * U * (g * hat).abs().mean(1, keepdim=True)
    e_dx = rstd * (e_c1 + hat.abs() * e_c2 + 6 * U * (g.abs() + c1.abs() + (hat * c2).abs()))
    if residual is not None:
        dx = dx + residual.double()
        e_dx = e_dx + U * (dx.abs() + residual.double().abs())
    e_dx = 2 * e_dx + unit(dt) * (dx.abs() + 2 * e_dx) + smallest(dt)
    # rows of a team one after another, the teams of a block, the blocks of a join
    rows = min(M, M / 256 + 2) + 32 + 32
    e_w = 2 * (rows + 4) * U * (dy * hat).abs().sum(0)
    e_b = 2 * rows * U * dy.abs().sum(0)
    return dx, (dy * hat).sum(0), dy.sum(0), (e_dx, e_w, e_b)


def inside(got, want, bound):
    """Whether every element of got is within its bound (and as many are NaN)."""
    off = (got.detach().cpu().double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} out of bound, at {bad.nonzero()[0].tolist()}: "
                           f"{float(got.cpu().double()[bad][0])} for {float(want[bad][0])}, "
                           f"bound {float(bound.expand_as(off)[bad][0])}")
