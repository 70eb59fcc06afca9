"""Microscaled 4-bit floating point in 64 bits on the CPU, written from the
format's definition, and the linear layer over it.

The codes of a block are its values over the scale, each at the nearest of the
16 values (both neighbours as far: the even code); nothing is rounded before
that, so codes and scales have to be equal.  Bounds of the linear layer are
moe_util's: a sum of n products in fp32 is off by at most n * 2^-23 * sum
|terms|, the activation as there, one rounding to the output's type.
"""
import torch

from moe_util import U32, act64, act_bound

MAGNITUDES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def quantize64(x):
    """(codes (rows, 16 blocks), scales (rows, blocks)), uint8, of a matrix."""
    rows, K = x.shape
    blocks = (K + 31) // 32
    v = torch.zeros(rows, blocks * 32, dtype=torch.float64)
    v[:, :K] = x.double()
    v = v.view(rows, blocks, 32)
    bad = ~torch.isfinite(v).all(2)
    v = torch.where(bad[..., None], torch.zeros_like(v), v)
    top = v.abs().amax(2)
    e = torch.frexp(top).exponent.long() - 1 - 2
    s = torch.where(top > 0, (e + 127).clamp(min=0), torch.zeros_like(e))
    m = v.abs() / torch.exp2(s.double() - 127)[..., None]
    off = (m[..., None] - MAGNITUDES).abs()
    near = off == off.amin(3, keepdim=True)
    # of two as near the even code
    rank = near.double() * (1 + (torch.arange(8) % 2 == 0).double() * 0.5)
    code = rank.argmax(3)
    code = code + 8 * torch.signbit(v).long()
    code = torch.where(bad[..., None], torch.zeros_like(code), code).view(rows, blocks * 16, 2)
    return (code[..., 0] + 16 * code[..., 1]).to(torch.uint8), torch.where(bad, 255, s).to(torch.uint8)


def values64(codes, scales, K):
    """(rows, K) in 64 bits."""
    rows, blocks = scales.shape
    c = torch.stack([codes.long() & 15, codes.long() >> 4], 2).view(rows, blocks, 32)
    v = MAGNITUDES[c & 7] * (1 - 2 * (c >> 3)).double()
    v = v * torch.exp2(scales.double() - 127)[..., None]
    v = torch.where((scales == 255)[..., None], torch.full_like(v, float("nan")), v)
    return v.view(rows, blocks * 32)[:, :K]


def linear64(a, b, bias, Y, R, act):
    """(out, its bound before the rounding) of the values a (M,K), b (N,K)."""
    K = a.shape[1]
    x, size = a @ b.t(), a.abs() @ b.abs().t()
    terms = K + 1
    for t in (bias, R):
        if t is not None:
            x, size, terms = x + t.double(), size + t.double().abs(), terms + 1
    ex = terms * U32 * size
    y = Y.double() if Y is not None else torch.zeros_like(x)
    return act64(x, y, act), act_bound(x, y, act, ex)
