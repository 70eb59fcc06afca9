"""Refusals and degenerate sizes of the microscaled 4-bit C ABI, without a GPU:
validation runs before any HIP call, and the fake pointers are never read; and
the 64-bit definition that the GPU tests hold the kernels to."""
import ctypes
import os
import re

import pytest
import torch

from activation_epilogue_amd import mx4
from mx4_util import quantize64, values64

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, F16, BF16 = 0, 1, 2
NONE, RELU, GELU, GLU = 0, 1, 2, 3
P = [0x100000000 * (i + 1) for i in range(12)]  # far apart, aligned


@pytest.fixture(scope="module")
def lib():
    return mx4._lib()


def quantize(lib, X=P[0], codes=P[1], scales=P[2], rows=8, K=64, transposed=0, dt=BF16):
    return lib.fl_quantize_mx4(X, codes, scales, rows, K, transposed, dt, None)


def dequantize(lib, codes=P[1], scales=P[2], X=P[0], rows=8, K=64, dt=BF16):
    return lib.fl_dequantize_mx4(codes, scales, X, rows, K, dt, None)


def linear(lib, A=P[0], As=P[1], B=P[2], Bs=P[3], bias=P[4], Y=None, R=None, out=P[7], M=8, N=32, K=64, act=RELU, dt=BF16,
           ws=P[8], wb=1 << 30):
    return lib.fl_fused_linear_mx4(A, As, B, Bs, bias, Y, R, out, M, N, K, act, dt, ws, wb, None)


def said(lib):
    return lib.fl_mx4_last_error().decode()


def test_every_export_is_declared(lib):
    text = open(os.path.join(ROOT, "include", "fused_mx4.h"), encoding="utf-8").read()
    assert set(re.findall(r"\bfl_status (fl_\w+)\s*\(", text)) == set(mx4.MX4_EXPORTS) - {"fl_mx4_last_error"}
    for name in mx4.MX4_EXPORTS:
        assert name in text and hasattr(lib, name)


@pytest.mark.parametrize("call,kw,status,text", [
    (quantize, dict(dt=5), INVALID, "unknown dtype"),
    (quantize, dict(rows=-1), INVALID, "negative size"),
    (quantize, dict(rows=2 ** 31), UNSUPPORTED, "2^31-1"),
    (quantize, dict(K=2 ** 24), UNSUPPORTED, "K (16777216)"),
    (quantize, dict(X=None), INVALID, "X is NULL"),
    (quantize, dict(codes=None), INVALID, "codes is NULL"),
    (quantize, dict(scales=None), INVALID, "scales is NULL"),
    (quantize, dict(codes=P[1] + 8), INVALID, "not aligned to 16"),
    (quantize, dict(X=P[0] + 1), INVALID, "not aligned to 2"),
    (quantize, dict(codes=P[0] + 16), INVALID, "codes overlaps X"),
    (quantize, dict(scales=P[1]), INVALID, "overlaps"),
    (quantize, dict(transposed=2), INVALID, "transposed"),
    (dequantize, dict(X=P[1]), INVALID, "X overlaps codes"),
    (dequantize, dict(X=None), INVALID, "X is NULL"),
    (dequantize, dict(codes=P[1] + 4), INVALID, "not aligned to 16"),
    (linear, dict(dt=3), INVALID, "unknown dtype"),
    (linear, dict(act=4), INVALID, "unknown activation"),
    (linear, dict(act=GLU), INVALID, "needs Y"),
    (linear, dict(Y=P[5]), INVALID, "only used by the gate"),
    (linear, dict(A=None), INVALID, "A is NULL"),
    (linear, dict(A=P[0] + 2), INVALID, "not aligned to 16"),
    (linear, dict(As=None, A=P[0] + 1), INVALID, "not aligned to 2"),
    (linear, dict(B=None), INVALID, "B is NULL"),
    (linear, dict(Bs=None), INVALID, "B_scales is NULL"),
    (linear, dict(B=P[2] + 4), INVALID, "not aligned to 16"),
    (linear, dict(out=None), INVALID, "out is NULL"),
    (linear, dict(out=P[0]), INVALID, "out overlaps A"),
    (linear, dict(out=P[4]), INVALID, "out overlaps bias"),
    (linear, dict(R=P[7] + 2), INVALID, "out overlaps R"),
    (linear, dict(act=GLU, Y=P[7], R=P[7] + 2), INVALID, "out overlaps R"),
    (linear, dict(N=2 ** 23), UNSUPPORTED, "N too large"),
    (linear, dict(K=2 ** 23 - 32, dt=F32), UNSUPPORTED, "K or N too large"),
])
def test_refused(lib, call, kw, status, text):
    assert call(lib, **kw) == status and text in said(lib)


def test_nothing_to_do(lib):
    assert quantize(lib, rows=0, X=None, codes=None, scales=None) == OK and said(lib) == ""
    assert quantize(lib, K=0, X=None, codes=None, scales=None) == OK
    assert dequantize(lib, rows=0, X=None, codes=None, scales=None) == OK
    for kw in (dict(M=0), dict(N=0)):
        assert linear(lib, A=None, B=None, Bs=None, bias=None, out=None, ws=None, wb=0, **kw) == OK


def test_workspace(lib):
    size = mx4.mx4_workspace_bytes
    assert size(0, 100, 64, True, torch.bfloat16) == size(100, 0, 64, True, torch.bfloat16) == 0
    assert size(300, 100, 0, True, torch.float32) == 0
    n = ctypes.c_size_t()
    assert lib.fl_mx4_workspace_bytes(1, 1, 1, 2, BF16, ctypes.byref(n)) == INVALID and "values" in said(lib)
    assert lib.fl_mx4_workspace_bytes(1, 1, 1, 1, BF16, None) == INVALID
    need = size(4096, 4096, 4096, True, torch.bfloat16)
    if need:
        big = dict(M=4096, N=4096, K=4096, As=None)
        assert linear(lib, **big, ws=None, wb=0) == INVALID and "workspace of 0 bytes" in said(lib)
        assert linear(lib, **big, wb=need - 1) == INVALID and f"{need} needed" in said(lib)
        assert linear(lib, **big, ws=P[8] + 4) == INVALID and "not aligned" in said(lib)
        assert linear(lib, **big, ws=P[7]) == INVALID and "overlaps" in said(lib)


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("values", [0, 1])
def test_the_longest_rows(lib, dt, values):
    """The same of every type, codes or values."""
    n = ctypes.c_size_t()
    assert lib.fl_mx4_workspace_bytes(8, 32, 2 ** 22 - 1, values, dt, ctypes.byref(n)) == OK
    assert lib.fl_mx4_workspace_bytes(8, 32, 2 ** 22, values, dt, ctypes.byref(n)) == UNSUPPORTED and "2^22" in said(lib)
    assert linear(lib, K=2 ** 22, dt=dt, **({} if values == 0 else dict(As=None))) == UNSUPPORTED


def test_the_definition():
    """Ties to the even code, saturation, the scale's exponent, the ends."""
    x = torch.zeros(4, 32)
    x[0, :10] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -0.25, -5.0])
    x[1, :3] = torch.tensor([4.0, 0.26, -0.24])
    x[2, 0], x[2, 1] = 2.0 ** -126, 2.0 ** -149
    x[3, 0] = float("inf")
    codes, scales = quantize64(x)
    assert scales[:, 0].tolist() == [127, 127, 0, 255]
    v = values64(codes, scales, 32)
    assert v[0, :10].tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, -0.0, -4.0]
    assert v[1, :3].tolist() == [4.0, 0.5, -0.0] and v[2, 0] == 2.0 ** -126
    assert torch.isnan(v[3]).all() and (codes[3] == 0).all()
