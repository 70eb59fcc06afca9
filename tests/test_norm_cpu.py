"""Refusals and degenerate sizes of the layer norm C ABI, without a GPU:
validation runs before any HIP call, and the fake pointers are never read."""
import ctypes
import os
import re

import pytest
import torch

from activation_epilogue_amd import norm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, F16, BF16 = 0, 1, 2
P = [0x100000000 * (i + 1) for i in range(12)]  # far apart, aligned


@pytest.fixture(scope="module")
def lib():
    return norm._lib()


def forward(lib, X=P[0], w=P[1], b=P[2], Y=P[3], mean=P[4], rstd=P[5], M=8, H=64, eps=1e-5, dt=BF16):
    return lib.fl_layer_norm(X, w, b, Y, mean, rstd, M, H, eps, dt, None)


def backward(lib, dY=P[0], X=P[1], w=P[2], mean=P[3], rstd=P[4], R=P[5], dX=P[6], dw=P[7], db=P[8], M=8, H=64, dt=BF16,
             ws=P[9], wb=1 << 20):
    return lib.fl_layer_norm_bwd(dY, X, w, mean, rstd, R, dX, dw, db, M, H, dt, ws, wb, None)


def test_every_export_is_declared(lib):
    text = open(os.path.join(ROOT, "include", "fused_norm.h"), encoding="utf-8").read()
    assert set(re.findall(r"\b(fl_\w+)\s*\(", text)) - {"fl_norm_last_error"} <= set(norm.NORM_EXPORTS)
    for name in norm.NORM_EXPORTS:
        assert name in text and hasattr(lib, name)


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("kw,status,text", [
    (dict(dt=7), INVALID, "unknown dtype 7"),
    (dict(M=-1), INVALID, "negative size"),
    (dict(H=2 ** 31), UNSUPPORTED, "2^31-1"),
    (dict(X=None), INVALID, "X is NULL"),
    (dict(X=P[0] + 1), INVALID, "X (0x100000001) is not aligned to 2 bytes"),
    (dict(w=P[1] + 1), INVALID, "weight"),
    (dict(mean=P[10] + 2), INVALID, "mean"),
])
def test_refused_of_both(lib, call, kw, status, text):
    assert call(lib, **kw) == status and text in lib.fl_norm_last_error().decode()


@pytest.mark.parametrize("kw,text", [
    (dict(Y=None), "Y is NULL"),
    (dict(Y=P[0] + 2), "Y overlaps X"),
    (dict(Y=P[1]), "Y overlaps weight"),
    (dict(mean=P[0]), "mean overlaps X"),
    (dict(mean=P[5] + 4), "mean overlaps rstd"),
    (dict(eps=-1e-5), "eps"),
    (dict(eps=float("nan")), "eps"),
    (dict(eps=float("inf")), "eps"),
])
def test_refused_forward(lib, kw, text):
    assert forward(lib, **kw) == INVALID and text in lib.fl_norm_last_error().decode()


@pytest.mark.parametrize("kw,text", [
    (dict(dY=None), "dY is NULL"),
    (dict(mean=None), "mean is NULL"),
    (dict(rstd=None), "rstd is NULL"),
    (dict(dX=None), "dX is NULL"),
    (dict(dX=P[1] + 4), "dX overlaps X"),
    (dict(dX=P[3]), "dX overlaps mean"),
    (dict(dw=P[8]), "dweight overlaps dbias"),
    (dict(dw=P[2]), "dweight overlaps weight"),
    (dict(R=P[6] + 2), "dX overlaps R"),
    (dict(dY=P[6], X=P[6] + 2), "dX overlaps X"),
    (dict(M=600, ws=None), "workspace of 0 bytes"),
    (dict(M=600, wb=16), "workspace of 16 bytes"),
    (dict(M=600, ws=P[9] + 8), "not aligned to 16"),
    (dict(M=600, ws=P[6]), "overlaps"),
])
def test_refused_backward(lib, kw, text):
    assert backward(lib, **kw) == INVALID and text in lib.fl_norm_last_error().decode()


def test_nothing_to_do(lib):
    assert forward(lib, M=0, X=None, Y=None, mean=None, rstd=None) == OK and lib.fl_norm_last_error() == b""
    assert forward(lib, H=0, X=None, Y=None) == OK
    assert backward(lib, H=0, dY=None, X=None, dX=None, mean=None, rstd=None, R=None, ws=None, wb=0) == OK
    assert backward(lib, M=0, dY=None, X=None, dX=None, mean=None, rstd=None, R=None, dw=None, db=None, ws=None,
                    wb=0) == OK


def test_workspace_sizes(lib):
    size = norm.layer_norm_bwd_workspace_bytes
    assert size(0, 100, torch.float32) == size(100, 0, torch.float32) == size(1, 4096, torch.bfloat16) == 0
    for M, H in ((600, 64), (16384, 4096), (300, 16384)):
        n = size(M, H, torch.bfloat16)
        assert n > 0 and n % (8 * H) == 0 and n <= 512 * 8 * H
    assert size(1, 40001, torch.bfloat16) == 8  # the two sums of a row too long for registers
    assert lib.fl_layer_norm_bwd_workspace_bytes(8, 8, BF16, None) == INVALID
    assert lib.fl_layer_norm_bwd_workspace_bytes(8, 8, 9, ctypes.byref(ctypes.c_size_t())) == INVALID
