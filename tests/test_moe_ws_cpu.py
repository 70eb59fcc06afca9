"""Refusals of the workspaces of the experts' products, without a GPU:
validation runs before any HIP call, and the fake pointers are never read."""
import ctypes

import pytest
import torch

import activation_epilogue_amd as fl
from activation_epilogue_amd import moe

OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16 = 0, 2
P = [0x100000000 * (i + 1) for i in range(8)]


@pytest.fixture(scope="module")
def lib():
    return moe._lib()


def grad(lib, A=P[0], G=P[1], offsets=P[2], dW=P[3], dbias=P[4], S=16, N=32, K=64, E=4, dt=BF16, dw=BF16, ws=None, wb=0):
    return lib.fl_grouped_weight_grad_ws(A, G, offsets, dW, dbias, S, N, K, E, dt, dw, ws, wb, None)


def linear(lib, ws=None, wb=0):
    """One token through an expert of 4096 x 64: parts of K, so a workspace."""
    return lib.fl_grouped_linear(P[0], None, P[1], P[2], None, None, P[3], None, 1, 1, 64, 4096, 1, 0, BF16, ws, wb, None)


def test_workspace_sizes(lib):
    assert moe.grouped_grad_workspace_bytes(16, 32, 64, 4, torch.bfloat16) == 0
    assert moe.grouped_grad_workspace_bytes(0, 0, 0, 1, torch.bfloat16) == 0
    n = moe.grouped_grad_workspace_bytes(40000, 100, 100, 2, torch.bfloat16)
    assert n > 0 and n % (2 * 100 * 100 * 4) == 0
    assert moe.grouped_workspace_bytes(1, 64, 4096, 1, torch.bfloat16) % (64 * 4) == 0
    with pytest.raises(fl.FusedLinearError, match="E \\(0\\)"):
        moe.grouped_grad_workspace_bytes(8, 8, 8, 0, torch.bfloat16)
    assert lib.fl_grouped_grad_workspace_bytes(8, 8, 8, 1, BF16, None) == INVALID


def test_refusals(lib):
    def message():
        return lib.fl_moe_last_error().decode()
    need = moe.grouped_grad_workspace_bytes(40000, 100, 100, 2, torch.bfloat16)
    long = dict(S=40000, N=100, K=100, E=2)
    assert grad(lib, **long, ws=P[6], wb=need - 1) == INVALID and f"{need} needed" in message()
    assert grad(lib, **long, ws=P[6] + 8, wb=need) == INVALID and "not aligned" in message()
    assert grad(lib, **long, ws=P[3], wb=need) == INVALID and "overlaps" in message()
    assert grad(lib, G=None) == INVALID and "G is NULL" in message()
    assert grad(lib, N=2 ** 21, dw=F32) == UNSUPPORTED and "N too large" in message()
    assert grad(lib, N=0) == OK and message() == ""
    need = moe.grouped_workspace_bytes(1, 64, 4096, 1, torch.bfloat16)
    assert need > 0
    assert linear(lib) == INVALID and "workspace of 0 bytes" in message()
    assert linear(lib, ws=P[6], wb=need - 4) == INVALID and "needed" in message()
    assert linear(lib, ws=P[6] + 4, wb=need) == INVALID and "not aligned" in message()
    assert linear(lib, ws=P[2] + 64, wb=need) == INVALID and "overlaps" in message()
