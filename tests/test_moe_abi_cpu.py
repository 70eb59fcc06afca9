"""Refusals and degenerate sizes of the routed-experts C ABI, without a GPU:
validation runs before any HIP call, and the fake pointers are never read."""
import ctypes
import os
import re

import pytest
import torch

import activation_epilogue_amd as fl
from activation_epilogue_amd import moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, F16, BF16 = 0, 1, 2
NONE, RELU, GELU, GLU = 0, 1, 2, 3
P = [0x100000000 * (i + 1) for i in range(12)]  # far apart, aligned


@pytest.fixture(scope="module")
def lib():
    return moe._lib()


def _opt(**kw):
    return moe.RouteOptions(**kw)


def route(lib, logits=P[0], bias=None, experts=P[1], weights=P[2], T=8, E=64, k=6, dt=BF16, opt=None):
    return lib.fl_moe_route(logits, bias, experts, weights, T, E, k, dt, ctypes.byref(opt) if opt else None, None)


def route_bwd(lib, logits=P[0], experts=P[1], dweights=P[2], dlogits=P[3], T=8, E=64, k=6, dt=BF16, opt=None):
    return lib.fl_moe_route_bwd(logits, experts, dweights, dlogits, T, E, k, dt, ctypes.byref(opt) if opt else None,
                                None)


def plan(lib, experts=P[0], offsets=P[1], token=P[2], row=P[3], T=8, k=2, E=4, ws=None, wb=0):
    return lib.fl_moe_plan(experts, offsets, token, row, T, k, E, ws, wb, None)


def gather(lib, X=P[0], index=P[1], rows=P[2], T=8, S=16, H=32, dt=BF16):
    return lib.fl_moe_gather(X, index, rows, T, S, H, dt, None)


def combine(lib, rows=P[0], slot=P[1], weights=P[2], R=None, out=P[3], T=8, k=2, S=16, H=32, dt=BF16):
    return lib.fl_moe_combine(rows, slot, weights, R, out, T, k, S, H, dt, None)


def combine_bwd(lib, dout=P[0], rows=P[1], slot=P[2], weights=P[3], drows=P[4], dweights=P[5], T=8, k=2, S=16, H=32,
                dt=BF16):
    return lib.fl_moe_combine_bwd(dout, rows, slot, weights, drows, dweights, T, k, S, H, dt, None)


def linear(lib, A=P[0], index=None, offsets=P[1], B=P[2], bias=P[3], Y=None, out=P[4], pre=None, A_rows=16, S=16, N=32,
           K=64, E=4, act=RELU, dt=BF16, ws=None, wb=0):
    return lib.fl_grouped_linear(A, index, offsets, B, bias, Y, out, pre, A_rows, S, N, K, E, act, dt, ws, wb, None)


def linear_bwd(lib, G=P[0], offsets=P[1], W=P[2], X=P[3], Y=None, dX=P[4], dY=None, S=16, N=32, K=64, E=4, act=RELU,
               dt=BF16):
    return lib.fl_grouped_linear_bwd(G, offsets, W, X, Y, dX, dY, S, N, K, E, act, dt, None)


def weight_grad(lib, A=P[0], G=P[1], offsets=P[2], dW=P[3], dbias=P[4], S=16, N=32, K=64, E=4, dt=BF16, dw=BF16):
    return lib.fl_grouped_weight_grad(A, G, offsets, dW, dbias, S, N, K, E, dt, dw, None)


def test_header_and_exports(lib):
    text = open(os.path.join(ROOT, "include", "fused_moe.h")).read()
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    declared = set(re.findall(r"\b(fl_[a-z0-9_]+)\s*\(", text))
    assert declared == set(moe.MOE_EXPORTS)
    for name in declared:
        assert hasattr(lib, name)


@pytest.mark.parametrize("call,kwargs,status,msg", [
    (route, dict(logits=None), INVALID, "logits is NULL"),
    (route, dict(experts=None), INVALID, "experts is NULL"),
    (route, dict(weights=None), INVALID, "weights is NULL"),
    (route, dict(dt=7), INVALID, "unknown dtype"),
    (route, dict(T=-1), INVALID, "negative size"),
    (route, dict(T=2 ** 31), UNSUPPORTED, "above 2^31-1"),
    (route, dict(T=2 ** 30, k=6), UNSUPPORTED, "slots"),
    (route, dict(E=0), UNSUPPORTED, "E (0)"),
    (route, dict(E=1025), UNSUPPORTED, "E (1025)"),
    (route, dict(k=0), INVALID, "k (0)"),
    (route, dict(k=65), INVALID, "k (65)"),
    (route, dict(k=65, E=128), UNSUPPORTED, "k (65) above 64"),
    (route, dict(logits=P[0] + 1), INVALID, "not aligned"),
    (route, dict(bias=P[5] + 2), INVALID, "not aligned"),
    (route, dict(weights=P[1] + 16), INVALID, "overlaps"),
    (route, dict(experts=P[0] + 64), INVALID, "overlaps logits"),
    (route, dict(opt=_opt(score=2)), INVALID, "unknown score"),
    (route, dict(opt=_opt(raw=2)), INVALID, "raw"),
    (route, dict(opt=_opt(scale=float("inf"))), INVALID, "scale"),
    (route, dict(opt=_opt(scale=float("nan"))), INVALID, "scale"),
    (route, dict(opt=_opt(groups=5)), INVALID, "must divide"),
    (route, dict(opt=_opt(groups=-1)), INVALID, "must divide"),
    (route, dict(E=128, opt=_opt(groups=128)), INVALID, "at most 64"),
    (route, dict(opt=_opt(groups=8, top_groups=9)), INVALID, "top_groups"),
    (route, dict(opt=_opt(groups=8, group_top=3)), INVALID, "group_top"),
    (route_bwd, dict(dlogits=None), INVALID, "dlogits is NULL"),
    (route_bwd, dict(dweights=None), INVALID, "dweights is NULL"),
    (route_bwd, dict(dlogits=P[0] + 2), INVALID, "dlogits overlaps logits"),
    (route_bwd, dict(dlogits=P[2]), INVALID, "dlogits overlaps dweights"),
    (plan, dict(experts=None), INVALID, "experts is NULL"),
    (plan, dict(offsets=None), INVALID, "offsets is NULL"),
    (plan, dict(row=None), INVALID, "row_of_slot is NULL"),
    (plan, dict(token=P[0]), INVALID, "token_of_row overlaps experts"),
    (plan, dict(E=0), UNSUPPORTED, "E (0)"),
    (plan, dict(E=1025), UNSUPPORTED, "E (1025)"),
    (plan, dict(T=2 ** 30, k=4), UNSUPPORTED, "slots"),
    (plan, dict(k=-1), INVALID, "negative size"),
    (plan, dict(T=10000), INVALID, "workspace of 0 bytes"),
    (plan, dict(T=10000, ws=P[6], wb=3), INVALID, "workspace of 3 bytes"),
    (plan, dict(T=10000, ws=P[1], wb=1 << 20), INVALID, "overlaps"),
    (gather, dict(X=None), INVALID, "X is NULL"),
    (gather, dict(index=P[1] + 1), INVALID, "not aligned"),
    (gather, dict(rows=P[0]), INVALID, "rows overlaps X"),
    (gather, dict(dt=-1), INVALID, "unknown dtype"),
    (combine, dict(rows=None), INVALID, "rows is NULL"),
    (combine, dict(out=P[0]), INVALID, "out overlaps rows"),
    (combine, dict(R=P[3] + 2), INVALID, "out overlaps R"),
    (combine, dict(k=-3), INVALID, "negative size"),
    (combine_bwd, dict(drows=None, dweights=None), INVALID, "both NULL"),
    (combine_bwd, dict(rows=None), INVALID, "rows is NULL"),
    (combine_bwd, dict(drows=P[0]), INVALID, "drows overlaps dout"),
    (combine_bwd, dict(drows=P[1] + 2), INVALID, "drows overlaps rows"),
    (linear, dict(A=None), INVALID, "A is NULL"),
    (linear, dict(B=None), INVALID, "B is NULL"),
    (linear, dict(out=None), INVALID, "out is NULL"),
    (linear, dict(offsets=None), INVALID, "offsets is NULL"),
    (linear, dict(act=GLU), INVALID, "the gate needs Y"),
    (linear, dict(Y=P[6]), INVALID, "only used by the gate"),
    (linear, dict(act=9), INVALID, "unknown activation"),
    (linear, dict(A_rows=15), INVALID, "A has 15 rows"),
    (linear, dict(E=0), UNSUPPORTED, "E (0)"),
    (linear, dict(E=2000), UNSUPPORTED, "E (2000)"),
    (linear, dict(S=-1), INVALID, "negative size"),
    (linear, dict(K=2 ** 22), UNSUPPORTED, "too large"),
    (linear, dict(K=32768, N=32768), UNSUPPORTED, "B too large"),
    (linear, dict(index=P[6], A_rows=2 ** 25), UNSUPPORTED, "A too large for an index"),
    (linear, dict(out=P[0]), INVALID, "out overlaps A"),
    (linear, dict(pre=P[4] + 64), INVALID, "overlaps"),
    (linear, dict(act=GLU, Y=P[4] + 2), INVALID, "out overlaps Y"),
    (linear, dict(out=P[4] + 1), INVALID, "not aligned"),
    (linear, dict(dt=F32, A=P[0] + 2), INVALID, "not aligned"),
    (linear_bwd, dict(X=None), INVALID, "X is NULL"),
    (linear_bwd, dict(act=GLU, dY=P[6]), INVALID, "the gate needs Y"),
    (linear_bwd, dict(act=GLU, Y=P[5]), INVALID, "dY is NULL"),
    (linear_bwd, dict(dY=P[6]), INVALID, "only used by the gate"),
    (linear_bwd, dict(dX=P[0]), INVALID, "dX overlaps G"),
    (linear_bwd, dict(dX=P[3] + 2), INVALID, "dX overlaps X"),
    (weight_grad, dict(G=None), INVALID, "G is NULL"),
    (weight_grad, dict(dW=None), INVALID, "dW is NULL"),
    (weight_grad, dict(dw=F16), INVALID, "operands' dtype or fp32"),
    (weight_grad, dict(dW=P[0]), INVALID, "dW overlaps A"),
    (weight_grad, dict(dbias=P[3]), INVALID, "overlaps"),
])
def test_refusals(lib, call, kwargs, status, msg):
    assert call(lib, **kwargs) == status
    assert msg in lib.fl_moe_last_error().decode()


def test_nothing_to_do_returns_ok_without_a_launch(lib):
    assert route(lib, T=0, logits=None, experts=None, weights=None) == OK
    assert route_bwd(lib, T=0) == OK
    assert gather(lib, S=0) == OK and gather(lib, H=0) == OK
    assert combine(lib, T=0) == OK and combine(lib, H=0) == OK
    assert combine_bwd(lib, T=0) == OK and combine_bwd(lib, k=0) == OK
    assert linear(lib, S=0, A_rows=0, A=None, B=None, out=None) == OK and linear(lib, N=0) == OK
    assert linear_bwd(lib, S=0) == OK and linear_bwd(lib, N=0) == OK
    assert weight_grad(lib, N=0) == OK and weight_grad(lib, K=0, dbias=None) == OK
    assert lib.fl_moe_last_error() == b""


def test_workspace_sizes():
    assert moe.moe_plan_workspace_bytes(8, 2, 4) == 0
    assert moe.moe_plan_workspace_bytes(0, 0, 4) == 0
    assert moe.moe_plan_workspace_bytes(65536, 8, 256) >= 256 * 4 * 2
    with pytest.raises(fl.FusedLinearError, match="E \\(0\\)"):
        moe.moe_plan_workspace_bytes(8, 2, 0)
    with pytest.raises(fl.FusedLinearError, match="negative"):
        moe.grouped_workspace_bytes(-1, 8, 8, 4, torch.bfloat16)


def test_binding_refuses_before_the_library():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device"):
        fl.moe_route(x, 2)
    with pytest.raises(ValueError, match="score"):
        fl.moe_route(x, 2, score="tanh")
    with pytest.raises(ValueError, match="scale"):
        fl.moe_route(x, 2, scale=0.0)
    with pytest.raises(TypeError, match="dtype"):
        fl.moe_route(x.double(), 2)
    with pytest.raises(ValueError, match="matrix"):
        fl.moe_route(x[0], 2)
    with pytest.raises(ValueError, match="B must be"):
        fl.grouped_linear(x, torch.zeros(2, 7, 5), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="W must be"):
        fl.grouped_linear_bwd(x, torch.zeros(2, 8, 5), None, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(AttributeError):
        fl.moe_nothing
