"""Which kernels the 4-bit linear layer takes: the sizes of the GPU tests still reach each, and no size
takes one that they do not reach.  Without a GPU: the plan is the host's."""
import ctypes
import random

import pytest
import torch

import activation_epilogue_amd as fl
from activation_epilogue_amd import mx4
from mx4_kernels import KERNELS, depth, plan_of

DTYPES = (torch.float32, torch.float16, torch.bfloat16)


@pytest.mark.parametrize("name", KERNELS)
def test_sizes_reach_their_kernel(name):
    k = KERNELS[name]
    assert k.deep in k.sweep
    for blocks in k.sweep:
        for dtype in DTYPES:
            for values in (False, True):
                p = fl.mx4_plan(k.M, k.N, depth(blocks), values, dtype)
                assert plan_of(p) == k.plan, (blocks, values)
                assert p.quantize == (0 if not values else 2 if k.inside else 1), blocks
                sums = p.parts * k.M * k.N * 4 if p.parts > 1 else 0
                codes = k.M * blocks * 16 + (k.M * blocks + 15) // 16 * 16 if p.quantize == 1 else 0
                assert fl.mx4_workspace_bytes(k.M, k.N, depth(blocks), values, dtype) == sums + codes


def test_every_kernel_is_reached():
    """Of random sizes up to 8192 rows, 24576 columns and values."""
    known = {(k.plan, k.inside) for k in KERNELS.values()}
    known |= {(plan, False) for plan, inside in known if inside}  # the same with codes
    rng = random.Random(5)
    met = set()
    for _ in range(20000):
        M, N, K = (int(2 ** rng.uniform(a, b)) for a, b in ((0, 13), (0, 14.6), (0, 14.6)))
        for values in (False, True):
            p = fl.mx4_plan(M, N, K, values, torch.bfloat16)
            met.add((plan_of(p), p.quantize == 2))
            assert (plan_of(p), p.quantize == 2) in known, (M, N, K, values)
    assert len({plan for plan, _ in met}) >= 11  # and those of the table are no rarities but one


def test_nothing_to_multiply():
    for M, N, K in ((3, 5, 0), (0, 5, 64), (3, 0, 64)):
        p = fl.mx4_plan(M, N, K, True, torch.float32)
        assert p.kernel == 0 and p.parts == 1 and p.quantize == 0


def test_refused():
    lib, plan = mx4._lib(), mx4.Mx4Plan()
    call = lambda M=8, N=8, K=64, values=0, dt=2, to=ctypes.byref(plan): lib.fl_mx4_linear_plan(  # noqa: E731
        M, N, K, values, dt, to)
    assert call() == 0
    for kw, text in ((dict(M=-1), "negative"), (dict(dt=9), "dtype"), (dict(values=2), "values"), (dict(to=None), "plan is NULL"),
                     (dict(K=2 ** 22), "2^22"), (dict(N=2 ** 23), "N too large")):
        assert call(**kw) != 0 and text in lib.fl_mx4_last_error().decode()
