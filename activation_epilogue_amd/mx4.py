"""Microscaled 4-bit floating point (C ABI in ``include/fused_mx4.h``).

Binding in the manner of the package: it checks shapes, dtypes and devices,
takes device pointers and the current HIP stream from PyTorch and calls the
library; outputs are allocated with torch where they are not given.

  Mx4(codes, scales, K)                         rows of K values as 4-bit codes and a scale for every 32 of them
  quantize_mx4(X, transposed=False, out=None)   -> Mx4 of X's rows (of its columns)
  dequantize_mx4(q, dtype, out=None)            -> the values (rows,K)
  fused_linear_mx4(A, B, bias=None, Y=None, act="relu", ...) -> act(A @ B + bias [+ R]), A a matrix or an Mx4
  mx4_plan(M, N, K, values, dtype)              -> Mx4Plan, the kernels that such a call takes
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from . import ACTS, FusedLinearError, load_library
from .moe import _bytes, _code, _matrix, _On, _out, _ptr

MX4_EXPORTS = ("fl_quantize_mx4", "fl_dequantize_mx4", "fl_fused_linear_mx4", "fl_mx4_workspace_bytes",
               "fl_mx4_linear_plan", "fl_mx4_last_error")


class Mx4(NamedTuple):
    """Rows of K values in microscaled 4-bit floating point, on the device."""
    codes: torch.Tensor   # (rows, 16 * ceil(K/32)) uint8, two codes to a byte
    scales: torch.Tensor  # (rows, ceil(K/32)) uint8, E8M0
    K: int                # values of a row


class Mx4Plan(ctypes.Structure):
    """Mirror of fl_mx4_plan."""
    _fields_ = [("kernel", ctypes.c_int32), ("rows", ctypes.c_int32), ("columns", ctypes.c_int32),
                ("waves", ctypes.c_int32), ("quantize", ctypes.c_int32), ("parts", ctypes.c_int32),
                ("first_columns", ctypes.c_int64), ("second_rows", ctypes.c_int32),
                ("second_columns", ctypes.c_int32), ("second_waves", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_mx4 = None


def _lib():
    """libfused_linear.so with this module's argument types set (once)."""
    global _mx4
    if _mx4 is None:
        lib = load_library()
        vp, i64, i32, c_int, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_size_t
        lib.fl_quantize_mx4.argtypes = [vp, vp, vp, i64, i64, i32, c_int, vp]
        lib.fl_dequantize_mx4.argtypes = [vp, vp, vp, i64, i64, c_int, vp]
        lib.fl_fused_linear_mx4.argtypes = [vp] * 8 + [i64] * 3 + [c_int, c_int, vp, sz, vp]
        lib.fl_mx4_workspace_bytes.argtypes = [i64, i64, i64, i32, c_int, ctypes.POINTER(sz)]
        lib.fl_mx4_linear_plan.argtypes = [i64, i64, i64, i32, c_int, ctypes.POINTER(Mx4Plan)]
        for name in MX4_EXPORTS[:-1]:
            getattr(lib, name).restype = c_int
        lib.fl_mx4_last_error.restype = ctypes.c_char_p
        _mx4 = lib
    return _mx4


def _ok(status):
    if status != 0:
        raise FusedLinearError(status, _lib().fl_mx4_last_error().decode())


def _rows(q, name, like=None):
    """(rows, K, pointers of codes and scales) of an Mx4 whose parts fit
    together, on like's device."""
    codes, K = q.codes, int(q.K)
    rows = _matrix(codes, f"{name}.codes")[0]
    if K < 0:
        raise ValueError(f"{name}.K is negative")
    blocks = (K + 31) // 32
    return (rows, K, _ptr(codes, f"{name}.codes", torch.uint8, (rows, 16 * blocks), like),
            _ptr(q.scales, f"{name}.scales", torch.uint8, (rows, blocks), codes))


def quantize_mx4(X, transposed=False, out=None, *, stream=None):
    """The rows of X (rows,K) in 4 bits (fl_quantize_mx4); transposed=True: the
    columns of X (K,rows), which makes a weight of fused_linear the B of
    fused_linear_mx4.  `out`: an Mx4 to overwrite."""
    rows, K = _matrix(X, "X")
    if transposed:
        rows, K = K, rows
    code = _code(X.dtype)
    blocks = (K + 31) // 32
    with _On(X, stream) as st:
        if out is not None and out.K != K:
            raise ValueError(f"out.K is {out.K}, expected {K}")
        q = Mx4(_out(None if out is None else out.codes, "out.codes", (rows, 16 * blocks), torch.uint8, X),
                _out(None if out is None else out.scales, "out.scales", (rows, blocks), torch.uint8, X), K)
        _ok(_lib().fl_quantize_mx4(_ptr(X, "X"), q.codes.data_ptr() or None, q.scales.data_ptr() or None, rows, K,
                                   1 if transposed else 0, code, st))
    return q


def dequantize_mx4(q, dtype=torch.bfloat16, out=None, *, stream=None):
    """The values of q (rows,K) in dtype (fl_dequantize_mx4)."""
    rows, K, codes, scales = _rows(q, "q")
    code = _code(dtype)
    with _On(q.codes, stream) as st:
        out = _out(out, "out", (rows, K), dtype, q.codes)
        _ok(_lib().fl_dequantize_mx4(codes, scales, out.data_ptr() or None, rows, K, code, st))
    return out


@functools.lru_cache(maxsize=1024)
def mx4_workspace_bytes(M, N, K, values, dtype):
    """Bytes of workspace fl_fused_linear_mx4 needs; values: A is a matrix."""
    n = ctypes.c_size_t()
    _ok(_lib().fl_mx4_workspace_bytes(M, N, K, 1 if values else 0,
                                      _code(dtype) if not isinstance(dtype, int) else dtype, ctypes.byref(n)))
    return n.value


def mx4_plan(M, N, K, values, dtype):
    """How fused_linear_mx4 runs at these sizes (fl_mx4_linear_plan), as an Mx4Plan; values: A is a matrix."""
    plan = Mx4Plan()
    _ok(_lib().fl_mx4_linear_plan(M, N, K, 1 if values else 0, _code(dtype), ctypes.byref(plan)))
    return plan


def fused_linear_mx4(A, B, bias=None, Y=None, act="relu", out=None, *, R=None, dtype=None, stream=None,
                     workspace=None):
    """out = act(A @ B + bias [+ R]) with B, an Mx4 of N rows of K, in 4 bits
    (fl_fused_linear_mx4).  A: an Mx4 of M rows, or a matrix (M,K) that is
    quantised on its way in.  bias (N,), Y (M,N) for act="glu", R (M,N) and out
    (M,N) are in dtype, which is A's where A is a matrix (bfloat16 else, unless
    given).  out may be Y or R.  workspace: a device tensor of
    mx4_workspace_bytes(M, N, K, A is a matrix, dtype) bytes (allocated where it
    is needed and not given)."""
    values = isinstance(A, torch.Tensor)
    if values:
        M, AK = _matrix(A, "A")
        dtype = dtype or A.dtype
        if dtype != A.dtype:
            raise TypeError(f"A has dtype {A.dtype}, expected {dtype}")
        first, a_scales = A, None
        a = _ptr(A, "A")
    else:
        M, AK, a, a_scales = _rows(A, "A")
        dtype = dtype or torch.bfloat16
        first = A.codes
    N, K, b, b_scales = _rows(B, "B", first)
    if AK != K:
        raise ValueError(f"A has rows of {AK} values and B of {K}")
    code = _code(dtype)
    need = mx4_workspace_bytes(M, N, K, values, code)
    with _On(first, stream) as st:
        out = _out(out, "out", (M, N), dtype, first)
        if need and workspace is None:
            workspace = first.new_empty(need, dtype=torch.uint8)
        _ok(_lib().fl_fused_linear_mx4(
            a, a_scales, b, b_scales, _ptr(bias, "bias", dtype, (N,), first), _ptr(Y, "Y", dtype, (M, N), first),
            _ptr(R, "R", dtype, (M, N), first), out.data_ptr() or None, M, N, K, ACTS[act], code,
            _ptr(workspace, "workspace", None, None, first), _bytes(workspace), st))
    return out
