"""Layer norm (C ABI in ``include/fused_norm.h``).

Binding in the manner of the package: it checks shapes, dtypes and devices,
takes device pointers and the current HIP stream from PyTorch and calls the
library; outputs are allocated with torch where they are not given.

  layer_norm(X, weight=None, bias=None, eps=1e-5, ...)  -> out (M,H), or (out, mean, rstd) with stats=True
  layer_norm_bwd(dout, X, mean, rstd, weight=None, R=None, ...) -> (dX, dweight, dbias)
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import FusedLinearError, load_library
from .moe import _bytes, _code, _matrix, _On, _out, _ptr

NORM_EXPORTS = ("fl_layer_norm", "fl_layer_norm_bwd", "fl_layer_norm_bwd_workspace_bytes", "fl_norm_last_error")

_norm = None


def _lib():
    """libfused_linear.so with this module's argument types set (once)."""
    global _norm
    if _norm is None:
        lib = load_library()
        vp, i64, c_int, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        lib.fl_layer_norm.argtypes = [vp] * 6 + [i64, i64, ctypes.c_float, c_int, vp]
        lib.fl_layer_norm_bwd.argtypes = [vp] * 9 + [i64, i64, c_int, vp, sz, vp]
        lib.fl_layer_norm_bwd_workspace_bytes.argtypes = [i64, i64, c_int, ctypes.POINTER(sz)]
        for name in NORM_EXPORTS[:-1]:
            getattr(lib, name).restype = c_int
        lib.fl_norm_last_error.restype = ctypes.c_char_p
        _norm = lib
    return _norm


def _ok(status):
    if status != 0:
        raise FusedLinearError(status, _lib().fl_norm_last_error().decode())


def layer_norm(X, weight=None, bias=None, eps=1e-5, out=None, stats=False, mean=None, rstd=None, *, stream=None):
    """The norm of every row of X (M,H), times weight (H,) plus bias (H,)
    (fl_layer_norm).  stats=True also returns what the backward pass needs, as
    (out, mean (M,) fp32, rstd (M,) fp32), in the tensors mean and rstd where
    they are given.  out may be X."""
    M, H = _matrix(X, "X")
    code = _code(X.dtype)
    with _On(X, stream) as st:
        out = torch.empty_like(X) if out is None else _out(out, "out", (M, H), X.dtype, X)
        if stats:
            mean = _out(mean, "mean", (M,), torch.float32, X)
            rstd = _out(rstd, "rstd", (M,), torch.float32, X)
        elif mean is not None or rstd is not None:
            raise ValueError("mean and rstd are written with stats=True only")
        _ok(_lib().fl_layer_norm(_ptr(X, "X"), _ptr(weight, "weight", X.dtype, (H,), X),
                                 _ptr(bias, "bias", X.dtype, (H,), X), out.data_ptr() or None,
                                 mean.data_ptr() or None if stats else None,
                                 rstd.data_ptr() or None if stats else None, M, H, eps, code, st))
    return (out, mean, rstd) if stats else out


@functools.lru_cache(maxsize=1024)
def layer_norm_bwd_workspace_bytes(M, H, dtype):
    """Bytes of workspace fl_layer_norm_bwd needs for the weight's or the bias's gradient (for neither: 8 M of
    rows above 16384, else none)."""
    n = ctypes.c_size_t()
    _ok(_lib().fl_layer_norm_bwd_workspace_bytes(M, H, _code(dtype) if not isinstance(dtype, int) else dtype,
                                                 ctypes.byref(n)))
    return n.value


def layer_norm_bwd(dout, X, mean, rstd, weight=None, R=None, dX=None, dweight=True, dbias=True, *, stream=None,
                   workspace=None):
    """The gradients of layer_norm (fl_layer_norm_bwd) from dout (M,H), X and
    the mean and rstd that layer_norm(stats=True) gave: (dX, dweight (H,) fp32,
    dbias (H,) fp32).  R (M,H) is added to dX, the gradient of a path around the
    norm.  dweight/dbias: True allocates the result, a tensor is overwritten,
    None/False skips it.  dX may be dout, X or R.  workspace: a device tensor of
    layer_norm_bwd_workspace_bytes(M, H, dtype) bytes (allocated where it is
    needed and not given; with neither gradient 8 M bytes for H above 16384, else none)."""
    M, H = _matrix(dout, "dout")
    dt = dout.dtype
    code = _code(dt)
    with _On(dout, stream) as st:
        dX = torch.empty_like(dout) if dX is None else _out(dX, "dX", (M, H), dt, dout)
        sums = []
        for name, t in (("dweight", dweight), ("dbias", dbias)):
            sums.append(None if t is None or t is False else
                        _out(None if t is True else t, name, (H,), torch.float32, dout))
        if sums[0] is None and sums[1] is None:
            need = 8 * M if H > 16384 else 0
        else:
            need = layer_norm_bwd_workspace_bytes(M, H, code)
        if need and workspace is None:
            workspace = dout.new_empty(need, dtype=torch.uint8)
        _ok(_lib().fl_layer_norm_bwd(
            _ptr(dout, "dout"), _ptr(X, "X", dt, (M, H), dout), _ptr(weight, "weight", dt, (H,), dout),
            _ptr(mean, "mean", torch.float32, (M,), dout), _ptr(rstd, "rstd", torch.float32, (M,), dout),
            _ptr(R, "R", dt, (M, H), dout), dX.data_ptr() or None,
            *(None if t is None else t.data_ptr() or None for t in sums), M, H, code,
            _ptr(workspace, "workspace", None, None, dout), _bytes(workspace), st))
    return dX, *sums
