"""The routed-experts operators (C ABI in ``include/fused_moe.h``).

Binding in the manner of the package: it checks shapes, dtypes and devices,
takes device pointers and the current HIP stream from PyTorch and calls the
library; outputs are allocated with torch where they are not given.

  moe_route(logits, k, bias=None, ...)     -> (weights (T,k) fp32, experts (T,k) int32)
  moe_route_bwd(logits, experts, dweights) -> dlogits (T,E)
  moe_plan(experts, E)                     -> Plan(offsets, token_of_row, row_of_slot)
  moe_gather(X, index)                     -> rows (S,H), rows[r] = X[index[r]]
  moe_combine(rows, row_of_slot, weights)  -> out (T,H), the weighted sum of every token's rows (+ R)
  moe_combine_bwd(dout, rows, row_of_slot, weights) -> (drows, dweights)
  grouped_linear(A, B, offsets, ...)       -> act(A[e] @ B[e] + bias[e]) of every expert's rows
  grouped_linear_bwd(G, W, X, offsets)     -> (dX, dY or None), dX = (G @ W[e]^T) * act'(X)
  grouped_weight_grad(A, G, offsets)       -> (dW (E,K,N), dbias (E,N) fp32)

The plan's arrays stay on the device: no call waits for the GPU.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from . import ACTS, FusedLinearError, _dev_ptr, _dtype_code, load_library

SCORES = {"softmax": 0, "sigmoid": 1}
_CODES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
MOE_EXPORTS = ("fl_moe_route", "fl_moe_route_bwd", "fl_moe_plan", "fl_moe_plan_workspace_bytes", "fl_moe_gather",
               "fl_moe_combine", "fl_moe_combine_bwd", "fl_grouped_linear", "fl_grouped_workspace_bytes",
               "fl_grouped_linear_bwd", "fl_grouped_weight_grad", "fl_grouped_weight_grad_ws",
               "fl_grouped_grad_workspace_bytes", "fl_moe_last_error")


class RouteOptions(ctypes.Structure):
    """Mirror of fl_route_options."""
    _fields_ = [("score", ctypes.c_int32), ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("raw", ctypes.c_int32), ("scale", ctypes.c_float)]


class Plan(NamedTuple):
    """What moe_plan makes of a choice of experts, int32 on the device."""
    offsets: torch.Tensor       # (E+1,) first row of every expert
    token_of_row: torch.Tensor  # (T*k,) token of every row, -1 past the last
    row_of_slot: torch.Tensor   # (T,k) row of every choice, -1 without an expert


_moe = None


def _lib():
    """libfused_linear.so with this module's argument types set (once)."""
    global _moe
    if _moe is None:
        lib = load_library()
        vp, i64, c_int, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        opt, psz = ctypes.POINTER(RouteOptions), ctypes.POINTER(ctypes.c_size_t)
        lib.fl_moe_route.argtypes = [vp, vp, vp, vp, i64, i64, i64, c_int, opt, vp]
        lib.fl_moe_route_bwd.argtypes = [vp, vp, vp, vp, i64, i64, i64, c_int, opt, vp]
        lib.fl_moe_plan.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, sz, vp]
        lib.fl_moe_plan_workspace_bytes.argtypes = [i64, i64, i64, psz]
        lib.fl_moe_gather.argtypes = [vp, vp, vp, i64, i64, i64, c_int, vp]
        lib.fl_moe_combine.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, c_int, vp]
        lib.fl_moe_combine_bwd.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, c_int, vp]
        lib.fl_grouped_linear.argtypes = [vp] * 8 + [i64] * 5 + [c_int, c_int, vp, sz, vp]
        lib.fl_grouped_workspace_bytes.argtypes = [i64, i64, i64, i64, c_int, psz]
        lib.fl_grouped_linear_bwd.argtypes = [vp] * 7 + [i64] * 4 + [c_int, c_int, vp]
        lib.fl_grouped_weight_grad.argtypes = [vp] * 5 + [i64] * 4 + [c_int, c_int, vp]
        lib.fl_grouped_weight_grad_ws.argtypes = [vp] * 5 + [i64] * 4 + [c_int, c_int, vp, sz, vp]
        lib.fl_grouped_grad_workspace_bytes.argtypes = [i64, i64, i64, i64, c_int, psz]
        for name in MOE_EXPORTS[:-1]:
            getattr(lib, name).restype = c_int
        lib.fl_moe_last_error.restype = ctypes.c_char_p
        _moe = lib
    return _moe


def _ok(status):
    if status != 0:
        raise FusedLinearError(status, _lib().fl_moe_last_error().decode())


class _On:
    """The stream a call runs on: the given one (of t's device), or the current
    one of t's device; that device and stream are current while the call allocates and
    launches, so its temporary and result tensors belong to that stream."""
    __slots__ = ("ctx", "index")

    def __init__(self, t, stream):
        if not t.is_cuda:
            raise ValueError("operands must be device tensors")
        self.ctx = None
        self.index = t.device.index
        if stream is not None:
            if stream.device != t.device:
                raise ValueError(f"stream is on {stream.device}, expected {t.device}")
            self.ctx = torch.cuda.stream(stream)
        elif self.index != torch.cuda.current_device():
            self.ctx = torch.cuda.device(self.index)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return torch._C._cuda_getCurrentRawStream(self.index)

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _out(t, name, shape, dtype, like):
    """`t` checked, or a new tensor where it is None."""
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    _ptr(t, name, dtype, shape, like)
    return t


def _ptr(t, name, dtype=None, shape=None, like=None):
    """The device pointer of a contiguous tensor of that dtype and shape on
    like's device (None for None and for nothing)."""
    if t is None:
        return None
    if (t.is_cuda and t.is_contiguous() and (dtype is None or t.dtype is dtype) and (shape is None or t.shape == shape)
            and (like is None or t.get_device() == like.get_device())):
        return t.data_ptr() or None
    _dev_ptr(t, name, dtype, shape)  # says what is wrong
    raise ValueError(f"{name} is on {t.device}, expected {like.device}")


def _code(dtype):
    code = _CODES.get(dtype)
    return _dtype_code(dtype) if code is None else code


_options = {}


def _route_options(*how):
    """The RouteOptions of (score, groups, top_groups, group_top, renorm,
    scale), by reference.  Kept for plain values only: a tensor among them would
    be found again by its identity, whatever it holds by then."""
    opt = _options.get(how)
    if opt is None:
        opt = _new_route_options(*how)
        if all(type(v) in (str, int, float, bool) for v in how):
            if len(_options) >= 64:
                _options.clear()
            _options[how] = opt
    return opt


def _new_route_options(score, groups, top_groups, group_top, renorm, scale):
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    opt = RouteOptions(SCORES[score], int(groups), int(top_groups), int(group_top), 0 if renorm else 1, float(scale))
    if opt.scale == 0.0:  # (the library's default)
        raise ValueError(f"scale must not be 0 in 32 bits, got {scale}")
    return ctypes.byref(opt)


def _bytes(t):
    return t.numel() * t.element_size() if t is not None else 0


def _matrix(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, got shape {tuple(t.shape)}")
    return t.shape


def moe_route(logits, k, bias=None, score="softmax", groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0,
              weights=None, experts=None, *, stream=None):
    """k experts for every token and their weights (fl_moe_route): logits
    (T,E); bias (E,) fp32 is added to the scores for the choice only.  Returns
    (weights (T,k) fp32, experts (T,k) int32), experts in falling order of
    their keys; -1 with weight 0 where no unmasked expert is left."""
    T, E = _matrix(logits, "logits")
    opt = _route_options(score, groups, top_groups, group_top, renorm, scale)
    code = _code(logits.dtype)
    with _On(logits, stream) as st:
        weights = _out(weights, "weights", (T, k), torch.float32, logits)
        experts = _out(experts, "experts", (T, k), torch.int32, logits)
        _ok(_lib().fl_moe_route(_ptr(logits, "logits"), _ptr(bias, "bias", torch.float32, (E,), logits),
                                experts.data_ptr() or None, weights.data_ptr() or None, T, E, k, code,
                                opt, st))
    return weights, experts


def moe_route_bwd(logits, experts, dweights, score="softmax", renorm=True, scale=1.0, dlogits=None, *, stream=None):
    """The gradient of the logits from that of the weights (fl_moe_route_bwd)."""
    T, E = _matrix(logits, "logits")
    k = _matrix(experts, "experts")[1]
    opt = _route_options(score, 1, 1, 1, renorm, scale)
    code = _code(logits.dtype)
    with _On(logits, stream) as st:
        dlogits = _out(dlogits, "dlogits", (T, E), logits.dtype, logits)
        _ok(_lib().fl_moe_route_bwd(_ptr(logits, "logits"), _ptr(experts, "experts", torch.int32, (T, k), logits),
                                    _ptr(dweights, "dweights", torch.float32, (T, k), logits),
                                    dlogits.data_ptr() or None, T, E, k, code, opt, st))
    return dlogits


@functools.lru_cache(maxsize=1024)
def moe_plan_workspace_bytes(T, k, E):
    """Bytes of workspace fl_moe_plan needs."""
    n = ctypes.c_size_t()
    _ok(_lib().fl_moe_plan_workspace_bytes(T, k, E, ctypes.byref(n)))
    return n.value


def moe_plan(experts, E, out=None, *, stream=None, workspace=None):
    """The slots of experts (T,k) int32 sorted by expert (fl_moe_plan): a Plan.
    Values outside [0,E) are slots without an expert.  `out`: a Plan to
    overwrite.  workspace: a device tensor of moe_plan_workspace_bytes(T, k, E)
    bytes (allocated where it is needed and not given)."""
    T, k = _matrix(experts, "experts")
    need = moe_plan_workspace_bytes(T, k, E)
    with _On(experts, stream) as st:
        o = out or (None, None, None)
        plan = Plan(_out(o[0], "offsets", (E + 1,), torch.int32, experts),
                    _out(o[1], "token_of_row", (T * k,), torch.int32, experts),
                    _out(o[2], "row_of_slot", (T, k), torch.int32, experts))
        if need and workspace is None:
            workspace = experts.new_empty(need, dtype=torch.uint8)
        _ok(_lib().fl_moe_plan(_ptr(experts, "experts", torch.int32), plan.offsets.data_ptr(),
                               plan.token_of_row.data_ptr() or None, plan.row_of_slot.data_ptr() or None, T, k, E,
                               _ptr(workspace, "workspace", None, None, experts),
                               _bytes(workspace), st))
    return plan


def moe_gather(X, index, rows=None, *, stream=None):
    """rows[r] = X[index[r]] (zeros where index[r] is outside X) (fl_moe_gather)."""
    T, H = _matrix(X, "X")
    S = index.numel()
    with _On(X, stream) as st:
        rows = _out(rows, "rows", (S, H), X.dtype, X)
        _ok(_lib().fl_moe_gather(_ptr(X, "X"), _ptr(index, "index", torch.int32, (S,), X), rows.data_ptr() or None, T,
                                 S, H, _code(X.dtype), st))
    return rows


def moe_combine(rows, row_of_slot, weights=None, R=None, out=None, *, stream=None):
    """out[t] = R[t] + sum_j weights[t,j] * rows[row_of_slot[t,j]] (fl_moe_combine);
    without weights all count 1, which is the gradient of moe_gather."""
    S, H = _matrix(rows, "rows")
    T, k = _matrix(row_of_slot, "row_of_slot")
    with _On(rows, stream) as st:
        out = _out(out, "out", (T, H), rows.dtype, rows)
        _ok(_lib().fl_moe_combine(_ptr(rows, "rows"), _ptr(row_of_slot, "row_of_slot", torch.int32, None, rows),
                                  _ptr(weights, "weights", torch.float32, (T, k), rows),
                                  _ptr(R, "R", rows.dtype, (T, H), rows), out.data_ptr() or None, T, k, S, H,
                                  _code(rows.dtype), st))
    return out


def moe_combine_bwd(dout, rows, row_of_slot, weights=None, drows=None, dweights=None, *, stream=None):
    """The gradients of moe_combine's rows and weights (fl_moe_combine_bwd).
    Rows that no slot points at keep what drows held (unset where it is
    allocated here).  drows=False or dweights=False leaves one of them out (None
    in its place); rows are read for dweights only."""
    T, H = _matrix(dout, "dout")
    S = _matrix(rows, "rows")[0]
    k = _matrix(row_of_slot, "row_of_slot")[1]
    with _On(dout, stream) as st:
        drows = None if drows is False else _out(drows, "drows", (S, H), dout.dtype, dout)
        dweights = None if dweights is False else _out(dweights, "dweights", (T, k), torch.float32, dout)
        _ok(_lib().fl_moe_combine_bwd(_ptr(dout, "dout"), _ptr(rows, "rows", dout.dtype, (S, H), dout),
                                      _ptr(row_of_slot, "row_of_slot", torch.int32, (T, k), dout),
                                      _ptr(weights, "weights", torch.float32, (T, k), dout),
                                      None if drows is None else drows.data_ptr() or None,
                                      None if dweights is None else dweights.data_ptr() or None, T, k, S, H,
                                      _code(dout.dtype), st))
    return drows, dweights


@functools.lru_cache(maxsize=1024)
def grouped_workspace_bytes(S, N, K, E, dtype):
    """Bytes of workspace fl_grouped_linear needs."""
    n = ctypes.c_size_t()
    _ok(_lib().fl_grouped_workspace_bytes(S, N, K, E, _code(dtype) if not isinstance(dtype, int) else dtype,
                                          ctypes.byref(n)))
    return n.value


@functools.lru_cache(maxsize=1024)
def grouped_grad_workspace_bytes(S, N, K, E, dtype):
    """Bytes of workspace fl_grouped_weight_grad_ws takes."""
    n = ctypes.c_size_t()
    _ok(_lib().fl_grouped_grad_workspace_bytes(S, N, K, E, _code(dtype) if not isinstance(dtype, int) else dtype,
                                               ctypes.byref(n)))
    return n.value


def grouped_linear(A, B, offsets, bias=None, Y=None, act="relu", out=None, *, index=None, pre=None, stream=None,
                   workspace=None):
    """out[r] = act(A[r] @ B[e] + bias[e]) for the rows offsets[e] <= r <
    offsets[e+1] of every expert e (fl_grouped_linear): A (S,K), or with index
    (S,) int32 a matrix whose row index[r] is row r; B (E,K,N); bias (E,N); Y
    (S,N) for act="glu".  Rows at and past offsets[E] keep what out held.
    pre=True also returns the pre-activation X = A @ B[e] + bias[e] (a tensor is
    overwritten with it): then the result is (out, X)."""
    A_rows, K = _matrix(A, "A")
    if B.dim() != 3 or B.shape[1] != K:
        raise ValueError(f"B must be (E,{K},N), got {tuple(B.shape)}")
    E, _, N = B.shape
    S = A_rows if index is None else index.numel()
    dt = A.dtype
    code = _code(dt)
    need = grouped_workspace_bytes(S, N, K, E, code)
    with _On(A, stream) as st:
        out = _out(out, "out", (S, N), dt, A)
        if pre is True:
            pre = A.new_empty((S, N))
        elif pre is False:
            pre = None
        if need and workspace is None:
            workspace = A.new_empty(need, dtype=torch.uint8)
        _ok(_lib().fl_grouped_linear(
            _ptr(A, "A"), _ptr(index, "index", torch.int32, (S,), A),
            _ptr(offsets, "offsets", torch.int32, (E + 1,), A), _ptr(B, "B", dt, None, A),
            _ptr(bias, "bias", dt, (E, N), A), _ptr(Y, "Y", dt, (S, N), A), out.data_ptr() or None,
            _ptr(pre, "pre", dt, (S, N), A), A_rows, S, N, K, E, ACTS[act], code,
            _ptr(workspace, "workspace", None, None, A),
            _bytes(workspace), st))
    return out if pre is None else (out, pre)


def grouped_linear_bwd(G, W, X, offsets, Y=None, act="relu", dX=None, dY=None, *, stream=None):
    """The backward epilogue over the experts' rows (fl_grouped_linear_bwd): D =
    G @ W[e]^T with G (S,K) and W (E,N,K), dX = D * act'(X) at the saved
    pre-activation X (S,N) (None with act="none"), for the gate also dY = D * X.
    Returns (dX, dY or None)."""
    S, K = _matrix(G, "G")
    if W.dim() != 3 or W.shape[2] != K:
        raise ValueError(f"W must be (E,N,{K}), got {tuple(W.shape)}")
    E, N, _ = W.shape
    dt = G.dtype
    with _On(G, stream) as st:
        dX = _out(dX, "dX", (S, N), dt, G)
        if act == "glu":
            dY = _out(dY, "dY", (S, N), dt, G)
        _ok(_lib().fl_grouped_linear_bwd(
            _ptr(G, "G"), _ptr(offsets, "offsets", torch.int32, (E + 1,), G), _ptr(W, "W", dt, None, G),
            _ptr(X, "X", dt, (S, N), G), _ptr(Y, "Y", dt, (S, N), G), dX.data_ptr() or None,
            _ptr(dY, "dY", dt, (S, N), G), S, N, K, E, ACTS[act], _code(dt), st))
    return dX, dY


def grouped_weight_grad(A, G, offsets, dbias=True, dW=None, dw_dtype=None, *, stream=None, workspace=None):
    """dW[e] = A[e]^T G[e] over every expert's rows and dbias[e] = the sum of
    its rows of G (fl_grouped_weight_grad_ws): A (S,K), G (S,N).  dW is (E,K,N)
    in dw_dtype (the operands' dtype by default, or float32).  dbias=True
    allocates the (E,N) fp32 result, a tensor is overwritten, None/False skips
    it.  Returns (dW, dbias or None)."""
    S, K = _matrix(A, "A")
    N = _matrix(G, "G")[1]
    E = offsets.numel() - 1
    dt = A.dtype
    code = _code(dt)
    dw_dtype = dw_dtype or (dW.dtype if dW is not None else dt)
    need = grouped_grad_workspace_bytes(S, N, K, E, code)
    with _On(A, stream) as st:
        dW = _out(dW, "dW", (E, K, N), dw_dtype, A)
        if dbias is True:
            dbias = A.new_empty((E, N), dtype=torch.float32)
        elif dbias is False:
            dbias = None
        if need and workspace is None:
            workspace = A.new_empty(need, dtype=torch.uint8)
        _ok(_lib().fl_grouped_weight_grad_ws(
            _ptr(A, "A"), _ptr(G, "G", dt, (S, N), A), _ptr(offsets, "offsets", torch.int32, (E + 1,), A),
            dW.data_ptr() or None, _ptr(dbias, "dbias", torch.float32, (E, N), A), S, N, K, E, code,
            _code(dw_dtype), _ptr(workspace, "workspace", None, None, A), _bytes(workspace), st))
    return dW, dbias
