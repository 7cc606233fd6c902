"""Language-model operators beside the table-batched embedding (include/tbe_lm.h).

  token    tbe_token_forward, tbe_token_backward: lookup of one token table
           with a scale, and the table's dense gradient
  expert   tbe_expert_plan, tbe_expert_dispatch, tbe_expert_combine and their
           backward calls: tokens sorted by expert and back with weights
  distill  tbe_distill_forward, tbe_distill_backward, tbe_distill_step: the
           loss against a teacher's top logits, and its gradient

Matrices are 2-D device tensors with unit column stride and any row stride (an
output's at least its width); ids and per-row vectors are contiguous; all are on
one device, the stream's. The checks of a call's tensors and the call itself are
compiled (csrc/lm_call.cpp); the functions here check the description's kind and
turn a status into an error. The ctypes declarations give the descriptions their
workspace sizes, the compiled calls their addresses and tests the plain C ABI.
"""
from __future__ import annotations

import ctypes

import torch

from . import DTYPE_CODES, LIB_PATH, TBE_ERR_ARG, TBE_ERR_UNSUPPORTED, TbeError, _lib

try:
    from . import _lmcall
except ImportError as e:
    raise ImportError("_lmcall.so is missing, or built for another Python or torch: build it with "
                      f"`python bwd_tbe_pooled_amd/build.py` ({e})") from e

_P, _I64, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t


class tbe_token_desc(ctypes.Structure):
    _fields_ = [("N", _I64), ("V", _I64), ("D", ctypes.c_int32), ("wdtype", ctypes.c_int),
                ("xdtype", ctypes.c_int), ("idx64", ctypes.c_int32), ("scale", ctypes.c_float)]


class tbe_expert_desc(ctypes.Structure):
    _fields_ = [("N", _I64), ("K", ctypes.c_int32), ("E", ctypes.c_int32), ("D", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("idx64", ctypes.c_int32)]


class tbe_distill_desc(ctypes.Structure):
    _fields_ = [("N", _I64), ("V", _I64), ("K", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("tdtype", ctypes.c_int), ("idx64", ctypes.c_int32),
                ("temperature", ctypes.c_float)]


def _declare(name, *args, restype=ctypes.c_int):
    try:
        f = getattr(_lib, name)
    except AttributeError as e:
        raise ImportError(f"{LIB_PATH} has no language-model operators ({e})") from e
    f.restype, f.argtypes = restype, list(args)
    return f


# desc and stream stand first and last; m: matrix (pointer, row stride)
_m = (_P, _I64)
_ws = (_P, _SZ)
_token_forward = _declare("tbe_token_forward", _P, *_m, _P, *_m, _P)
_token_workspace_bytes = _declare("tbe_token_workspace_bytes", _P, restype=_SZ)
_token_backward = _declare("tbe_token_backward", _P, *_m, _P, *_m, *_ws, _P)
_expert_workspace_bytes = _declare("tbe_expert_workspace_bytes", _P, restype=_SZ)
_expert_plan = _declare("tbe_expert_plan", _P, _P, _P, _P, _P, *_ws, _P)
_expert_dispatch = _declare("tbe_expert_dispatch", _P, *_m, _P, *_m, _P)
_expert_dispatch_backward = _declare("tbe_expert_dispatch_backward", _P, *_m, _P, *_m, _P)
_expert_combine = _declare("tbe_expert_combine", _P, *_m, _P, _P, *_m, _P)
_expert_combine_backward = _declare("tbe_expert_combine_backward", _P, *_m, *_m, _P, _P, *_m, _P, _P)
_distill_workspace_bytes = _declare("tbe_distill_workspace_bytes", _P, restype=_SZ)
_distill_forward = _declare("tbe_distill_forward", _P, *_m, _P, _P, _P, _P, *_ws, _P)
_distill_backward = _declare("tbe_distill_backward", _P, *_m, _P, _P, _P, _P, *_m, _P)
_distill_step = _declare("tbe_distill_step", _P, *_m, _P, _P, _P, _P, *_m, *_ws, _P)


# checks of a call's tensors, and the call: in C++ (csrc/lm_call.cpp)
_lmcall.bind(tuple(ctypes.cast(f, _P).value for f in (
    _token_forward, _token_backward, _expert_plan, _expert_dispatch, _expert_dispatch_backward,
    _expert_combine, _expert_combine_backward, _distill_forward, _distill_backward, _distill_step)))


def _need_desc(desc, kind):
    """Raise TypeError unless `desc` is a `kind`: the library reads the memory of a
    description as what the call is for."""
    if not isinstance(desc, kind):
        raise TypeError(f"desc: expected {kind.__name__}, got {type(desc).__name__}")


def _workspace(bytes_of, desc, where, device):
    n = int(bytes_of(desc.ref))
    if n == 0:
        raise TbeError(TBE_ERR_ARG, where)
    return torch.empty(n, dtype=torch.uint8, device=device)


class _LmDesc:
    """Owns the C description `c`; `ref` is its address."""

    def _own(self, c_type, *values):
        c = c_type(*values)
        for (name, _), v in zip(c_type._fields_, values):
            # ctypes keeps the low bits of a whole number that a field cannot hold
            if isinstance(v, int) and getattr(c, name) != v:
                raise TbeError(TBE_ERR_UNSUPPORTED, f"{type(self).__name__}: {name} = {v}")
        self.c = c
        self.ref = ctypes.addressof(c)


# --- token table -------------------------------------------------------------------
class TokenDesc(_LmDesc):
    """N tokens of a table of V rows and D columns. wdtype: type of the table
    and its gradient, xdtype: of the rows looked up and their gradient."""

    def __init__(self, N: int, V: int, D: int, wdtype: str = "bf16", xdtype: str = "bf16",
                 idx64: bool = True, scale: float = 1.0):
        self.N, self.V, self.D = int(N), int(V), int(D)
        self._own(tbe_token_desc, self.N, self.V, self.D, DTYPE_CODES[wdtype], DTYPE_CODES[xdtype],
                  int(bool(idx64)), float(scale))


def token_workspace(desc: TokenDesc, device="cuda"):
    """Workspace of tbe_token_backward."""
    _need_desc(desc, TokenDesc)
    return _workspace(_token_workspace_bytes, desc, "tbe_token_workspace_bytes", device)


def tbe_token_forward(desc: TokenDesc, W, ids, out, stream=None):
    """out[n] = scale * W[ids[n]]; zeros where the id is outside [0, V)."""
    if type(desc) is not TokenDesc:
        _need_desc(desc, TokenDesc)
    status = _lmcall.token_forward(desc.ref, W, ids, out, stream)
    if status:
        raise TbeError(status, "tbe_token_forward")


def tbe_token_backward(desc: TokenDesc, g, ids, gW, ws, stream=None):
    """gW[v] = scale * sum of g[n] over the tokens with ids[n] = v, all V rows."""
    if type(desc) is not TokenDesc:
        _need_desc(desc, TokenDesc)
    status = _lmcall.token_backward(desc.ref, g, ids, gW, ws, stream)
    if status:
        raise TbeError(status, "tbe_token_backward")


# --- experts -----------------------------------------------------------------------
class ExpertDesc(_LmDesc):
    """N tokens with K assignments each to E experts, rows of D columns."""

    def __init__(self, N: int, K: int, E: int, D: int, dtype: str = "bf16", idx64: bool = True):
        self.N, self.K, self.E, self.D = int(N), int(K), int(E), int(D)
        self.M = self.N * self.K
        self._own(tbe_expert_desc, self.N, self.K, self.E, self.D, DTYPE_CODES[dtype],
                  int(bool(idx64)))


class ExpertPlan:
    """Device buffers of a plan: `offsets` [E+1], `order` [N*K], `slots` [N*K]."""

    def __init__(self, desc: ExpertDesc, device="cuda"):
        _need_desc(desc, ExpertDesc)
        self.offsets = torch.empty(desc.E + 1, dtype=torch.int32, device=device)
        self.order = torch.empty(desc.M, dtype=torch.int32, device=device)
        self.slots = torch.empty(desc.M, dtype=torch.int32, device=device)


def expert_workspace(desc: ExpertDesc, device="cuda"):
    """Workspace of tbe_expert_plan."""
    _need_desc(desc, ExpertDesc)
    return _workspace(_expert_workspace_bytes, desc, "tbe_expert_workspace_bytes", device)


def tbe_expert_plan(desc: ExpertDesc, ids, plan: ExpertPlan, ws, stream=None):
    """Sorts the assignments by expert into `plan` (dropped ones at the end)."""
    if type(desc) is not ExpertDesc:
        _need_desc(desc, ExpertDesc)
    status = _lmcall.expert_plan(desc.ref, ids, plan.offsets, plan.order, plan.slots, ws, stream)
    if status:
        raise TbeError(status, "tbe_expert_plan")


def tbe_expert_dispatch(desc: ExpertDesc, x, slots, xs, stream=None):
    """xs[place of (n, k)] = x[n]; zeros at the places of dropped assignments."""
    if type(desc) is not ExpertDesc:
        _need_desc(desc, ExpertDesc)
    status = _lmcall.expert_dispatch(desc.ref, x, slots, xs, stream)
    if status:
        raise TbeError(status, "tbe_expert_dispatch")


def tbe_expert_dispatch_backward(desc: ExpertDesc, dxs, slots, dx, stream=None):
    """dx[n] = sum over kept k of dxs[place of (n, k)]."""
    if type(desc) is not ExpertDesc:
        _need_desc(desc, ExpertDesc)
    status = _lmcall.expert_dispatch_backward(desc.ref, dxs, slots, dx, stream)
    if status:
        raise TbeError(status, "tbe_expert_dispatch_backward")


def tbe_expert_combine(desc: ExpertDesc, ys, slots, w, out, stream=None):
    """out[n] = sum over kept k of w[n, k] * ys[place of (n, k)]."""
    if type(desc) is not ExpertDesc:
        _need_desc(desc, ExpertDesc)
    status = _lmcall.expert_combine(desc.ref, ys, slots, w, out, stream)
    if status:
        raise TbeError(status, "tbe_expert_combine")


def tbe_expert_combine_backward(desc: ExpertDesc, dout, ys, slots, w, dys, dw, stream=None):
    """dys[place of (n, k)] = w[n, k] * dout[n], dw[n, k] = <dout[n], ys[place]>;
    zeros where the assignment is dropped. dys may be ys."""
    if type(desc) is not ExpertDesc:
        _need_desc(desc, ExpertDesc)
    status = _lmcall.expert_combine_backward(desc.ref, dout, ys, slots, w, dys, dw, stream)
    if status:
        raise TbeError(status, "tbe_expert_combine_backward")


# --- distillation --------------------------------------------------------------------
class DistillDesc(_LmDesc):
    """N rows of V logits (dtype) against K teacher's logits a row (tdtype)."""

    def __init__(self, N: int, V: int, K: int, dtype: str = "bf16", tdtype: str = "f32",
                 idx64: bool = True, temperature: float = 1.0):
        self.N, self.V, self.K = int(N), int(V), int(K)
        self._own(tbe_distill_desc, self.N, self.V, self.K, DTYPE_CODES[dtype], DTYPE_CODES[tdtype],
                  int(bool(idx64)), float(temperature))


def distill_workspace(desc: DistillDesc, device="cuda"):
    """Workspace of tbe_distill_forward and tbe_distill_step."""
    _need_desc(desc, DistillDesc)
    return _workspace(_distill_workspace_bytes, desc, "tbe_distill_workspace_bytes", device)


def tbe_distill_forward(desc: DistillDesc, x, ids, t, loss, stats, ws, stream=None):
    """loss[n] = tau^2 KL(teacher || student) of row n; stats [N, 2] for the backward."""
    if type(desc) is not DistillDesc:
        _need_desc(desc, DistillDesc)
    status = _lmcall.distill_forward(desc.ref, x, ids, t, loss, stats, ws, stream)
    if status:
        raise TbeError(status, "tbe_distill_forward")


def tbe_distill_backward(desc: DistillDesc, x, ids, t, stats, gl, gx, stream=None):
    """gx = gl * tau * (softmax(x / tau) - teacher). gx may be x."""
    if type(desc) is not DistillDesc:
        _need_desc(desc, DistillDesc)
    status = _lmcall.distill_backward(desc.ref, x, ids, t, stats, gl, gx, stream)
    if status:
        raise TbeError(status, "tbe_distill_backward")


def tbe_distill_step(desc: DistillDesc, x, ids, t, gl, loss, gx, ws, stream=None):
    """Loss and gradient in one call. gx may be x."""
    if type(desc) is not DistillDesc:
        _need_desc(desc, DistillDesc)
    status = _lmcall.distill_step(desc.ref, x, ids, t, gl, loss, gx, ws, stream)
    if status:
        raise TbeError(status, "tbe_distill_step")
