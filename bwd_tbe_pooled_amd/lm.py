"""Language-model operators beside the table-batched embedding (include/tbe_lm.h).

  token    tbe_token_forward, tbe_token_backward: lookup of one token table
           with a scale, and the table's dense gradient
  expert   tbe_expert_plan, tbe_expert_dispatch, tbe_expert_combine and their
           backward calls: tokens sorted by expert and back with weights
  distill  tbe_distill_forward, tbe_distill_backward, tbe_distill_step: the
           loss against a teacher's top logits, and its gradient
  norm     tbe_norm_forward, tbe_norm_backward: layer norm of rows, and its
           gradients
  ffn      tbe_ffn_forward, tbe_ffn_backward: the experts' gated feed-forward
           products over rows sorted by expert, and their gradients
  adamw    tbe_adamw_step: one AdamW step over many tensors

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


class tbe_norm_desc(ctypes.Structure):
    _fields_ = [("N", _I64), ("D", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("wdtype", ctypes.c_int), ("eps", ctypes.c_float)]


class tbe_ffn_desc(ctypes.Structure):
    _fields_ = [("M", _I64), ("E", ctypes.c_int32), ("D", ctypes.c_int32), ("F", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("act", ctypes.c_int32)]


class tbe_stack(ctypes.Structure):
    _fields_ = [("data", _P), ("ld", _I64), ("stride", _I64)]


class tbe_adamw_desc(ctypes.Structure):
    _fields_ = [("pdtype", ctypes.c_int), ("gdtype", ctypes.c_int), ("cdtype", ctypes.c_int32),
                ("bits", ctypes.c_int32), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double)]


class tbe_adamw_tensor(ctypes.Structure):
    _fields_ = [("p", _P), ("g", _P), ("m", _P), ("v", _P), ("mscale", _P), ("vscale", _P),
                ("c", _P), ("n", _I64)]


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
_norm_forward = _declare("tbe_norm_forward", _P, *_m, _P, _P, *_m, _P, _P)
_norm_workspace_bytes = _declare("tbe_norm_workspace_bytes", _P, restype=_SZ)
_norm_backward = _declare("tbe_norm_backward", _P, *_m, *_m, _P, _P, *_m, _P, _P, *_ws, _P)
_ffn_workspace_bytes = _declare("tbe_ffn_workspace_bytes", _P, restype=_SZ)
_ffn_forward = _declare("tbe_ffn_forward", _P, *_m, _P, _P, _P, _P, *_m, *_m, *_ws, _P)
_ffn_backward = _declare("tbe_ffn_backward", _P, *_m, *_m, _P, _P, _P, _P, *_m, *_m, _P, _P, _P,
                         *_ws, _P)
_adamw_step = _declare("tbe_adamw_step", _P, _P, _I64, _P, _P, _P, _P)


# checks of a call's tensors, and the call: in C++ (csrc/lm_call.cpp)
_lmcall.bind(tuple(ctypes.cast(f, _P).value for f in (
    _token_forward, _token_backward, _expert_plan, _expert_dispatch, _expert_dispatch_backward,
    _expert_combine, _expert_combine_backward, _distill_forward, _distill_backward, _distill_step,
    _norm_forward, _norm_backward, _ffn_forward, _ffn_backward, _adamw_step)))


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


# --- layer norm ------------------------------------------------------------------------
class NormDesc(_LmDesc):
    """N rows of D columns (dtype); wdtype: type of weight, bias and their gradients."""

    def __init__(self, N: int, D: int, dtype: str = "bf16", wdtype: str = "f32", eps: float = 1e-5):
        self.N, self.D = int(N), int(D)
        self._own(tbe_norm_desc, self.N, self.D, DTYPE_CODES[dtype], DTYPE_CODES[wdtype], float(eps))


def norm_workspace(desc: NormDesc, device="cuda"):
    """Workspace of tbe_norm_backward."""
    _need_desc(desc, NormDesc)
    return _workspace(_norm_workspace_bytes, desc, "tbe_norm_workspace_bytes", device)


def tbe_norm_forward(desc: NormDesc, x, w, b, y, stats, stream=None):
    """y = (x - mean) * rstd * w + b by rows; stats [N, 2] for the backward. w, b: a
    tensor [D], or None for ones and zeros."""
    if type(desc) is not NormDesc:
        _need_desc(desc, NormDesc)
    status = _lmcall.norm_forward(desc.ref, x, w, b, y, stats, stream)
    if status:
        raise TbeError(status, "tbe_norm_forward")


def tbe_norm_backward(desc: NormDesc, dy, x, w, stats, dx, dw, db, ws, stream=None):
    """Gradients of rows, weight and bias. dw, db: a tensor [D], or None to leave it out."""
    if type(desc) is not NormDesc:
        _need_desc(desc, NormDesc)
    status = _lmcall.norm_backward(desc.ref, dy, x, w, stats, dx, dw, db, ws, stream)
    if status:
        raise TbeError(status, "tbe_norm_backward")


# --- experts' gated feed-forward ----------------------------------------------------------
ACT_CODES = {"silu": 0, "gelu": 1}


class FfnDesc(_LmDesc):
    """M rows of D columns sorted by expert, E experts of F columns between their products."""

    def __init__(self, M: int, E: int, D: int, F: int, dtype: str = "bf16", act: str = "silu"):
        self.M, self.E, self.D, self.F = int(M), int(E), int(D), int(F)
        self._own(tbe_ffn_desc, self.M, self.E, self.D, self.F, DTYPE_CODES[dtype], ACT_CODES[act])


def ffn_workspace(desc: FfnDesc, device="cuda"):
    """Workspace of tbe_ffn_forward and tbe_ffn_backward."""
    _need_desc(desc, FfnDesc)
    return _workspace(_ffn_workspace_bytes, desc, "tbe_ffn_workspace_bytes", device)


def tbe_ffn_forward(desc: FfnDesc, xs, offsets, gate, up, down, pre, ys, ws, stream=None):
    """ys = (act(xs gate[e]^T) * (xs up[e]^T)) down[e]^T for the rows of each expert e
    (offsets[e] on); pre [M, 2 F]: both products, kept for the backward, or None."""
    if type(desc) is not FfnDesc:
        _need_desc(desc, FfnDesc)
    status = _lmcall.ffn_forward(desc.ref, xs, offsets, gate, up, down, pre, ys, ws, stream)
    if status:
        raise TbeError(status, "tbe_ffn_forward")


def tbe_ffn_backward(desc: FfnDesc, dys, xs, offsets, gate, up, down, pre, dxs, dgate, dup, ddown, ws,
                     stream=None):
    """Gradients of the rows and of all experts' matrices."""
    if type(desc) is not FfnDesc:
        _need_desc(desc, FfnDesc)
    status = _lmcall.ffn_backward(desc.ref, dys, xs, offsets, gate, up, down, pre, dxs, dgate, dup,
                                  ddown, ws, stream)
    if status:
        raise TbeError(status, "tbe_ffn_backward")


# --- AdamW ---------------------------------------------------------------------------------
ADAMW_BLOCK = 256   # elements that share a scale of an 8-bit moment


class AdamWDesc(_LmDesc):
    """An AdamW step. pdtype: type of the parameters, gdtype: of their gradients, cdtype: of
    16-bit copies of float32 parameters (None: no copies), bits: of a moment (32 or 8)."""

    def __init__(self, pdtype: str = "f32", gdtype: str = "bf16", cdtype: str = None, bits: int = 32,
                 beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                 weight_decay: float = 0.01):
        self.bits = int(bits)
        self._own(tbe_adamw_desc, DTYPE_CODES[pdtype], DTYPE_CODES[gdtype],
                  -1 if cdtype is None else DTYPE_CODES[cdtype], self.bits, float(beta1),
                  float(beta2), float(eps), float(weight_decay))


class AdamWState:
    """The moments of `params`, zero before the first step: `m` and `v` of each tensor, and
    with 8 bits the scales `ms` and `vs` of their blocks (v's numbers are roots). Each kind
    is one buffer (`m_flat` ...) in which tensors begin at whole blocks. The step writes
    through addresses taken here: saved moments are copied in (`state.m_flat.copy_(...)`),
    other tensors cannot be put in the buffers' place."""

    def __init__(self, desc: AdamWDesc, params, device=None):
        _need_desc(desc, AdamWDesc)
        if desc.bits not in (8, 32):
            raise TbeError(TBE_ERR_ARG, "AdamWState")
        self.bits = desc.bits
        params = list(params)
        sizes = [p.numel() for p in params]
        blocks = [-(-n // ADAMW_BLOCK) for n in sizes]
        if device is None:
            device = params[0].device if len(sizes) else "cuda"
        total, kind = sum(blocks), torch.float32 if desc.bits == 32 else torch.float8_e4m3fn
        bytes_of = 4 if desc.bits == 32 else 1
        # zeros are written as bytes: e4m3 has no fill
        self.m_flat, self.v_flat = (torch.zeros(total * ADAMW_BLOCK * bytes_of, dtype=torch.uint8,
                                                device=device).view(kind) for _ in "mv")
        m, v, ms, vs = [], [], [], []
        flats = (self.m_flat, self.v_flat)
        if desc.bits == 8:
            self.ms_flat, self.vs_flat = (torch.zeros(total, device=device) for _ in "mv")
            flats += (self.ms_flat, self.vs_flat)
        self._c = (tbe_adamw_tensor * max(1, len(sizes)))()
        at = 0
        for i, (p, n, b) in enumerate(zip(params, sizes, blocks)):
            a = at * ADAMW_BLOCK
            m.append(self.m_flat[a:a + n].view(p.shape))
            v.append(self.v_flat[a:a + n].view(p.shape))
            self._c[i].n = n
            self._c[i].m, self._c[i].v = (f.data_ptr() + a * bytes_of for f in (self.m_flat, self.v_flat))
            if desc.bits == 8:
                ms.append(self.ms_flat[at:at + b])
                vs.append(self.vs_flat[at:at + b])
                self._c[i].mscale, self._c[i].vscale = (f.data_ptr() + 4 * at
                                                        for f in (self.ms_flat, self.vs_flat))
            at += b
        self.m, self.v = tuple(m), tuple(v)
        self.ms, self.vs = (tuple(ms), tuple(vs)) if desc.bits == 8 else (None, None)
        self._table = (ctypes.addressof(self._c), len(sizes), flats, tuple(f.data_ptr() for f in flats))

    def __setattr__(self, name, value):
        if "_table" in self.__dict__:
            raise AttributeError(f"AdamWState: {name} stays what it is; copy into the buffers")
        object.__setattr__(self, name, value)

    def __delattr__(self, name):
        raise AttributeError(f"AdamWState: {name} stays what it is")


def tbe_adamw_step(desc: AdamWDesc, params, grads, state: AdamWState, step, lr, scale=None, copies=None,
                   stream=None):
    """One step over the lists `params` and `grads`. step (int64 [1], counted from 1), lr and
    scale (float32 [1]; scale multiplies the gradients, None for 1) are device tensors; copies:
    a list of tensors that take the new parameters in 16 bits. Gradients and copies have their
    parameter's shape, or either of the two is flat."""
    if type(desc) is not AdamWDesc:
        _need_desc(desc, AdamWDesc)
    if not isinstance(state, AdamWState) or state.bits != desc.bits:
        raise TypeError("state: expected an AdamWState of the description's bits")
    status = _lmcall.adamw_step(desc.ref, state._table, params, grads, step, lr, scale, copies, stream)
    if status:
        raise TbeError(status, "tbe_adamw_step")
