// Python calls of the language-model operators (module _lmcall): checks the
// tensors of a call against its description, takes their addresses and row
// strides, and calls the C ABI (include/tbe_lm.h) on the given or the current
// stream. Argument marshalling only; in Python it took 1.8 us a call, half of
// what a launch takes, and a decoding step is a few such calls.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstdio>

#include "tbe_lm.h"

namespace {

// The library's entry points, from the loaded library's symbols (bind).
struct Entry {
  decltype(&tbe_token_forward) token_forward;
  decltype(&tbe_token_backward) token_backward;
  decltype(&tbe_expert_plan) expert_plan;
  decltype(&tbe_expert_dispatch) expert_dispatch;
  decltype(&tbe_expert_dispatch_backward) expert_dispatch_backward;
  decltype(&tbe_expert_combine) expert_combine;
  decltype(&tbe_expert_combine_backward) expert_combine_backward;
  decltype(&tbe_distill_forward) distill_forward;
  decltype(&tbe_distill_backward) distill_backward;
  decltype(&tbe_distill_step) distill_step;
  decltype(&tbe_norm_forward) norm_forward;
  decltype(&tbe_norm_backward) norm_backward;
  decltype(&tbe_ffn_forward) ffn_forward;
  decltype(&tbe_ffn_backward) ffn_backward;
  decltype(&tbe_adamw_step) adamw_step;
} lib;

// A refused argument; the Python error is set.
struct Refused {};

[[noreturn]] void refuse(const char* name, const char* what) {
  PyErr_Format(PyExc_TypeError, "%s: %s", name, what);
  throw Refused{};
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kHalf: return "torch.float16";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kInt: return "torch.int32";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return "torch.int64";
  }
}

// (A code that is none is refused by the library.)
at::ScalarType type_of(tbe_dtype t) {
  return t == TBE_F32 ? at::kFloat : t == TBE_F16 ? at::kHalf : at::kBFloat16;
}
at::ScalarType index_type(int32_t idx64) { return idx64 ? at::kLong : at::kInt; }

// The device of the call's tensors, -1 before the first: a kernel may fault on
// another device's memory, so all of them and the stream have to be of one.
thread_local int call_device = -1;

void on_call_device(const at::Tensor& x, const char* name) {
  const int device = (int)x.get_device();
  if (call_device < 0) call_device = device;
  else if (device != call_device) refuse(name, "must be on the device of the call's other tensors");
}

const at::Tensor& tensor(PyObject* o, const char* name, at::ScalarType t) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: expected a torch.Tensor, got %s", name, Py_TYPE(o)->tp_name);
    throw Refused{};
  }
  const at::Tensor& x = THPVariable_Unpack(o);
  if (!x.is_cuda()) refuse(name, "must be a device tensor");
  if (x.scalar_type() != t) {
    PyErr_Format(PyExc_TypeError, "%s: expected %s, got %s", name, type_name(t),
                 c10::toString(x.scalar_type()));
    throw Refused{};
  }
  on_call_device(x, name);
  return x;
}

[[noreturn]] void refuse_shape(const char* name, int64_t rows, int64_t cols) {
  char s[96];
  if (cols < 0) std::snprintf(s, sizeof s, "expected shape (%lld,)", (long long)rows);
  else std::snprintf(s, sizeof s, "expected shape (%lld, %lld)", (long long)rows, (long long)cols);
  refuse(name, s);
}

// A contiguous tensor of shape [rows], or [rows, cols] with cols >= 0.
void* vec(PyObject* o, const char* name, at::ScalarType t, int64_t rows, int64_t cols = -1) {
  const at::Tensor& x = tensor(o, name, t);
  const auto size = x.sizes();
  if (cols < 0 ? size.size() != 1 || size[0] != rows
               : size.size() != 2 || size[0] != rows || size[1] != cols)
    refuse_shape(name, rows, cols);
  if (!x.is_contiguous()) refuse(name, "must be contiguous");
  return x.data_ptr();
}

// A matrix with unit column stride.
struct Mat {
  void* p;
  int64_t ld;
};
Mat mat(PyObject* o, const char* name, at::ScalarType t, int64_t rows, int64_t cols,
        bool out = false) {
  const at::Tensor& x = tensor(o, name, t);
  const auto size = x.sizes();
  if (size.size() != 2 || size[0] != rows || size[1] != cols) refuse_shape(name, rows, cols);
  const auto stride = x.strides();
  if (stride[1] != 1 && cols > 1) refuse(name, "columns must be contiguous");
  int64_t ld = stride[0];
  if (rows <= 1) ld = cols;
  else if (out && ld < cols) refuse(name, "rows of an output must not overlap");
  return {x.data_ptr(), ld};
}

struct Scratch {
  void* p;
  size_t bytes;
};
Scratch scratch(PyObject* o) {
  if (THPVariable_Check(o)) {
    const at::Tensor& x = THPVariable_Unpack(o);
    if (x.is_cuda() && x.is_contiguous()) {
      on_call_device(x, "workspace");
      return {x.data_ptr(), x.nbytes()};
    }
  }
  refuse("workspace", "expected a contiguous device tensor");
}

// The stream's handle, after the call's tensors. A null handle is the default
// stream of the current device.
void* stream_of(PyObject* o) {
  constexpr const char* kOther = "must be of the tensors' device";
  if (o == Py_None) {
    const auto s = c10::hip::getCurrentHIPStream();
    if (s.device_index() != call_device)
      refuse("stream", "the current device must be the tensors' device");
    return s.stream();
  }
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  if (!h) throw Refused{};
  void* s = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (PyErr_Occurred()) throw Refused{};
  if (PyObject* d = PyObject_GetAttrString(o, "device_index")) {
    const long device = PyLong_AsLong(d);
    Py_DECREF(d);
    if (PyErr_Occurred()) throw Refused{};
    if (device != call_device) refuse("stream", kOther);
  } else {
    PyErr_Clear();  // a handle alone
  }
  if (!s && c10::hip::current_device() != call_device) refuse("stream", kOther);
  return s;
}

template <typename D>
const D& desc(PyObject* ref) {
  const void* p = PyLong_AsVoidPtr(ref);
  if (!p) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "desc: expected a description");
    throw Refused{};
  }
  return *static_cast<const D*>(p);
}

// The call's arguments: the description's address first, the stream last.
template <int N, typename F>
PyObject* call(PyObject* const* a, Py_ssize_t n, F f) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  call_device = -1;
  try {
    return PyLong_FromLong(f(a));
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
using Args = PyObject* const*;

PyObject* token_forward(PyObject*, Args args, Py_ssize_t n) {
  return call<5>(args, n, [](Args a) {
    const auto& d = desc<tbe_token_desc>(a[0]);
    const Mat W = mat(a[1], "W", type_of(d.wdtype), d.V, d.D);
    const void* ids = vec(a[2], "ids", index_type(d.idx64), d.N);
    const Mat out = mat(a[3], "out", type_of(d.xdtype), d.N, d.D, true);
    return lib.token_forward(&d, W.p, W.ld, ids, out.p, out.ld, stream_of(a[4]));
  });
}

PyObject* token_backward(PyObject*, Args args, Py_ssize_t n) {
  return call<6>(args, n, [](Args a) {
    const auto& d = desc<tbe_token_desc>(a[0]);
    const Mat g = mat(a[1], "g", type_of(d.xdtype), d.N, d.D);
    const void* ids = vec(a[2], "ids", index_type(d.idx64), d.N);
    const Mat gW = mat(a[3], "gW", type_of(d.wdtype), d.V, d.D, true);
    const Scratch ws = scratch(a[4]);
    return lib.token_backward(&d, g.p, g.ld, ids, gW.p, gW.ld, ws.p, ws.bytes, stream_of(a[5]));
  });
}

int32_t* slots_of(PyObject* o, const tbe_expert_desc& d) {
  return static_cast<int32_t*>(vec(o, "slots", at::kInt, d.N * d.K));
}
float* weights(PyObject* o, const char* name, const tbe_expert_desc& d) {
  return static_cast<float*>(vec(o, name, at::kFloat, d.N, d.K));
}

PyObject* expert_plan(PyObject*, Args args, Py_ssize_t n) {
  return call<7>(args, n, [](Args a) {
    const auto& d = desc<tbe_expert_desc>(a[0]);
    const int64_t M = d.N * d.K;
    const void* ids = vec(a[1], "ids", index_type(d.idx64), d.N, d.K);
    auto* offsets = static_cast<int32_t*>(vec(a[2], "plan.offsets", at::kInt, (int64_t)d.E + 1));
    auto* order = static_cast<int32_t*>(vec(a[3], "plan.order", at::kInt, M));
    auto* slots = static_cast<int32_t*>(vec(a[4], "plan.slots", at::kInt, M));
    const Scratch ws = scratch(a[5]);
    return lib.expert_plan(&d, ids, offsets, order, slots, ws.p, ws.bytes, stream_of(a[6]));
  });
}

PyObject* expert_dispatch(PyObject*, Args args, Py_ssize_t n) {
  return call<5>(args, n, [](Args a) {
    const auto& d = desc<tbe_expert_desc>(a[0]);
    const Mat x = mat(a[1], "x", type_of(d.dtype), d.N, d.D);
    const int32_t* slots = slots_of(a[2], d);
    const Mat xs = mat(a[3], "xs", type_of(d.dtype), d.N * d.K, d.D, true);
    return lib.expert_dispatch(&d, x.p, x.ld, slots, xs.p, xs.ld, stream_of(a[4]));
  });
}

PyObject* expert_dispatch_backward(PyObject*, Args args, Py_ssize_t n) {
  return call<5>(args, n, [](Args a) {
    const auto& d = desc<tbe_expert_desc>(a[0]);
    const Mat dxs = mat(a[1], "dxs", type_of(d.dtype), d.N * d.K, d.D);
    const int32_t* slots = slots_of(a[2], d);
    const Mat dx = mat(a[3], "dx", type_of(d.dtype), d.N, d.D, true);
    return lib.expert_dispatch_backward(&d, dxs.p, dxs.ld, slots, dx.p, dx.ld, stream_of(a[4]));
  });
}

PyObject* expert_combine(PyObject*, Args args, Py_ssize_t n) {
  return call<6>(args, n, [](Args a) {
    const auto& d = desc<tbe_expert_desc>(a[0]);
    const Mat ys = mat(a[1], "ys", type_of(d.dtype), d.N * d.K, d.D);
    const int32_t* slots = slots_of(a[2], d);
    const float* w = weights(a[3], "w", d);
    const Mat out = mat(a[4], "out", type_of(d.dtype), d.N, d.D, true);
    return lib.expert_combine(&d, ys.p, ys.ld, slots, w, out.p, out.ld, stream_of(a[5]));
  });
}

PyObject* expert_combine_backward(PyObject*, Args args, Py_ssize_t n) {
  return call<8>(args, n, [](Args a) {
    const auto& d = desc<tbe_expert_desc>(a[0]);
    const int64_t M = d.N * d.K;
    const Mat dout = mat(a[1], "dout", type_of(d.dtype), d.N, d.D);
    const Mat ys = mat(a[2], "ys", type_of(d.dtype), M, d.D);
    const int32_t* slots = slots_of(a[3], d);
    const float* w = weights(a[4], "w", d);
    const Mat dys = mat(a[5], "dys", type_of(d.dtype), M, d.D, true);
    float* dw = weights(a[6], "dw", d);
    return lib.expert_combine_backward(&d, dout.p, dout.ld, ys.p, ys.ld, slots, w, dys.p, dys.ld,
                                       dw, stream_of(a[7]));
  });
}

// What the distillation calls begin with.
struct Rows {
  const tbe_distill_desc& d;
  Mat x;
  const void *ids, *t;
  explicit Rows(Args a)
      : d(desc<tbe_distill_desc>(a[0])),
        x(mat(a[1], "x", type_of(d.dtype), d.N, d.V)),
        ids(vec(a[2], "ids", index_type(d.idx64), d.N, d.K)),
        t(vec(a[3], "t", type_of(d.tdtype), d.N, d.K)) {}
  float* row_vector(PyObject* o, const char* name) const {
    return static_cast<float*>(vec(o, name, at::kFloat, d.N));
  }
  float* stats(PyObject* o) const {
    return static_cast<float*>(vec(o, "stats", at::kFloat, d.N, 2));
  }
  Mat gx(PyObject* o) const { return mat(o, "gx", type_of(d.dtype), d.N, d.V, true); }
};

PyObject* distill_forward(PyObject*, Args args, Py_ssize_t n) {
  return call<8>(args, n, [](Args a) {
    const Rows r(a);
    float* loss = r.row_vector(a[4], "loss");
    float* stats = r.stats(a[5]);
    const Scratch ws = scratch(a[6]);
    return lib.distill_forward(&r.d, r.x.p, r.x.ld, r.ids, r.t, loss, stats, ws.p, ws.bytes,
                               stream_of(a[7]));
  });
}

PyObject* distill_backward(PyObject*, Args args, Py_ssize_t n) {
  return call<8>(args, n, [](Args a) {
    const Rows r(a);
    const float* stats = r.stats(a[4]);
    const float* gl = r.row_vector(a[5], "gl");
    const Mat gx = r.gx(a[6]);
    return lib.distill_backward(&r.d, r.x.p, r.x.ld, r.ids, r.t, stats, gl, gx.p, gx.ld,
                                stream_of(a[7]));
  });
}

PyObject* distill_step(PyObject*, Args args, Py_ssize_t n) {
  return call<9>(args, n, [](Args a) {
    const Rows r(a);
    const float* gl = r.row_vector(a[4], "gl");
    float* loss = r.row_vector(a[5], "loss");
    const Mat gx = r.gx(a[6]);
    const Scratch ws = scratch(a[7]);
    return lib.distill_step(&r.d, r.x.p, r.x.ld, r.ids, r.t, gl, loss, gx.p, gx.ld, ws.p, ws.bytes,
                            stream_of(a[8]));
  });
}

// A vector of the norm's weights' type, or NULL for None.
void* weight_vec(PyObject* o, const char* name, const tbe_norm_desc& d) {
  return o == Py_None ? nullptr : vec(o, name, type_of(d.wdtype), d.D);
}

PyObject* norm_forward(PyObject*, Args args, Py_ssize_t n) {
  return call<7>(args, n, [](Args a) {
    const auto& d = desc<tbe_norm_desc>(a[0]);
    const Mat x = mat(a[1], "x", type_of(d.dtype), d.N, d.D);
    const void* w = weight_vec(a[2], "w", d);
    const void* b = weight_vec(a[3], "b", d);
    const Mat y = mat(a[4], "y", type_of(d.dtype), d.N, d.D, true);
    auto* stats = static_cast<float*>(vec(a[5], "stats", at::kFloat, d.N, 2));
    return lib.norm_forward(&d, x.p, x.ld, w, b, y.p, y.ld, stats, stream_of(a[6]));
  });
}

PyObject* norm_backward(PyObject*, Args args, Py_ssize_t n) {
  return call<10>(args, n, [](Args a) {
    const auto& d = desc<tbe_norm_desc>(a[0]);
    const Mat dy = mat(a[1], "dy", type_of(d.dtype), d.N, d.D);
    const Mat x = mat(a[2], "x", type_of(d.dtype), d.N, d.D);
    const void* w = weight_vec(a[3], "w", d);
    auto* stats = static_cast<const float*>(vec(a[4], "stats", at::kFloat, d.N, 2));
    const Mat dx = mat(a[5], "dx", type_of(d.dtype), d.N, d.D, true);
    void* dw = weight_vec(a[6], "dw", d);
    void* db = weight_vec(a[7], "db", d);
    const Scratch ws = scratch(a[8]);
    return lib.norm_backward(&d, dy.p, dy.ld, x.p, x.ld, w, stats, dx.p, dx.ld, dw, db, ws.p,
                             ws.bytes, stream_of(a[9]));
  });
}

// E matrices of rows x cols with unit column stride.
tbe_stack stack(PyObject* o, const char* name, at::ScalarType t, int64_t E, int64_t rows,
                int64_t cols, bool out = false) {
  const at::Tensor& x = tensor(o, name, t);
  const auto size = x.sizes();
  if (size.size() != 3 || size[0] != E || size[1] != rows || size[2] != cols) {
    char s[96];
    std::snprintf(s, sizeof s, "expected shape (%lld, %lld, %lld)", (long long)E, (long long)rows,
                  (long long)cols);
    refuse(name, s);
  }
  const auto stride = x.strides();
  if (stride[2] != 1 && cols > 1) refuse(name, "columns must be contiguous");
  const int64_t ld = rows <= 1 ? cols : stride[1];
  const int64_t each = E <= 1 ? rows * ld : stride[0];
  // (rows without columns are the library's to refuse)
  if (out && cols > 0 && (ld < cols || each / ld < rows)) refuse(name, "rows of an output must not overlap");
  return {x.data_ptr(), ld, each};
}

const int32_t* offsets_of(PyObject* o, const tbe_ffn_desc& d) {
  return static_cast<const int32_t*>(vec(o, "offsets", at::kInt, (int64_t)d.E + 1));
}

PyObject* ffn_forward(PyObject*, Args args, Py_ssize_t n) {
  return call<10>(args, n, [](Args a) {
    const auto& d = desc<tbe_ffn_desc>(a[0]);
    const at::ScalarType t = type_of(d.dtype);
    const Mat xs = mat(a[1], "xs", t, d.M, d.D);
    const int32_t* offsets = offsets_of(a[2], d);
    const tbe_stack gate = stack(a[3], "gate", t, d.E, d.F, d.D);
    const tbe_stack up = stack(a[4], "up", t, d.E, d.F, d.D);
    const tbe_stack down = stack(a[5], "down", t, d.E, d.D, d.F);
    Mat pre{nullptr, 0};
    if (a[6] != Py_None) pre = mat(a[6], "pre", t, d.M, 2 * (int64_t)d.F, true);
    const Mat ys = mat(a[7], "ys", t, d.M, d.D, true);
    const Scratch ws = scratch(a[8]);
    return lib.ffn_forward(&d, xs.p, xs.ld, offsets, &gate, &up, &down, pre.p, pre.ld, ys.p, ys.ld,
                           ws.p, ws.bytes, stream_of(a[9]));
  });
}

PyObject* ffn_backward(PyObject*, Args args, Py_ssize_t n) {
  return call<14>(args, n, [](Args a) {
    const auto& d = desc<tbe_ffn_desc>(a[0]);
    const at::ScalarType t = type_of(d.dtype);
    const Mat dys = mat(a[1], "dys", t, d.M, d.D);
    const Mat xs = mat(a[2], "xs", t, d.M, d.D);
    const int32_t* offsets = offsets_of(a[3], d);
    const tbe_stack gate = stack(a[4], "gate", t, d.E, d.F, d.D);
    const tbe_stack up = stack(a[5], "up", t, d.E, d.F, d.D);
    const tbe_stack down = stack(a[6], "down", t, d.E, d.D, d.F);
    const Mat pre = mat(a[7], "pre", t, d.M, 2 * (int64_t)d.F);
    const Mat dxs = mat(a[8], "dxs", t, d.M, d.D, true);
    const tbe_stack dgate = stack(a[9], "dgate", t, d.E, d.F, d.D, true);
    const tbe_stack dup = stack(a[10], "dup", t, d.E, d.F, d.D, true);
    const tbe_stack ddown = stack(a[11], "ddown", t, d.E, d.D, d.F, true);
    const Scratch ws = scratch(a[12]);
    return lib.ffn_backward(&d, dys.p, dys.ld, xs.p, xs.ld, offsets, &gate, &up, &down, pre.p,
                            pre.ld, dxs.p, dxs.ld, &dgate, &dup, &ddown, ws.p, ws.bytes,
                            stream_of(a[13]));
  });
}

// A list or tuple of `count` tensors.
struct List {
  PyObject** item;
  List(PyObject* o, const char* name, Py_ssize_t count) {
    if (!PyList_Check(o) && !PyTuple_Check(o)) refuse(name, "expected a list or tuple of tensors");
    if (PySequence_Fast_GET_SIZE(o) != count) {
      PyErr_Format(PyExc_TypeError, "%s: expected %zd tensors, got %zd", name, count,
                   PySequence_Fast_GET_SIZE(o));
      throw Refused{};
    }
    item = PySequence_Fast_ITEMS(o);
  }
};
// A dense tensor of any shape with n elements.
void* dense(PyObject* o, const char* name, at::ScalarType t, int64_t n) {
  const at::Tensor& x = tensor(o, name, t);
  if (x.numel() != n) {
    PyErr_Format(PyExc_TypeError, "%s: expected %lld elements, got %lld", name, (long long)n,
                 (long long)x.numel());
    throw Refused{};
  }
  if (!x.is_contiguous()) refuse(name, "must be contiguous");
  return x.data_ptr();
}

// The same for what goes with a parameter: of its shape, or one of the two is flat and
// memory's order says which element is which.
void* beside(PyObject* o, const char* name, at::ScalarType t, PyObject* param, int64_t n) {
  void* const p = dense(o, name, t, n);
  const at::Tensor &x = THPVariable_Unpack(o), &y = THPVariable_Unpack(param);
  if (x.sizes() != y.sizes() && x.dim() != 1 && y.dim() != 1) refuse(name, "expected its parameter's shape");
  return p;
}

// The state's array of tbe_adamw_tensor with the moments filled in: `table` is its address,
// its length, the moments' buffers and the addresses these had when it was filled.
struct Table {
  tbe_adamw_tensor* t;
  Py_ssize_t count;
  Table(PyObject* o, const tbe_adamw_desc& d) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) refuse("state", "expected an AdamWState");
    t = static_cast<tbe_adamw_tensor*>(PyLong_AsVoidPtr(PyTuple_GET_ITEM(o, 0)));
    count = PyLong_AsSsize_t(PyTuple_GET_ITEM(o, 1));
    PyObject *flats = PyTuple_GET_ITEM(o, 2), *at = PyTuple_GET_ITEM(o, 3);
    const Py_ssize_t kinds = d.bits == 32 ? 2 : 4;
    if (!PyTuple_Check(flats) || !PyTuple_Check(at) || PyTuple_GET_SIZE(flats) != kinds ||
        PyTuple_GET_SIZE(at) != kinds)
      refuse("state", "expected an AdamWState of the description's bits");
    for (Py_ssize_t i = 0; i < kinds; ++i) {
      PyObject* const f = PyTuple_GET_ITEM(flats, i);
      if (!THPVariable_Check(f) || THPVariable_Unpack(f).data_ptr() != PyLong_AsVoidPtr(PyTuple_GET_ITEM(at, i)))
        refuse("state", "its buffers are not where they were when it was made");
    }
    if (PyErr_Occurred()) throw Refused{};
    for (Py_ssize_t i = 0; i < kinds; ++i)
      tensor(PyTuple_GET_ITEM(flats, i), "state", i < 2 && d.bits == 8 ? at::kFloat8_e4m3fn : at::kFloat);
  }
};

// adamw_step(desc, table, params, grads, step, lr, scale, copies, stream): the call fills
// in what the state's table lacks.
PyObject* adamw_step(PyObject*, Args args, Py_ssize_t n) {
  return call<9>(args, n, [](Args a) {
    const auto& d = desc<tbe_adamw_desc>(a[0]);
    const Table table(a[1], d);
    tbe_adamw_tensor* const t = table.t;
    const Py_ssize_t count = table.count;
    const List params(a[2], "params", count), grads(a[3], "grads", count);
    const bool copy = d.cdtype >= 0;
    if (copy == (a[7] == Py_None))
      refuse("copies", copy ? "expected a list or tuple of tensors" : "the description has none");
    PyObject** const copies = copy ? List(a[7], "copies", count).item : nullptr;
    for (Py_ssize_t i = 0; i < count; ++i) {
      t[i].p = dense(params.item[i], "params", type_of(d.pdtype), t[i].n);
      t[i].g = beside(grads.item[i], "grads", type_of(d.gdtype), params.item[i], t[i].n);
      t[i].c = copy ? beside(copies[i], "copies", type_of((tbe_dtype)d.cdtype), params.item[i], t[i].n) : nullptr;
    }
    auto* step = static_cast<const int64_t*>(vec(a[4], "step", at::kLong, 1));
    auto* lr = static_cast<const float*>(vec(a[5], "lr", at::kFloat, 1));
    auto* scale = a[6] == Py_None ? nullptr
                                  : static_cast<const float*>(vec(a[6], "scale", at::kFloat, 1));
    return lib.adamw_step(&d, t, count, step, lr, scale, stream_of(a[8]));
  });
}

// bind(addresses): the entry points' addresses, in Entry's order.
PyObject* bind(PyObject*, PyObject* addresses) {
  constexpr Py_ssize_t kEntries = sizeof(Entry) / sizeof(void*);
  if (!PyTuple_Check(addresses) || PyTuple_GET_SIZE(addresses) != kEntries) {
    PyErr_SetString(PyExc_TypeError, "bind: expected the entry points' addresses");
    return nullptr;
  }
  void* p[kEntries];
  for (Py_ssize_t i = 0; i < kEntries; ++i) {
    p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(addresses, i));
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null address");
      return nullptr;
    }
  }
  int i = 0;
  auto take = [&](auto& f) { f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(p[i++]); };
  take(lib.token_forward);
  take(lib.token_backward);
  take(lib.expert_plan);
  take(lib.expert_dispatch);
  take(lib.expert_dispatch_backward);
  take(lib.expert_combine);
  take(lib.expert_combine_backward);
  take(lib.distill_forward);
  take(lib.distill_backward);
  take(lib.distill_step);
  take(lib.norm_forward);
  take(lib.norm_backward);
  take(lib.ffn_forward);
  take(lib.ffn_backward);
  take(lib.adamw_step);
  Py_RETURN_NONE;
}

#define TBE_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", bind, METH_O, nullptr},
    TBE_METHOD(token_forward),
    TBE_METHOD(token_backward),
    TBE_METHOD(expert_plan),
    TBE_METHOD(expert_dispatch),
    TBE_METHOD(expert_dispatch_backward),
    TBE_METHOD(expert_combine),
    TBE_METHOD(expert_combine_backward),
    TBE_METHOD(distill_forward),
    TBE_METHOD(distill_backward),
    TBE_METHOD(distill_step),
    TBE_METHOD(norm_forward),
    TBE_METHOD(norm_backward),
    TBE_METHOD(ffn_forward),
    TBE_METHOD(ffn_backward),
    TBE_METHOD(adamw_step),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lmcall", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lmcall() { return PyModule_Create(&module); }
