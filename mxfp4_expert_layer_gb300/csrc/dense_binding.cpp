// Python binding of the dense operators for torch tensors: checks, output and workspace
// allocation and the call of the C ABI, in one native function per operator.  The same
// steps in Python (ctypes) cost 15 to 30 us a call, several times what the kernels of a
// decoded token take; here they cost 3 to 6.
//
// Every call runs on the current stream of its tensors' device, with that device current,
// takes its workspace from torch's allocator and keeps no state.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <initializer_list>
#include <sstream>
#include <string>
#include <utility>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe_mxfp4.h"

namespace {

PyObject* g_error_class = nullptr;  // MoEError(function, status)

struct Raised {};  // a Python error has been set
[[noreturn]] void value_error(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Raised{};
}

// None or a tensor.
const at::Tensor* optional(const char* name, PyObject* o) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: a tensor is needed, got %s", name, Py_TYPE(o)->tp_name);
    throw Raised{};
  }
  return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(const char* name, PyObject* o) {
  const at::Tensor* t = optional(name, o);
  if (!t) value_error(std::string(name) + ": a tensor is needed, got None");
  return *t;
}

// The results carry no history: where autograd records, a tensor that requires grad would
// lose its gradient without a word.
void no_history(std::initializer_list<std::pair<const char*, const at::Tensor*>> ts) {
  if (!c10::GradMode::is_enabled()) return;
  for (const auto& [name, t] : ts)
    if (t && t->requires_grad())
      value_error(std::string(name) + " requires grad, but gradients of this operator are explicit calls: call it under "
                                      "torch.no_grad(), or with detached tensors");
}

using Shape = std::initializer_list<int64_t>;

// The address of a contiguous tensor of this shape, type and device (null for null).
void* need(const char* name, const at::Tensor* t, Shape shape, at::ScalarType type, const at::Device& device) {
  if (!t) return nullptr;
  if (t->scalar_type() != type || t->sizes() != c10::IntArrayRef(shape) || t->device() != device || !t->is_contiguous()) {
    std::ostringstream s;
    s << name << ": a contiguous " << c10::toString(type) << " tensor of shape " << c10::IntArrayRef(shape) << " on " << device
      << " is needed, got " << c10::toString(t->scalar_type()) << " " << t->sizes() << " on " << t->device()
      << (t->is_contiguous() ? "" : ", not contiguous");
    value_error(s.str());
  }
  return t->data_ptr();
}

int dtype16(const at::Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return MOE_DTYPE_BF16;
  if (t.scalar_type() == at::kHalf) return MOE_DTYPE_F16;
  value_error(std::string("bf16 or f16 tensors are needed, got ") + c10::toString(t.scalar_type()));
}

void matrix(const char* name, const at::Tensor& t) {
  if (t.dim() != 2) value_error(std::string(name) + ": a matrix is needed");
}
int narrow(int64_t v) {
  if (v > INT32_MAX) value_error("a size beyond 2^31 - 1");
  return static_cast<int>(v);
}

at::Tensor empty(Shape shape, at::ScalarType type, const at::Device& device) {
  return at::detail::empty_cuda(shape, type, device, std::nullopt);
}
// Element `i` of a contiguous tensor's first dimension, sharing its storage.
at::Tensor row_of(const at::Tensor& m, int64_t i) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(m.storage()), m.key_set(), m.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(i * (m.numel() / m.size(0)));
  t.unsafeGetTensorImpl()->set_sizes_contiguous(m.sizes().slice(1));
  return t;
}
// Results of up to this many bytes together share one allocation: each costs host time that a
// decoded token's norm waits for (4.6 us a call among others, 4.1 shared), while larger
// results had better be freed one by one.
constexpr int64_t kShareBytes = 64 * 1024;
void* address(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
PyObject* wrap(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
PyObject* tuple(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) PyTuple_SET_ITEM(r, i++, wrap(t));
  return r;
}

void on_cuda(const at::Device& device) {
  if (!device.is_cuda()) value_error("CUDA tensors are needed");
}
void refuse(const char* name, int status) {
  PyObject* e = PyObject_CallFunction(g_error_class, "si", name, status);
  if (e) {
    PyErr_SetObject(g_error_class, e);
    Py_DECREF(e);
  }
  throw Raised{};
}
// One library call on the device's current stream, without the interpreter's lock.
template <typename F>
void call(const char* name, const at::Device& device, F f) {
  const moe_stream_t stream = reinterpret_cast<moe_stream_t>(c10::cuda::getCurrentCUDAStream(device.index()).stream());
  int status;
  PyThreadState* state = PyEval_SaveThread();
  status = f(stream);
  PyEval_RestoreThread(state);
  if (status != MOE_OK) refuse(name, status);
}

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
int integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (v < INT32_MIN || v > INT32_MAX) value_error("an integer beyond 32 bits");
  return static_cast<int>(v);
}
bool flag(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v == 1;
}
bool arguments(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments are needed, got %zd", want, got);
  return false;
}

// ------------------------------------------------------------------ norms around a block
struct Gate {
  int kind;
  void* ptr;
};
Gate gate_of(const at::Tensor* g, int64_t T, int64_t H, at::ScalarType type, const at::Device& device) {
  if (!g) return {MOE_GATE_NONE, nullptr};
  if (g->dim() == 1) return {MOE_GATE_FEATURE, need("gate", g, {H}, type, device)};
  if (g->dim() == 2 && g->size(0) == T && g->size(1) == 1) return {MOE_GATE_TOKEN, need("gate", g, {T, 1}, at::kFloat, device)};
  return {MOE_GATE_FULL, need("gate", g, {T, H}, type, device)};
}
int stream_dtype(at::ScalarType stream, at::ScalarType type, int code) {
  if (stream == type) return code;
  if (stream == at::kFloat) return MOE_DTYPE_F32;
  value_error(std::string("the residual stream has block's type or float32, got ") + c10::toString(stream));
}

// block, residual, norm_weight, gate, residual_scale, next_weight, eps, residual_out, out
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& block = tensor("block", a[0]);
    const at::Tensor *residual = optional("residual", a[1]), *norm_w = optional("norm_weight", a[2]),
                     *gate = optional("gate", a[3]), *next_w = optional("next_weight", a[5]),
                     *given_res = optional("residual_out", a[7]), *given_out = optional("out", a[8]);
    const float scale = (float)number(a[4]), eps = (float)number(a[6]);
    no_history({{"block", &block}, {"residual", residual}, {"norm_weight", norm_w}, {"gate", gate}, {"next_weight", next_w},
                {"residual_out", given_res}, {"out", given_out}});
    matrix("block", block);
    const int64_t T = block.size(0), H = block.size(1);
    const at::ScalarType type = block.scalar_type();
    const at::Device device = block.device();
    const int code = dtype16(block);
    const at::ScalarType stype = residual ? residual->scalar_type() : given_res ? given_res->scalar_type() : type;
    const int scode = stream_dtype(stype, type, code);
    const Gate g = gate_of(gate, T, H, type, device);
    if (given_out && !next_w) value_error("out needs next_weight");
    on_cuda(device);
    const c10::cuda::CUDAGuard guard(device);
    void *z = need("block", &block, {T, H}, type, device), *r = need("residual", residual, {T, H}, stype, device),
         *wz = need("norm_weight", norm_w, {H}, type, device), *wn = need("next_weight", next_w, {H}, type, device);
    need("residual_out", given_res, {T, H}, stype, device);
    need("out", given_out, {T, H}, type, device);
    at::Tensor res, out;
    if (!given_res && !given_out && next_w && stype == type && T > 0 && 4 * T * H <= kShareBytes) {
      const at::Tensor both = empty({2, T, H}, type, device);
      res = row_of(both, 0);
      out = row_of(both, 1);
    } else {
      res = given_res ? *given_res : empty({T, H}, stype, device);
      if (next_w) out = given_out ? *given_out : empty({T, H}, type, device);
    }
    const int t = narrow(T), h = narrow(H);
    call("moe_block_norm", device, [&](moe_stream_t s) {
      return moe_block_norm(z, wz, g.ptr, g.kind, r, scale, wn, eps, t, h, code, scode, res.data_ptr(), address(out), s);
    });
    return tuple({res, out});
  });
}

// d_residual_out, d_out, block, residual_out, norm_weight, gate, residual_scale, next_weight, eps, has_residual
PyObject* block_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 10)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor *ds = optional("d_residual_out", a[0]), *dy = optional("d_out", a[1]);
    const at::Tensor& block = tensor("block", a[2]);
    const at::Tensor *res = optional("residual_out", a[3]), *norm_w = optional("norm_weight", a[4]),
                     *gate = optional("gate", a[5]), *next_w = optional("next_weight", a[7]);
    const float scale = (float)number(a[6]), eps = (float)number(a[8]);
    const bool has_residual = flag(a[9]);
    no_history({{"d_residual_out", ds}, {"d_out", dy}});
    matrix("block", block);
    const int64_t T = block.size(0), H = block.size(1);
    const at::ScalarType type = block.scalar_type();
    const at::Device device = block.device();
    const int code = dtype16(block);
    const at::ScalarType stype = ds ? ds->scalar_type() : res ? res->scalar_type() : type;
    const int scode = stream_dtype(stype, type, code);
    const Gate g = gate_of(gate, T, H, type, device);
    on_cuda(device);
    const c10::cuda::CUDAGuard guard(device);
    void *pds = need("d_residual_out", ds, {T, H}, stype, device), *pdy = need("d_out", dy, {T, H}, type, device),
         *z = need("block", &block, {T, H}, type, device), *s = need("residual_out", res, {T, H}, stype, device),
         *wz = need("norm_weight", norm_w, {H}, type, device), *wn = need("next_weight", next_w, {H}, type, device);
    const int t = narrow(T), h = narrow(H);
    const size_t bytes = moe_block_norm_workspace_bytes(t, h);
    if (!bytes) refuse("moe_block_norm_backward", MOE_ERR_UNSUPPORTED_SHAPE);
    at::Tensor d_block = empty({T, H}, type, device), d_res, d_norm, d_gate, d_next;
    if (has_residual) d_res = empty({T, H}, stype, device);
    // the f32 rows in one allocation (each takes half a microsecond of the call's ten)
    const bool of_feature = g.kind == MOE_GATE_FEATURE;
    const int rows = (norm_w != nullptr) + (next_w != nullptr) + of_feature;
    if (rows) {
      const at::Tensor all = empty({rows, H}, at::kFloat, device);
      int row = 0;
      if (norm_w) d_norm = row_of(all, row++);
      if (next_w) d_next = row_of(all, row++);
      if (of_feature) d_gate = row_of(all, row++);
    }
    if (g.kind == MOE_GATE_TOKEN) d_gate = empty({T, 1}, at::kFloat, device);
    if (g.kind == MOE_GATE_FULL) d_gate = empty({T, H}, type, device);
    const at::Tensor ws = empty({(int64_t)bytes}, at::kByte, device);
    call("moe_block_norm_backward", device, [&](moe_stream_t st) {
      return moe_block_norm_backward(pds, pdy, z, wz, g.ptr, g.kind, s, scale, wn, eps, t, h, code, scode, d_block.data_ptr(),
                                     address(d_res), static_cast<float*>(address(d_norm)), address(d_gate),
                                     static_cast<float*>(address(d_next)), ws.data_ptr(), bytes, st);
    });
    return tuple({d_block, d_res, d_norm, d_gate, d_next});
  });
}

// ------------------------------------------------------------------ gated feed-forward block
struct FfnShape {
  int64_t T, H, I;
};
FfnShape ffn_shape(const at::Tensor& x, const at::Tensor& w_gateup) {
  matrix("x", x);
  matrix("w_gateup", w_gateup);
  return {x.size(0), x.size(1), w_gateup.size(0) / 2};
}

// x, w_gateup, w_down, act, save, out
PyObject* ffn_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 6)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &x = tensor("x", a[0]), &wgu = tensor("w_gateup", a[1]), &wd = tensor("w_down", a[2]);
    const int act = integer(a[3]);
    const bool save = flag(a[4]);
    const at::Tensor* given = optional("out", a[5]);
    no_history({{"x", &x}, {"w_gateup", &wgu}, {"w_down", &wd}, {"out", given}});
    const auto [T, H, I] = ffn_shape(x, wgu);
    const at::ScalarType type = x.scalar_type();
    const at::Device device = x.device();
    const int code = dtype16(x);
    on_cuda(device);
    const c10::cuda::CUDAGuard guard(device);
    void *px = need("x", &x, {T, H}, type, device), *pgu = need("w_gateup", &wgu, {2 * I, H}, type, device),
         *pd = need("w_down", &wd, {H, I}, type, device);
    need("out", given, {T, H}, type, device);
    const int t = narrow(T), h = narrow(H), i = narrow(I);
    const size_t bytes = moe_ffn_workspace_bytes(t, h, i, 0);
    if (!bytes) refuse("moe_ffn_forward", MOE_ERR_UNSUPPORTED_SHAPE);
    at::Tensor out = given ? *given : empty({T, H}, type, device), gateup;
    if (save) gateup = empty({T, 2 * I}, at::kFloat, device);
    const at::Tensor ws = empty({(int64_t)bytes}, at::kByte, device);
    call("moe_ffn_forward", device, [&](moe_stream_t s) {
      return moe_ffn_forward(px, pgu, pd, t, h, i, act, code, static_cast<float*>(address(gateup)), out.data_ptr(),
                             ws.data_ptr(), bytes, s);
    });
    return tuple({out, gateup});
  });
}

// d_out, x, gateup, w_gateup, w_down, act, need_x, need_weights
PyObject* ffn_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 8)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &dout = tensor("d_out", a[0]), &x = tensor("x", a[1]), &gateup = tensor("gateup", a[2]),
                     &wgu = tensor("w_gateup", a[3]), &wd = tensor("w_down", a[4]);
    const int act = integer(a[5]);
    const bool need_x = flag(a[6]), need_w = flag(a[7]);
    no_history({{"d_out", &dout}});
    const auto [T, H, I] = ffn_shape(x, wgu);
    const at::ScalarType type = x.scalar_type();
    const at::Device device = x.device();
    const int code = dtype16(x);
    on_cuda(device);
    const c10::cuda::CUDAGuard guard(device);
    void *pdo = need("d_out", &dout, {T, H}, type, device), *px = need("x", &x, {T, H}, type, device),
         *pg = need("gateup", &gateup, {T, 2 * I}, at::kFloat, device),
         *pgu = need("w_gateup", &wgu, {2 * I, H}, type, device), *pd = need("w_down", &wd, {H, I}, type, device);
    const int t = narrow(T), h = narrow(H), i = narrow(I);
    const size_t bytes = moe_ffn_workspace_bytes(t, h, i, 1);
    if (!bytes) refuse("moe_ffn_backward", MOE_ERR_UNSUPPORTED_SHAPE);
    at::Tensor d_x, d_wgu, d_wd;
    if (need_x) d_x = empty({T, H}, type, device);
    if (need_w) {
      d_wgu = empty({2 * I, H}, type, device);
      d_wd = empty({H, I}, type, device);
    }
    const at::Tensor ws = empty({(int64_t)bytes}, at::kByte, device);
    call("moe_ffn_backward", device, [&](moe_stream_t s) {
      return moe_ffn_backward(pdo, px, static_cast<const float*>(pg), pgu, pd, t, h, i, act, code, address(d_x),
                              address(d_wgu), address(d_wd), ws.data_ptr(), bytes, s);
    });
    return tuple({d_x, d_wgu, d_wd});
  });
}

// ------------------------------------------------------------------ a few tokens x MXFP4 weights
// x, weight (prepared), bias, rows, K, kind, act, out
PyObject* matvec(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 8)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &x = tensor("x", a[0]), &w = tensor("weight", a[1]);
    const at::Tensor *bias = optional("bias", a[2]), *given = optional("out", a[7]);
    const int rows = integer(a[3]), K = integer(a[4]), kind = integer(a[5]), act = integer(a[6]);
    no_history({{"x", &x}, {"bias", bias}, {"out", given}});
    matrix("x", x);
    const int64_t T = x.size(0), n_out = kind == MOE_WEIGHTS_GATEUP ? rows / 2 : rows;
    const at::ScalarType type = x.scalar_type();
    const at::Device device = w.device();
    const int code = dtype16(x);
    on_cuda(device);
    const c10::cuda::CUDAGuard guard(device);
    void* px = need("x", &x, {T, K}, type, device);
    void* pb = need("bias", bias, {rows}, at::kFloat, device);
    need("weight", &w, {(int64_t)moe_prepared_matvec_bytes(rows, K, kind)}, at::kByte, device);
    need("out", given, {T, n_out}, type, device);
    const int t = narrow(T);
    const at::Tensor out = given ? *given : empty({T, n_out}, type, device);
    const size_t bytes = moe_matvec_workspace_bytes(t, K);
    at::Tensor ws;
    if (bytes) ws = empty({(int64_t)bytes}, at::kByte, device);
    call("moe_matvec_mxfp4", device, [&](moe_stream_t s) {
      return moe_matvec_mxfp4(px, w.data_ptr(), static_cast<const float*>(pb), t, rows, K, kind, act, code, out.data_ptr(),
                              address(ws), bytes, s);
    });
    return wrap(out);
  });
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error_class, cls);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(block_norm),   FAST(block_norm_backward),
                         FAST(ffn_forward),  FAST(ffn_backward),
                         FAST(matvec),       {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dense_ext", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dense_ext() { return PyModule_Create(&module); }
