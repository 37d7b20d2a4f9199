// rowops_bind.cpp -- the binding of the operators between the GEMMs: checks
// of tensors, allocation of outputs and scratch, and the calls of the C ABI.
//
// These calls take 3 to 20 us on the GPU, and a call made of Python
// statements 8 to 17 us (torch.empty 1.2 to 1.7 each, a view 0.8, the checks
// 2 to 3; a kernel launch 2.7), so the statements are here.  int8_gemm_amd
// documents the functions and gives them their defaults; it passes the C
// ABI's addresses to init(), with a function that gives torch's current
// stream of a device and one that raises I8GError for a status.
//
// Every function takes its arguments by position and returns tensors; what it
// refuses is a ValueError.  No HIP call is made here but by the C ABI.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/int8_gemm.h"
#include "i8g_overlap.h"

namespace {

// ---- the C ABI ----
struct Api {
  decltype(&::layer_norm) layer_norm;
  decltype(&::layer_norm_quantize_rows) layer_norm_quantize_rows;
  decltype(&::layer_norm_bwd) layer_norm_bwd;
  decltype(&::layer_norm_bwd_workspace_bytes) layer_norm_bwd_workspace_bytes;
  decltype(&::layer_norm_bwd_checkpoint) layer_norm_bwd_checkpoint;
  decltype(&::checkpoint_i8) checkpoint_i8;
  decltype(&::checkpoint_restore) checkpoint_restore;
  decltype(&::checkpoint_act_bwd) checkpoint_act_bwd;
  decltype(&::checkpoint_quantize_cols) checkpoint_quantize_cols;
  decltype(&::checkpoint_quantize_cols_workspace_bytes) checkpoint_quantize_cols_workspace_bytes;
  decltype(&::token_logprobs) token_logprobs;
  decltype(&::token_logprobs_workspace_bytes) token_logprobs_workspace_bytes;
  decltype(&::token_logprobs_bwd) token_logprobs_bwd;
} api;
PyObject* stream_of = nullptr;   // device index -> stream handle
PyObject* raise_status = nullptr;

// A Python error that has been set.
struct Failed {};
template <class... A>
[[noreturn]] void refuse(const char* format, A... args) {
  PyErr_Format(PyExc_ValueError, format, args...);
  throw Failed{};
}

// ---- checks ----
const at::Tensor& tensor_of(PyObject* o, const char* name, const char* what) {
  if (!THPVariable_Check(o)) refuse("%s must be %s", name, what);
  return THPVariable_Unpack(o);
}

// A matrix with unit column stride and rows that do not overlap, on the GPU.
struct Matrix {
  const at::Tensor* t;
  int64_t rows, cols, ld;
  void* data() const { return t->data_ptr(); }
};

void on_device(const at::Tensor& t, const char* name, const at::Tensor* like) {
  if (!t.is_cuda()) refuse("%s must be on a GPU", name);
  if (like && t.device() != like->device())
    refuse("%s must be on %s, got %s", name, like->device().str().c_str(), t.device().str().c_str());
}

Matrix layout(const at::Tensor& t, const char* name, const at::Tensor* like) {
  on_device(t, name, like);
  Matrix m{&t, t.size(0), t.size(1), 0};
  if (m.cols > 1 && m.rows > 0 && t.stride(1) != 1) refuse("%s must be row-major (unit column stride)", name);
  if (m.rows > 1 && t.stride(0) < m.cols) refuse("%s has overlapping rows (expanded?): call .contiguous() first", name);
  m.ld = m.rows > 1 ? t.stride(0) : m.cols > 1 ? m.cols : 1;
  return m;
}

// Where the elements of a matrix, and of a contiguous vector, are.
i8g::ByteRows bytes_of(const Matrix& m) {
  const int64_t size = (int64_t)m.t->element_size();
  return i8g::ByteRows{(uintptr_t)m.data(), m.rows, m.cols * size, m.ld * size};
}
i8g::ByteRows bytes_of(const at::Tensor& v) {
  const int64_t size = (int64_t)v.nbytes();
  return i8g::ByteRows{(uintptr_t)v.data_ptr(), 1, size, size};
}

uint32_t dtype_code(at::ScalarType s) {
  return s == at::kFloat ? I8G_F32 : s == at::kBFloat16 ? I8G_BF16 : s == at::kHalf ? I8G_F16 : 99u;
}

// Values in f32, bf16 or f16 (with `like`: of its dtype, shape and device).
Matrix values(PyObject* o, const char* name, const at::Tensor* like = nullptr) {
  const at::Tensor& t = tensor_of(o, name, "a 2-D tensor");
  if (t.dim() != 2) refuse("%s must be a 2-D tensor", name);
  if (dtype_code(t.scalar_type()) == 99u)
    refuse("%s must be float32, bfloat16 or float16, got %s", name, at::toString(t.scalar_type()));
  if (like && (t.scalar_type() != like->scalar_type() || t.sizes() != like->sizes()))
    refuse("%s must have the dtype and shape of the other values", name);
  return layout(t, name, like);
}

// The address of a contiguous f32 vector of n values (null for None).
float* vector(PyObject* o, int64_t n, const char* name, const at::Tensor& like, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  const at::Tensor& t = tensor_of(o, name, "a 1-D float32 tensor");
  if (t.scalar_type() != at::kFloat || t.dim() != 1 || t.numel() != n)
    refuse("%s must be a 1-D float32 tensor of %lld values", name, (long long)n);
  on_device(t, name, &like);
  if (!t.is_contiguous()) refuse("%s must be contiguous", name);
  return static_cast<float*>(t.data_ptr());
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Failed{};
  return v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Failed{};
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Failed{};
  return v != 0;
}

// An 8-bit checkpoint (with `like`: of its shape and device).
struct Ck {
  Matrix q;
  const int8_t* Q;
  const float* scale;
  int64_t lds;
  int32_t group;
};
Ck checkpoint(PyObject* q, PyObject* s, PyObject* g, const at::Tensor* like = nullptr) {
  const at::Tensor& Q = tensor_of(q, "Q", "a 2-D int8 tensor");
  if (Q.dim() != 2 || Q.scalar_type() != at::kChar) refuse("Q must be a 2-D int8 tensor");
  if (like && Q.sizes() != like->sizes()) refuse("Q must have the shape of the values");
  Ck c{layout(Q, "Q", like), nullptr, nullptr, 0, 0};
  const int64_t group = integer(g);
  if (group != 0 && group != 32 && group != 64 && group != 128 && group != 256)
    refuse("group must be 32, 64, 128 or 256, or 0 for one scale per row");
  const int64_t groups = group ? (c.q.cols + group - 1) / group : c.q.cols > 0 ? 1 : 0;
  const at::Tensor& S = tensor_of(s, "scale", "a float32 tensor");
  const bool by_group = S.dim() == 2 && S.size(0) == c.q.rows && S.size(1) == groups;
  const bool by_row = group == 0 && S.dim() == 1 && S.size(0) == c.q.rows;
  if (S.scalar_type() != at::kFloat || !(by_group || by_row))
    refuse("scale must be a float32 tensor of shape (%lld, %lld)%s", (long long)c.q.rows, (long long)groups,
           group ? "" : ", or of one value a row");
  on_device(S, "scale", &Q);
  if (by_group && groups > 1 && S.stride(1) != 1) refuse("scale must be row-major (unit column stride)");
  c.lds = c.q.rows > 1 ? S.stride(0) : groups > 1 ? groups : 1;
  if (c.lds < groups) refuse("scale has overlapping rows (expanded?): call .contiguous() first");
  c.Q = static_cast<const int8_t*>(Q.data_ptr());
  c.scale = static_cast<const float*>(S.data_ptr());
  c.group = (int32_t)group;
  return c;
}

// ---- outputs ----
at::Tensor fresh(at::IntArrayRef size, at::ScalarType type, const at::Tensor& like) {
  return at::empty(size, at::TensorOptions().dtype(type).device(like.device()));
}
at::Tensor floats(int64_t n, const at::Tensor& like) { return fresh({n}, at::kFloat, like); }
at::Tensor values_like(const Matrix& m) { return fresh({m.rows, m.cols}, m.t->scalar_type(), *m.t); }
int64_t ld_of(int64_t cols) { return cols > 1 ? cols : 1; }

// rows x cols codes in a buffer whose rows are padded to 16 bytes.
struct Codes {
  at::Tensor t;
  int64_t ld;
  int8_t* data() const { return static_cast<int8_t*>(t.data_ptr()); }
};
Codes codes(int64_t rows, int64_t cols, const at::Tensor& like) {
  const int64_t ld = cols > 16 ? (cols + 15) / 16 * 16 : 16;
  at::Tensor buf = fresh({rows, ld}, at::kChar, like);
  return Codes{ld == cols ? buf : buf.narrow(1, 0, cols), ld};
}
at::Tensor scratch(size_t bytes, const at::Tensor& like) { return fresh({(int64_t)bytes}, at::kByte, like); }

float* f32(const at::Tensor& t) { return t.defined() ? static_cast<float*>(t.data_ptr()) : nullptr; }
PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
template <class... T>
PyObject* tuple(const T&... t) {
  PyObject* items[] = {wrap(t)...};
  PyObject* r = PyTuple_New(sizeof...(t));
  for (size_t i = 0; i < sizeof...(t); ++i) {
    if (r && items[i]) PyTuple_SET_ITEM(r, (Py_ssize_t)i, items[i]);
    else if (items[i]) Py_DECREF(items[i]);
  }
  for (PyObject* o : items)
    if (!o) {
      Py_XDECREF(r);
      return nullptr;
    }
  return r;
}

// fn(args..., stream) on torch's current stream of the tensor's device.
template <class F, class... A>
void enqueue(F fn, const at::Tensor& like, A... args) {
  const c10::DeviceGuard guard(like.device());
  PyObject* index = PyLong_FromLong(like.device().index());
  PyObject* handle = index ? PyObject_CallOneArg(stream_of, index) : nullptr;
  Py_XDECREF(index);
  if (!handle) throw Failed{};
  void* stream = PyLong_AsVoidPtr(handle);
  Py_DECREF(handle);
  if (!stream && PyErr_Occurred()) throw Failed{};
  const int status = fn(args..., stream);
  if (status != I8G_OK) {
    PyObject* r = PyObject_CallFunction(raise_status, "i", status);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "int8_gemm status %d", status);
    throw Failed{};
  }
}

// ---- the functions ----
using Args = PyObject* const*;

PyObject* layer_norm_(Args a) {   // X, weight, bias, eps
  const Matrix x = values(a[0], "X");
  const float *w = vector(a[1], x.cols, "weight", *x.t, true), *b = vector(a[2], x.cols, "bias", *x.t, true);
  const double eps = real(a[3]);
  const at::Tensor y = values_like(x), mean = floats(x.rows, *x.t), rstd = floats(x.rows, *x.t);
  enqueue(api.layer_norm, *x.t, x.data(), dtype_code(x.t->scalar_type()), x.rows, x.cols, x.ld, w, b, eps,
          y.data_ptr(), ld_of(x.cols), f32(mean), f32(rstd));
  return tuple(y, mean, rstd);
}

PyObject* layer_norm_quantize_rows_(Args a) {   // X, weight, bias, eps
  const Matrix x = values(a[0], "X");
  const float *w = vector(a[1], x.cols, "weight", *x.t, true), *b = vector(a[2], x.cols, "bias", *x.t, true);
  const double eps = real(a[3]);
  const Codes q = codes(x.rows, x.cols, *x.t);
  const at::Tensor s = floats(x.rows, *x.t), mean = floats(x.rows, *x.t), rstd = floats(x.rows, *x.t);
  enqueue(api.layer_norm_quantize_rows, *x.t, x.data(), dtype_code(x.t->scalar_type()), x.rows, x.cols, x.ld, w, b,
          eps, q.data(), q.ld, f32(s), f32(mean), f32(rstd));
  return tuple(q.t, s, mean, rstd);
}

// dX, and with weight_grad the sums' outputs and scratch.
struct Grads {
  at::Tensor dx, dw, db, ws;
  size_t bytes = 0;
  Grads(const Matrix& dy, bool weight_grad) : dx(values_like(dy)) {
    if (!weight_grad) return;
    bytes = api.layer_norm_bwd_workspace_bytes(dy.rows, dy.cols);
    ws = scratch(bytes, *dy.t);
    dw = floats(dy.cols, *dy.t);
    db = floats(dy.cols, *dy.t);
  }
  void* work() const { return ws.defined() ? ws.data_ptr() : nullptr; }
};

PyObject* layer_norm_bwd_(Args a) {   // dY, X, mean, rstd, weight, weight_grad
  const Matrix dy = values(a[0], "dY"), x = values(a[1], "X", dy.t);
  const float *mean = vector(a[2], dy.rows, "mean", *dy.t), *rstd = vector(a[3], dy.rows, "rstd", *dy.t);
  const float* w = vector(a[4], dy.cols, "weight", *dy.t, true);
  const Grads g(dy, truth(a[5]));
  enqueue(api.layer_norm_bwd, *dy.t, dy.data(), dy.ld, x.data(), x.ld, dtype_code(dy.t->scalar_type()), dy.rows,
          dy.cols, w, mean, rstd, g.dx.data_ptr(), ld_of(dy.cols), f32(g.dw), f32(g.db), g.work(), g.bytes);
  return tuple(g.dx, g.dw, g.db);
}

PyObject* layer_norm_bwd_checkpoint_(Args a) {   // dY, Q, scale, group, mean, rstd, weight, weight_grad
  const Matrix dy = values(a[0], "dY");
  const Ck c = checkpoint(a[1], a[2], a[3], dy.t);
  const float *mean = vector(a[4], dy.rows, "mean", *dy.t), *rstd = vector(a[5], dy.rows, "rstd", *dy.t);
  const float* w = vector(a[6], dy.cols, "weight", *dy.t, true);
  const Grads g(dy, truth(a[7]));
  enqueue(api.layer_norm_bwd_checkpoint, *dy.t, dy.data(), dy.ld, dtype_code(dy.t->scalar_type()), c.Q, c.q.ld, c.scale,
          c.lds, c.group, dy.rows, dy.cols, w, mean, rstd, g.dx.data_ptr(), ld_of(dy.cols), f32(g.dw), f32(g.db),
          g.work(), g.bytes);
  return tuple(g.dx, g.dw, g.db);
}

PyObject* checkpoint_i8_(Args a) {   // X, group
  const Matrix x = values(a[0], "X");
  const int64_t group = integer(a[1]);
  if (group != 32 && group != 64 && group != 128 && group != 256) refuse("group must be 32, 64, 128 or 256");
  const int64_t groups = (x.cols + group - 1) / group;
  const Codes q = codes(x.rows, x.cols, *x.t);
  const at::Tensor s = fresh({x.rows, groups}, at::kFloat, *x.t);
  enqueue(api.checkpoint_i8, *x.t, x.data(), dtype_code(x.t->scalar_type()), x.rows, x.cols, x.ld, (int32_t)group,
          q.data(), q.ld, f32(s), groups);
  return tuple(q.t, s);
}

PyObject* checkpoint_restore_(Args a) {   // Q, scale, group, dtype code
  const Ck c = checkpoint(a[0], a[1], a[2]);
  const int64_t dtype = integer(a[3]);
  const at::ScalarType type = dtype == I8G_F32 ? at::kFloat : dtype == I8G_BF16 ? at::kBFloat16 : at::kHalf;
  const at::Tensor y = fresh({c.q.rows, c.q.cols}, type, *c.q.t);
  enqueue(api.checkpoint_restore, *c.q.t, c.Q, c.q.ld, c.scale, c.lds, c.group, c.q.rows, c.q.cols, y.data_ptr(),
          (uint32_t)dtype, ld_of(c.q.cols));
  return wrap(y);
}

PyObject* checkpoint_act_bwd_(Args a) {   // dY, Q, scale, group, act code
  const Matrix dy = values(a[0], "dY");
  const Ck c = checkpoint(a[1], a[2], a[3], dy.t);
  const int64_t act = integer(a[4]);
  const at::Tensor dx = values_like(dy);
  enqueue(api.checkpoint_act_bwd, *dy.t, c.Q, c.q.ld, c.scale, c.lds, c.group, dy.rows, dy.cols, (uint32_t)act,
          dy.data(), dy.ld, dx.data_ptr(), ld_of(dy.cols), dtype_code(dy.t->scalar_type()));
  return wrap(dx);
}

PyObject* checkpoint_quantize_cols_(Args a) {   // Q, scale, group
  const Ck c = checkpoint(a[0], a[1], a[2]);
  const Codes qt = codes(c.q.cols, c.q.rows, *c.q.t);
  const at::Tensor s = floats(c.q.cols, *c.q.t);
  const size_t bytes = api.checkpoint_quantize_cols_workspace_bytes(c.q.rows, c.q.cols);
  const at::Tensor ws = scratch(bytes, *c.q.t);
  enqueue(api.checkpoint_quantize_cols, *c.q.t, c.Q, c.q.ld, c.scale, c.lds, c.group, c.q.rows, c.q.cols, qt.data(),
          qt.ld, f32(s), ws.data_ptr(), bytes);
  return tuple(qt.t, s);
}

const int64_t* targets(PyObject* o, int64_t rows, const at::Tensor& like) {
  const at::Tensor& t = tensor_of(o, "targets", "a 1-D int64 tensor");
  if (t.scalar_type() != at::kLong || t.dim() != 1 || t.numel() != rows)
    refuse("targets must be a 1-D int64 tensor of %lld token numbers", (long long)rows);
  on_device(t, "targets", &like);
  if (!t.is_contiguous()) refuse("targets must be contiguous");
  return static_cast<const int64_t*>(t.data_ptr());
}

PyObject* token_logprobs_(Args a) {   // logits, targets, topk
  const Matrix x = values(a[0], "logits");
  const int64_t* t = targets(a[1], x.rows, *x.t);
  const int64_t topk = integer(a[2]);
  if (topk < 0 || topk > I8G_TOPK_MAX || (x.rows > 0 && topk > x.cols))
    refuse("topk must be between 0 and min(%d, %lld), got %lld", I8G_TOPK_MAX, (long long)x.cols, (long long)topk);
  const at::Tensor lp = floats(x.rows, *x.t), h = floats(x.rows, *x.t), lse = floats(x.rows, *x.t);
  at::Tensor index, top, ws;
  if (topk > 0) {
    index = fresh({x.rows, topk}, at::kInt, *x.t);
    top = fresh({x.rows, topk}, at::kFloat, *x.t);
  }
  const size_t bytes = api.token_logprobs_workspace_bytes(x.rows, x.cols, (int32_t)topk);
  if (bytes > 0) ws = scratch(bytes, *x.t);
  enqueue(api.token_logprobs, *x.t, x.data(), dtype_code(x.t->scalar_type()), x.rows, x.cols, x.ld, t, (int32_t)topk,
          f32(lp), f32(h), f32(lse), index.defined() ? static_cast<int32_t*>(index.data_ptr()) : nullptr, f32(top),
          ws.defined() ? ws.data_ptr() : nullptr, bytes);
  return tuple(lp, h, lse, index, top);
}

PyObject* token_logprobs_bwd_(Args a) {   // logits, targets, lse, entropy, g_logprob, g_entropy, out
  const Matrix x = values(a[0], "logits");
  const int64_t* t = a[1] == Py_None ? nullptr : targets(a[1], x.rows, *x.t);
  if (a[4] == Py_None && a[5] == Py_None) refuse("g_logprob or g_entropy is needed");
  if (a[4] != Py_None && a[1] == Py_None) refuse("targets are needed with g_logprob");
  if (a[5] != Py_None && a[3] == Py_None) refuse("entropy is needed with g_entropy");
  const float *lse = vector(a[2], x.rows, "lse", *x.t), *h = vector(a[3], x.rows, "entropy", *x.t, true);
  const float *g = vector(a[4], x.rows, "g_logprob", *x.t, true), *gh = vector(a[5], x.rows, "g_entropy", *x.t, true);
  at::Tensor dx;
  Matrix out{nullptr, 0, 0, 0};
  if (a[6] == Py_None) {
    dx = values_like(x);
    out = Matrix{&dx, x.rows, x.cols, ld_of(x.cols)};
  } else {
    out = values(a[6], "out", x.t);
    dx = *out.t;
    if (!i8g::itself_or_apart(bytes_of(out), bytes_of(x)))
      refuse("out must be the logits themselves or not overlap them");
    static const char* const names[] = {"targets", "lse", "entropy", "g_logprob", "g_entropy"};
    for (int i = 0; i < 5; ++i)
      if (a[i + 1] != Py_None && i8g::share_bytes(bytes_of(out), bytes_of(THPVariable_Unpack(a[i + 1]))))
        refuse("out must not overlap %s", names[i]);
  }
  enqueue(api.token_logprobs_bwd, *x.t, x.data(), dtype_code(x.t->scalar_type()), x.rows, x.cols, x.ld, t, lse, h, g, gh,
          out.data(), out.ld);
  return wrap(dx);
}

template <PyObject* (*F)(Args), int N>
PyObject* entry(PyObject*, Args args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments are needed, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Failed&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// init({name: address}, stream of a device, raise for a status)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 3 || !PyDict_Check(a[0])) {
    PyErr_SetString(PyExc_TypeError, "init(addresses, stream_of, raise_status)");
    return nullptr;
  }
  bool ok = true;
  auto take = [&](auto& f, const char* name) {
    PyObject* v = PyDict_GetItemString(a[0], name);
    void* p = v ? PyLong_AsVoidPtr(v) : nullptr;
    if (!p) {
      if (!PyErr_Occurred()) PyErr_Format(PyExc_KeyError, "no address of %s", name);
      ok = false;
      return;
    }
    f = reinterpret_cast<std::decay_t<decltype(f)>>(p);
  };
#define TAKE(name) if (ok) take(api.name, #name)
  TAKE(layer_norm); TAKE(layer_norm_quantize_rows); TAKE(layer_norm_bwd); TAKE(layer_norm_bwd_workspace_bytes);
  TAKE(layer_norm_bwd_checkpoint); TAKE(checkpoint_i8); TAKE(checkpoint_restore); TAKE(checkpoint_act_bwd);
  TAKE(checkpoint_quantize_cols); TAKE(checkpoint_quantize_cols_workspace_bytes); TAKE(token_logprobs);
  TAKE(token_logprobs_workspace_bytes); TAKE(token_logprobs_bwd);
#undef TAKE
  if (!ok) return nullptr;
  Py_INCREF(a[1]);
  Py_INCREF(a[2]);
  stream_of = a[1];
  raise_status = a[2];
  Py_RETURN_NONE;
}

#define ENTRY(name, n) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name##_, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&init)), METH_FASTCALL, nullptr},
    ENTRY(layer_norm, 4),
    ENTRY(layer_norm_quantize_rows, 4),
    ENTRY(layer_norm_bwd, 6),
    ENTRY(layer_norm_bwd_checkpoint, 8),
    ENTRY(checkpoint_i8, 2),
    ENTRY(checkpoint_restore, 4),
    ENTRY(checkpoint_act_bwd, 5),
    ENTRY(checkpoint_quantize_cols, 3),
    ENTRY(token_logprobs, 3),
    ENTRY(token_logprobs_bwd, 7),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "rowops_bind", "Binding of the operators between the GEMMs.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit_rowops_bind(void) { return PyModule_Create(&module); }
