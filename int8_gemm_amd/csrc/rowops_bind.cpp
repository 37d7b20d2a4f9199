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
  decltype(&::gemm_i8_logprobs) gemm_i8_logprobs;
  decltype(&::gemm_i8_logprobs_workspace_bytes) gemm_i8_logprobs_workspace_bytes;
  decltype(&::gemm_i8_logprobs_bwd) gemm_i8_logprobs_bwd;
  decltype(&::gemm_i8_logprobs_bwd_workspace_bytes) gemm_i8_logprobs_bwd_workspace_bytes;
  decltype(&::embedding) embedding;
  decltype(&::embedding_i8) embedding_i8;
  decltype(&::embedding_bwd) embedding_bwd;
  decltype(&::embedding_bwd_workspace_bytes) embedding_bwd_workspace_bytes;
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

// A contiguous int64 vector of `rows` numbers.
const int64_t* numbers(PyObject* o, const char* name, const char* what, int64_t rows, const at::Tensor& like) {
  const at::Tensor& t = tensor_of(o, name, "a 1-D int64 tensor");
  if (t.scalar_type() != at::kLong || t.dim() != 1 || t.numel() != rows)
    refuse("%s must be a 1-D int64 tensor of %lld %s numbers", name, (long long)rows, what);
  on_device(t, name, &like);
  if (!t.is_contiguous()) refuse("%s must be contiguous", name);
  return static_cast<const int64_t*>(t.data_ptr());
}
const int64_t* targets(PyObject* o, int64_t rows, const at::Tensor& like) { return numbers(o, "targets", "token", rows, like); }

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

// The operands of the LM head's product.
struct Head {
  Matrix a, b;
  const float *s_row, *s_col;
  int64_t lda, ldb;
  const int8_t* A() const { return static_cast<const int8_t*>(a.data()); }
  const int8_t* B() const { return static_cast<const int8_t*>(b.data()); }
};
Matrix int8_matrix(PyObject* o, const char* name, const at::Tensor* like) {
  const at::Tensor& t = tensor_of(o, name, "a 2-D int8 tensor");
  if (t.dim() != 2 || t.scalar_type() != at::kChar) refuse("%s must be a 2-D int8 tensor", name);
  return layout(t, name, like);
}
// The stride of a single row of codes says how much of it may be read, a multiple
// of 16 bytes; whole 16s need no more than the row itself.
int64_t code_ld(const Matrix& m) {
  if (m.rows > 1) return m.ld;
  const int64_t k16 = (m.cols + 15) / 16 * 16;
  return m.rows == 0 || m.cols == k16 ? k16 : m.t->stride(0);
}
Head head(Args a) {   // QA, s_row, QBt, s_col
  Head h{int8_matrix(a[0], "QA", nullptr), {}, nullptr, nullptr, 0, 0};
  h.b = int8_matrix(a[2], "QBt", h.a.t);
  if (h.a.cols != h.b.cols) refuse("K mismatch: QA has %lld, QBt has %lld", (long long)h.a.cols, (long long)h.b.cols);
  if (h.b.rows == 0 && h.a.rows > 0) refuse("QBt has no rows");
  h.s_row = vector(a[1], h.a.rows, "s_row", *h.a.t);
  h.s_col = vector(a[3], h.b.rows, "s_col", *h.a.t);
  h.lda = code_ld(h.a);
  h.ldb = code_ld(h.b);
  return h;
}

PyObject* gemm_i8_logprobs_(Args a) {   // QA, s_row, QBt, s_col, targets
  const Head h = head(a);
  const at::Tensor& like = *h.a.t;
  const int64_t* t = targets(a[4], h.a.rows, like);
  const at::Tensor lp = floats(h.a.rows, like), lse = floats(h.a.rows, like);
  const size_t bytes = api.gemm_i8_logprobs_workspace_bytes(h.a.rows, h.b.rows, h.a.cols);
  const at::Tensor ws = scratch(bytes, like);
  enqueue(api.gemm_i8_logprobs, like, h.A(), h.lda, h.s_row, h.B(), h.ldb, h.s_col, h.a.rows, h.b.rows, h.a.cols, t, f32(lp),
          f32(lse), ws.data_ptr(), bytes);
  return tuple(lp, lse);
}

PyObject* gemm_i8_logprobs_bwd_(Args a) {   // QA, s_row, QBt, s_col, targets, lse, g_logprob, g_lse, dtype code
  const Head h = head(a);
  const at::Tensor& like = *h.a.t;
  if (a[6] == Py_None && a[7] == Py_None) refuse("g_logprob or g_lse is needed");
  if (a[6] != Py_None && a[4] == Py_None) refuse("targets are needed with g_logprob");
  const int64_t* t = a[4] == Py_None ? nullptr : targets(a[4], h.a.rows, like);
  const float* lse = vector(a[5], h.a.rows, "lse", like);
  const float *g = vector(a[6], h.a.rows, "g_logprob", like, true), *gl = vector(a[7], h.a.rows, "g_lse", like, true);
  const int64_t dtype = integer(a[8]);
  const at::ScalarType type = dtype == I8G_F32 ? at::kFloat : dtype == I8G_BF16 ? at::kBFloat16 : at::kHalf;
  const at::Tensor da = fresh({h.a.rows, h.a.cols}, type, like), db = fresh({h.b.rows, h.b.cols}, type, like);
  const size_t bytes = api.gemm_i8_logprobs_bwd_workspace_bytes(h.a.rows, h.b.rows, h.a.cols, (uint32_t)dtype);
  const at::Tensor ws = scratch(bytes, like);
  enqueue(api.gemm_i8_logprobs_bwd, like, h.A(), h.lda, h.s_row, h.B(), h.ldb, h.s_col, h.a.rows, h.b.rows, h.a.cols, t, lse, g,
          gl, da.data_ptr(), ld_of(h.a.cols), db.data_ptr(), ld_of(h.a.cols), (uint32_t)dtype, ws.data_ptr(), bytes);
  return tuple(da, db);
}

int64_t token_count(PyObject* o) {
  const at::Tensor& t = tensor_of(o, "tokens", "a 1-D int64 tensor");
  if (t.dim() != 1) refuse("tokens must be a 1-D int64 tensor");
  return t.numel();
}

// pos_table and positions, of a type and as many columns as the output.
struct Positions {
  Matrix p{nullptr, 0, 0, 0};
  const int64_t* at = nullptr;
  Positions(PyObject* table, PyObject* numbers_of, int64_t rows, int64_t cols, at::ScalarType type, const at::Tensor& like) {
    if ((table == Py_None) != (numbers_of == Py_None)) refuse("pos_table and positions go together");
    if (table == Py_None) return;
    p = values(table, "pos_table");
    on_device(*p.t, "pos_table", &like);
    if (p.t->scalar_type() != type || p.cols != cols)
      refuse("pos_table must have %lld columns of %s", (long long)cols, at::toString(type));
    at = numbers(numbers_of, "positions", "position", rows, like);
  }
  const void* data() const { return p.t ? p.data() : nullptr; }
};

PyObject* embedding_(Args a) {   // table, tokens, alpha, pos_table, positions
  const Matrix w = values(a[0], "table");
  const int64_t rows = token_count(a[1]);
  const int64_t* t = numbers(a[1], "tokens", "token", rows, *w.t);
  const float alpha = (float)real(a[2]);
  const at::ScalarType type = w.t->scalar_type();
  const Positions p(a[3], a[4], rows, w.cols, type, *w.t);
  const at::Tensor y = fresh({rows, w.cols}, type, *w.t);
  enqueue(api.embedding, *w.t, w.data(), dtype_code(type), w.rows, w.cols, w.ld, t, rows, alpha, p.data(), p.p.rows, p.p.ld, p.at,
          y.data_ptr(), ld_of(w.cols));
  return wrap(y);
}

PyObject* embedding_i8_(Args a) {   // Q, scale, tokens, alpha, pos_table, positions, dtype code
  const Matrix q = int8_matrix(a[0], "Q", nullptr);
  const float* s = vector(a[1], q.rows, "scale", *q.t);
  const int64_t rows = token_count(a[2]);
  const int64_t* t = numbers(a[2], "tokens", "token", rows, *q.t);
  const float alpha = (float)real(a[3]);
  const int64_t dtype = integer(a[6]);
  const at::ScalarType type = dtype == I8G_F32 ? at::kFloat : dtype == I8G_BF16 ? at::kBFloat16 : at::kHalf;
  const Positions p(a[4], a[5], rows, q.cols, type, *q.t);
  const at::Tensor y = fresh({rows, q.cols}, type, *q.t);
  enqueue(api.embedding_i8, *q.t, static_cast<const int8_t*>(q.data()), q.ld, s, q.rows, q.cols, t, rows, alpha, p.data(),
          p.p.rows, p.p.ld, p.at, y.data_ptr(), (uint32_t)dtype, ld_of(q.cols));
  return wrap(y);
}

Matrix f32_matrix(PyObject* o, const char* name, int64_t rows, int64_t cols, const at::Tensor& like) {
  const at::Tensor& t = tensor_of(o, name, "a 2-D float32 tensor");
  if (t.dim() != 2 || t.scalar_type() != at::kFloat || t.size(0) != rows || t.size(1) != cols)
    refuse("%s must be a float32 tensor of shape (%lld, %lld)", name, (long long)rows, (long long)cols);
  return layout(t, name, &like);
}

PyObject* embedding_bwd_(Args a) {   // dY, tokens, vocab, alpha, add, out
  const Matrix dy = values(a[0], "dY");
  const int64_t* t = numbers(a[1], "tokens", "token", dy.rows, *dy.t);
  const int64_t vocab = integer(a[2]);
  if (vocab < 0 || vocab > INT32_MAX) refuse("vocab must be between 0 and 2^31 - 1, got %lld", (long long)vocab);
  const float alpha = (float)real(a[3]);
  Matrix add{nullptr, 0, 0, 0}, out{nullptr, 0, 0, 0};
  if (a[4] != Py_None) add = f32_matrix(a[4], "add", vocab, dy.cols, *dy.t);
  at::Tensor dw;
  if (a[5] == Py_None) {
    dw = fresh({vocab, dy.cols}, at::kFloat, *dy.t);
    out = Matrix{&dw, vocab, dy.cols, ld_of(dy.cols)};
  } else {
    out = f32_matrix(a[5], "out", vocab, dy.cols, *dy.t);
    dw = *out.t;
    if (add.t && !i8g::itself_or_apart(bytes_of(out), bytes_of(add))) refuse("out must be `add` itself or not overlap it");
    if (i8g::share_bytes(bytes_of(out), bytes_of(dy)) || i8g::share_bytes(bytes_of(out), bytes_of(THPVariable_Unpack(a[1]))))
      refuse("out must not overlap dY or tokens");
  }
  const size_t bytes = api.embedding_bwd_workspace_bytes(dy.rows, dy.cols);
  const at::Tensor ws = scratch(bytes, *dy.t);
  enqueue(api.embedding_bwd, *dy.t, dy.data(), dtype_code(dy.t->scalar_type()), dy.rows, dy.cols, dy.ld, t, vocab, alpha,
          add.t ? static_cast<const float*>(add.data()) : nullptr, add.ld, static_cast<float*>(out.data()), out.ld,
          ws.data_ptr(), bytes);
  return wrap(dw);
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
  TAKE(token_logprobs_workspace_bytes); TAKE(token_logprobs_bwd); TAKE(gemm_i8_logprobs);
  TAKE(gemm_i8_logprobs_workspace_bytes); TAKE(gemm_i8_logprobs_bwd); TAKE(gemm_i8_logprobs_bwd_workspace_bytes);
  TAKE(embedding); TAKE(embedding_i8); TAKE(embedding_bwd); TAKE(embedding_bwd_workspace_bytes);
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
    ENTRY(gemm_i8_logprobs, 5),
    ENTRY(gemm_i8_logprobs_bwd, 9),
    ENTRY(embedding, 5),
    ENTRY(embedding_i8, 7),
    ENTRY(embedding_bwd, 6),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "rowops_bind", "Binding of the operators between the GEMMs.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit_rowops_bind(void) { return PyModule_Create(&module); }
