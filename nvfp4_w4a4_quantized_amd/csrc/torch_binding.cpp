// Marshalling of the key/value cache calls from torch tensors to the C ABI.
//
// These are called once per layer and token while serving, where the ctypes path's ~12
// microseconds a call (attribute reads and argument conversions in Python) was longer than
// the kernels.  Here a call reads its tensors directly; checks and errors are those of the
// Python binding: every function returns None or (status, message).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <exception>

#include "../../include/nvfp4.h"

namespace {

struct Refusal {
  int status;
  char text[240];
};

[[noreturn]] void refuse(int status, const char* fmt, ...) {
  Refusal r;
  r.status = status;
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(r.text, sizeof(r.text), fmt, ap);
  va_end(ap);
  throw r;
}

PyObject* pair(int status, const char* text) { return Py_BuildValue("(is)", status, text); }

// The call's arguments, taken in order.
class Args {
 public:
  Args(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : a_(a) {
    if (n != want) refuse(NVFP4_ERR_INVALID_ARG, "%zd arguments, %zd expected", n, want);
    device_ = (int)number("device");
    stream_ = reinterpret_cast<void*>((uintptr_t)number("stream"));
  }

  int64_t number(const char* name) {
    const long long v = PyLong_AsLongLong(a_[i_]);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      refuse(NVFP4_ERR_INVALID_ARG, "%s must be a whole number", name);
    }
    ++i_;
    return v;
  }

  // None: `otherwise`
  double real(const char* name, double otherwise) {
    if (a_[i_] == Py_None) {
      ++i_;
      return otherwise;
    }
    const double v = PyFloat_AsDouble(a_[i_]);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      refuse(NVFP4_ERR_INVALID_ARG, "%s must be a number", name);
    }
    ++i_;
    return v;
  }

  int32_t small(const char* name) {
    const int64_t v = number(name);
    if (v < INT32_MIN || v > INT32_MAX) refuse(NVFP4_ERR_INVALID_ARG, "%s=%lld is out of range", name, (long long)v);
    return (int32_t)v;
  }

  // A tensor on the current device; NULL for None where that is allowed.
  const at::Tensor* tensor(const char* name, bool optional = false) {
    PyObject* o = a_[i_++];
    if (o == Py_None) {
      if (!optional) refuse(NVFP4_ERR_INVALID_ARG, "%s is None", name);
      return nullptr;
    }
    if (!THPVariable_Check(o)) refuse(NVFP4_ERR_INVALID_ARG, "%s must be a tensor", name);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse(NVFP4_ERR_INVALID_ARG, "%s must be in device memory", name);
    if (t.get_device() != device_)
      refuse(NVFP4_ERR_INVALID_ARG, "%s is on device %d, not the current device %d", name, (int)t.get_device(), device_);
    return &t;
  }

  void* stream() const { return stream_; }

 private:
  PyObject* const* a_;
  Py_ssize_t i_ = 0;
  int device_;
  void* stream_;
};

struct Rows {
  void* p = nullptr;
  int64_t rows = 0, cols = 0, ld = 0;
};

// The stride of a dimension of one element means nothing (torch gives it any value).
Rows rows_of(const at::Tensor* t, const char* name) {
  if (!t) return {};
  if (t->dim() != 2 || (t->size(1) > 1 && t->stride(1) != 1))
    refuse(NVFP4_ERR_INVALID_ARG, "%s must be 2-D with unit column stride", name);
  return {t->data_ptr(), t->size(0), t->size(1), t->size(0) == 1 ? t->size(1) : t->stride(0)};
}

int dtype_of(const at::Tensor* t, const char* name) {
  if (t->scalar_type() == at::kFloat) return NVFP4_DTYPE_F32;
  if (t->scalar_type() == at::kBFloat16) return NVFP4_DTYPE_BF16;
  refuse(NVFP4_ERR_UNSUPPORTED, "dtype of %s is not float32 or bfloat16", name);
}

void same_dtype(const at::Tensor* t, int dtype, const char* name) {
  if (t && dtype_of(t, name) != dtype) refuse(NVFP4_ERR_UNSUPPORTED, "%s must have the others' dtype", name);
}

template <typename T>
T* indices(const at::Tensor* t, at::ScalarType type, const char* type_name, int64_t n, const char* name) {
  if (!t) return nullptr;
  if (t->scalar_type() != type || t->dim() != 1 || t->size(0) != n || !t->is_contiguous())
    refuse(NVFP4_ERR_INVALID_ARG, "%s must be contiguous %s [%lld]", name, type_name, (long long)n);
  return static_cast<T*>(t->data_ptr());
}

// The cache buffer and its global scales; the head dimension follows from the page's
// bytes (9/8 byte per token, head and element).
struct Cache {
  uint8_t* p;
  int64_t pages;
  int32_t page_size, heads, d;
  const float *kg, *vg;
};

Cache cache_of(Args& a) {
  const at::Tensor* t = a.tensor("cache");
  const at::Tensor* kg = a.tensor("k_gscale");
  const at::Tensor* vg = a.tensor("v_gscale");
  Cache c;
  c.page_size = a.small("page_size");
  if (t->scalar_type() != at::kByte || t->dim() != 2 || !t->is_contiguous())
    refuse(NVFP4_ERR_INVALID_ARG, "cache must be contiguous uint8 [n_pages, page bytes]");
  const int64_t heads = kg->dim() == 1 ? kg->size(0) : -1;
  c.kg = indices<float>(kg, at::kFloat, "float32", heads, "k_gscale");
  c.vg = indices<float>(vg, at::kFloat, "float32", heads, "v_gscale");
  const int64_t bytes = t->size(1), per = 9 * heads * c.page_size;
  const int64_t d = heads > 0 && c.page_size > 0 ? bytes * 8 / per : 0;
  if (d <= 0 || d > 65536 || heads > 65536 || per * d != bytes * 8)
    refuse(NVFP4_ERR_INVALID_ARG, "cache pages of %lld bytes do not hold %d tokens of %lld heads", (long long)bytes,
           c.page_size, (long long)heads);
  c.p = static_cast<uint8_t*>(t->data_ptr());
  c.pages = t->size(0);
  c.heads = (int32_t)heads;
  c.d = (int32_t)d;
  return c;
}

PyObject* done(int status) {
  if (status != NVFP4_OK) return pair(status, nvfp4_last_error());
  Py_RETURN_NONE;
}

template <int (*F)(Args&), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    Args args(a, n, N);
    return done(F(args));
  } catch (const Refusal& r) {
    return pair(r.status, r.text);
  } catch (const std::exception& e) {
    return pair(NVFP4_ERR_INVALID_ARG, e.what());
  }
}

// device, stream, cache, k_gscale, v_gscale, page_size, q, k, v, cos, sin, positions, slots, q_out, interleaved
int rope_append_kv(Args& a) {
  const Cache c = cache_of(a);
  const at::Tensor *tq = a.tensor("q", true), *tk = a.tensor("k"), *tv = a.tensor("v");
  const at::Tensor *cos = a.tensor("cos", true), *sin = a.tensor("sin", true);
  const at::Tensor *pos = a.tensor("positions"), *slots = a.tensor("slots"), *to = a.tensor("q_out", true);
  const int32_t interleaved = a.small("interleaved");
  const Rows q = rows_of(tq, "q"), k = rows_of(tk, "k"), v = rows_of(tv, "v"), o = rows_of(to, "q_out");
  const int64_t kv_cols = (int64_t)c.heads * c.d;
  if (v.rows != k.rows || k.cols != kv_cols || v.cols != kv_cols)
    refuse(NVFP4_ERR_INVALID_ARG, "k and v must both be [T, %lld]: %d heads of %d", (long long)kv_cols, c.heads, c.d);
  const int dtype = dtype_of(tk, "k");
  same_dtype(tv, dtype, "v");
  if (!tq != !to) refuse(NVFP4_ERR_INVALID_ARG, "q and q_out must both be given or both be None");
  if (tq) {
    if (q.rows != k.rows || o.rows != k.rows || o.cols != q.cols || q.cols % c.d || q.cols / c.d > INT32_MAX)
      refuse(NVFP4_ERR_INVALID_ARG, "q and q_out must be [%lld, n_q_heads * %d]", (long long)k.rows, c.d);
    same_dtype(tq, dtype, "q");
    same_dtype(to, dtype, "q_out");
  }
  if (!cos != !sin) refuse(NVFP4_ERR_INVALID_ARG, "cos and sin must both be given or both be None");
  int64_t n_pos = 0, half = 0;
  if (cos) {
    if (cos->scalar_type() != at::kFloat || sin->scalar_type() != at::kFloat || cos->dim() != 2 || sin->dim() != 2 ||
        cos->size(0) != sin->size(0) || cos->size(1) != sin->size(1) || !cos->is_contiguous() || !sin->is_contiguous())
      refuse(NVFP4_ERR_INVALID_ARG, "cos and sin must be contiguous float32 [n_pos, rot_dim / 2]");
    n_pos = cos->size(0);
    half = cos->size(1);
    if (2 * half > c.d) refuse(NVFP4_ERR_INVALID_ARG, "rot_dim=%lld exceeds the head's %d", (long long)(2 * half), c.d);
  }
  return nvfp4_rope_append_kv(
      q.p, q.ld, k.p, k.ld, v.p, v.ld, dtype, k.rows, (int32_t)(q.cols / c.d), c.heads, c.d,
      cos ? static_cast<const float*>(cos->data_ptr()) : nullptr,
      sin ? static_cast<const float*>(sin->data_ptr()) : nullptr, n_pos, (int32_t)(2 * half), interleaved,
      indices<int32_t>(pos, at::kInt, "int32", k.rows, "positions"),
      indices<int64_t>(slots, at::kLong, "int64", k.rows, "slots"), c.p, c.pages, c.page_size, c.kg, c.vg, o.p, o.ld,
      a.stream());
}

// device, stream, cache, k_gscale, v_gscale, page_size, slots, k_out, v_out
int kv_gather(Args& a) {
  const Cache c = cache_of(a);
  const at::Tensor *slots = a.tensor("slots"), *tk = a.tensor("k_out"), *tv = a.tensor("v_out");
  const Rows k = rows_of(tk, "k_out"), v = rows_of(tv, "v_out");
  const int64_t cols = (int64_t)c.heads * c.d;
  if (v.rows != k.rows || k.cols != cols || v.cols != cols)
    refuse(NVFP4_ERR_INVALID_ARG, "k_out and v_out must both be [T, %lld]", (long long)cols);
  const int dtype = dtype_of(tk, "k_out");
  same_dtype(tv, dtype, "v_out");
  return nvfp4_kv_gather(c.p, c.pages, c.page_size, c.heads, c.d, c.kg, c.vg,
                         indices<int64_t>(slots, at::kLong, "int64", k.rows, "slots"), k.rows, k.p, k.ld, v.p, v.ld,
                         dtype, a.stream());
}

// device, stream, cache, k_gscale, v_gscale, page_size, q, page_table, kv_len, o, max_kv_len, workspace, cu_q,
// max_q_len, scale (None: 1/sqrt(d)), window, lse
int kv_attention(Args& a) {
  const Cache c = cache_of(a);
  const at::Tensor *tq = a.tensor("q"), *table = a.tensor("page_table"), *kv_len = a.tensor("kv_len"),
                   *to = a.tensor("o");
  const int64_t max_kv_len = a.number("max_kv_len");
  const at::Tensor *ws = a.tensor("workspace", true), *cu = a.tensor("cu_q", true);
  const int64_t max_q_len = a.number("max_q_len");
  const double scale = a.real("scale", 1.0 / std::sqrt((double)c.d));
  const int32_t window = a.small("window");
  const at::Tensor* lse = a.tensor("lse", true);
  const Rows q = rows_of(tq, "q"), o = rows_of(to, "o");
  if (o.rows != q.rows || o.cols != q.cols || q.cols % c.d || q.cols / c.d > INT32_MAX)
    refuse(NVFP4_ERR_INVALID_ARG, "q and o must both be [T, n_q_heads * %d]", c.d);
  const int dtype = dtype_of(tq, "q");
  same_dtype(to, dtype, "o");
  const int64_t heads = q.cols / c.d;
  if (table->scalar_type() != at::kInt) refuse(NVFP4_ERR_UNSUPPORTED, "page_table must be int32");
  const Rows tab = rows_of(table, "page_table");
  if (tab.rows > INT32_MAX - 1) refuse(NVFP4_ERR_INVALID_ARG, "too many sequences");
  if (lse && (lse->scalar_type() != at::kFloat || lse->dim() != 2 || lse->size(0) != q.rows ||
              lse->size(1) != heads || !lse->is_contiguous()))
    refuse(NVFP4_ERR_INVALID_ARG, "lse must be contiguous float32 [%lld, %lld]", (long long)q.rows, (long long)heads);
  if (ws && !ws->is_contiguous()) refuse(NVFP4_ERR_INVALID_ARG, "workspace must be contiguous");
  return nvfp4_kv_attention(
      q.p, dtype, q.ld, q.rows, (int32_t)heads, c.heads, c.d, (int32_t)tab.rows,
      indices<int32_t>(cu, at::kInt, "int32", tab.rows + 1, "cu_q"), max_q_len,
      indices<int32_t>(kv_len, at::kInt, "int32", tab.rows, "kv_len"), max_kv_len,
      static_cast<const int32_t*>(tab.p), tab.cols, tab.ld, c.p, c.pages, c.page_size, c.kg, c.vg,
      (float)scale, window, o.p, o.ld,
      lse ? static_cast<float*>(lse->data_ptr()) : nullptr, ws ? ws->data_ptr() : nullptr,
      ws ? (int64_t)(ws->numel() * ws->element_size()) : 0, a.stream());
}

PyMethodDef methods[] = {
    {"rope_append_kv", reinterpret_cast<PyCFunction>(entry<rope_append_kv, 15>), METH_FASTCALL, nullptr},
    {"kv_gather", reinterpret_cast<PyCFunction>(entry<kv_gather, 9>), METH_FASTCALL, nullptr},
    {"kv_attention", reinterpret_cast<PyCFunction>(entry<kv_attention, 17>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_binding(void) { return PyModule_Create(&module); }
