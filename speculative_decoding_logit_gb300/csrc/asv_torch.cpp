// asv_torch.cpp -- the paged-cache calls of the Python binding, and the sampling's: checks of the tensors and their
// marshalling to the C entry points, in C++ because they are made for every layer of every step (as Python code over
// ctypes the first two took 6 us a call, of 10 in all).  A CPython module: asv_torch.paged_attention(...),
// paged_kv_append(...) and so on, positional arguments only; failures raise the binding's AsvError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <exception>
#include <initializer_list>
#include <type_traits>

#include "asv.h"

namespace {

PyObject* g_error = nullptr;  // AsvError(status, message)
decltype(&paged_attention) g_attention = nullptr;
decltype(&paged_kv_append) g_append = nullptr;
decltype(&paged_kv_append_ex) g_append_ex = nullptr;
decltype(&paged_plan) g_plan = nullptr;
decltype(&sample_tokens) g_sample = nullptr;
decltype(&asv_status_string) g_status_string = nullptr;
decltype(&asv_last_cuda_error) g_last_cuda_error = nullptr;

struct Refused {
  int status;
  char text[256];
};

[[noreturn]] void refuse(int status, const char* format, ...) {
  Refused r;
  r.status = status;
  va_list ap;
  va_start(ap, format);
  std::vsnprintf(r.text, sizeof(r.text), format, ap);
  va_end(ap);
  throw r;
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(ASV_ERR_SHAPE, "%s must be a tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse(-1, "inputs must be CUDA tensors (the library has no CPU path); %s is not", name);
  return t;
}

int extent(int64_t n, const char* what) {
  if (n > 0x7fffffff) refuse(ASV_ERR_SHAPE, "%s does not fit 32 bits", what);
  return int(n);
}

// int32 and contiguous, [n]
const int32_t* lengths(const at::Tensor& t, const char* name, int64_t n) {
  if (t.scalar_type() != at::kInt) refuse(ASV_ERR_DTYPE, "%s must be int32", name);
  if (t.dim() != 1 || t.size(0) != n) refuse(ASV_ERR_SHAPE, "%s must be [%lld]", name, (long long)n);
  if (n > 1 && t.stride(0) != 1) refuse(ASV_ERR_SHAPE, "%s must be contiguous", name);
  return static_cast<const int32_t*>(t.data_ptr());
}

struct Paged {
  asv_paged_cache cache;
  asv_paged_batch batch;
  at::ScalarType type;
  at::Device device;
};

Paged paged(const at::Tensor& k, const at::Tensor& v, const at::Tensor& table, const at::Tensor& cache_len,
            const at::Tensor& indptr, int64_t N) {
  if (k.dim() != 4 || v.dim() != 4 || k.sizes() != v.sizes())
    refuse(ASV_ERR_SHAPE, "k_cache and v_cache must share one [num_pages, page_size, kv_heads, head_dim] shape");
  Paged p{{}, {}, k.scalar_type(), k.device()};
  if ((p.type != at::kBFloat16 && p.type != at::kHalf) || v.scalar_type() != p.type)
    refuse(ASV_ERR_DTYPE, "k_cache and v_cache must share bfloat16 or float16");
  if (table.scalar_type() != at::kInt) refuse(ASV_ERR_DTYPE, "block_table must be int32");
  if (table.dim() != 2) refuse(ASV_ERR_SHAPE, "block_table must be [B, max_pages]");
  if ((k.size(3) > 1 && (k.stride(3) != 1 || v.stride(3) != 1)) || (table.size(1) > 1 && table.stride(1) != 1))
    refuse(ASV_ERR_ALIGN, "the last dimension of k_cache, v_cache and block_table must be contiguous");
  p.cache = {k.data_ptr(),
             v.data_ptr(),
             p.type == at::kBFloat16 ? ASV_BF16 : ASV_F16,
             extent(k.size(0), "num_pages"),
             extent(k.size(1), "page_size"),
             extent(k.size(2), "kv_heads"),
             extent(k.size(3), "head_dim"),
             k.stride(0),
             k.stride(1),
             k.stride(2),
             v.stride(0),
             v.stride(1),
             v.stride(2)};
  const int64_t B = table.size(0);
  p.batch = {extent(B, "B"),
             extent(N, "N"),
             lengths(indptr, "indptr", B + 1),
             lengths(cache_len, "cache_len", B),
             static_cast<const int32_t*>(table.data_ptr()),
             extent(table.size(1), "max_pages"),
             table.stride(0)};
  for (const at::Tensor* t : {&v, &table, &cache_len, &indptr})
    if (t->device() != p.device) refuse(ASV_ERR_SHAPE, "the tensors must be on one device");
  return p;
}

// Packed rows [N, heads, head_dim] of the cache's type.
asv_rows rows(const at::Tensor& t, const char* name, const Paged& p, int64_t heads) {
  if (t.dim() != 3 || t.size(0) != p.batch.N || t.size(1) != heads || t.size(2) != p.cache.head_dim)
    refuse(ASV_ERR_SHAPE, "%s must be [%d, %lld, %d]", name, p.batch.N, (long long)heads, p.cache.head_dim);
  if (t.scalar_type() != p.type) refuse(ASV_ERR_DTYPE, "%s must have the cache's type", name);
  if (t.stride(2) != 1 && t.size(2) > 1) refuse(ASV_ERR_ALIGN, "the last dimension of %s must be contiguous", name);
  if (t.device() != p.device) refuse(ASV_ERR_SHAPE, "the tensors must be on one device");
  return {t.data_ptr(), t.stride(0), t.stride(1)};
}

uint32_t* status_of(const at::Tensor& t, const Paged& p) {
  if (t.device() != p.device) refuse(ASV_ERR_SHAPE, "the tensors must be on one device");
  return reinterpret_cast<uint32_t*>(const_cast<int32_t*>(lengths(t, "req_status", p.batch.B)));
}

long long whole_number(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(ASV_ERR_PARAM, "%s must be a whole number", name);
  }
  return v;
}

bool truth(PyObject* o, const char* name) {
  const int t = PyObject_IsTrue(o);
  if (t < 0) {
    PyErr_Clear();
    refuse(ASV_ERR_PARAM, "%s must be true or false", name);
  }
  return t != 0;
}

cudaStream_t stream_of(PyObject* o) { return reinterpret_cast<cudaStream_t>(static_cast<uintptr_t>(whole_number(o, "stream"))); }

PyObject* result(asv_status st, const char* what) {
  if (st == ASV_OK) Py_RETURN_NONE;
  if (st == ASV_ERR_CUDA) refuse(st, "%s: %s (cudaError %d)", what, g_status_string(st), g_last_cuda_error());
  refuse(st, "%s: %s", what, g_status_string(st));
}

// f(), a call of the library, with the interpreter's lock released: a launch waits while the stream's queue is full, and
// what drains it may need the lock (a host function in Python).  Nothing in the library throws.
template <class F>
asv_status unlocked(F f) {
  PyThreadState* state = PyEval_SaveThread();
  const asv_status st = f();
  PyEval_RestoreThread(state);
  return st;
}

// Nothing but a Python exception leaves a call.
template <class F>
PyObject* guarded(const char* what, Py_ssize_t n, Py_ssize_t expected, F f) {
  if (!g_attention) return PyErr_Format(PyExc_RuntimeError, "%s: bind() has not been called", what);
  if (n != expected) return PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", what, expected, n);
  try {
    return f();
  } catch (const Refused& r) {
    PyObject* e = PyObject_CallFunction(g_error, "is", r.status, r.text);
    if (e) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, what);
  }
  return nullptr;
}

// q, k_cache, v_cache, block_table, cache_len, indptr, scale (None: head_dim ** -0.5), window, out, lse (or None),
// req_status, workspace, stream
PyObject* py_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("paged_attention", n, 13, [&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0], "q");
    if (q.dim() != 3) refuse(ASV_ERR_SHAPE, "q must be [N, q_heads, head_dim]");
    const Paged p = paged(tensor(a[1], "k_cache"), tensor(a[2], "v_cache"), tensor(a[3], "block_table"),
                          tensor(a[4], "cache_len"), tensor(a[5], "indptr"), q.size(0));
    const int heads = extent(q.size(1), "q_heads");
    const asv_rows qr = rows(q, "q", p, heads), out = rows(tensor(a[8], "out.out"), "out.out", p, heads);
    double scale = 0.0;
    if (a[6] == Py_None) {
      scale = 1.0 / std::sqrt(double(p.cache.head_dim));
    } else {
      scale = PyFloat_AsDouble(a[6]);
      if (scale == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(ASV_ERR_PARAM, "scale must be a number");
      }
    }
    const long long window = whole_number(a[7], "window");
    if (window < 0 || window > 0x7fffffff) refuse(ASV_ERR_PARAM, "window must be a whole number of 32 bits, 0 or more");
    float* lse = nullptr;
    if (a[9] != Py_None) {
      const at::Tensor& t = tensor(a[9], "out.lse");
      if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != q.size(0) || t.size(1) != heads ||
          !t.is_contiguous() || t.device() != p.device)
        refuse(ASV_ERR_SHAPE, "out.lse must be contiguous float32 [N, q_heads]");
      lse = static_cast<float*>(t.data_ptr());
    }
    const at::Tensor& ws = tensor(a[11], "workspace");
    if (!ws.is_contiguous() || ws.device() != p.device) refuse(ASV_ERR_WORKSPACE, "workspace must be contiguous, on the tensors' device");
    uint32_t* status = status_of(tensor(a[10], "req_status"), p);
    void* const room = ws.data_ptr();
    const size_t bytes = ws.nbytes();
    const cudaStream_t stream = stream_of(a[12]);
    return result(unlocked([&]() {
                    return g_attention(&p.cache, &p.batch, &qr, &out, heads, float(scale), int(window), lse, status, room,
                                       bytes, stream);
                  }),
                  "paged_attention");
  });
}

// k, v, k_cache, v_cache, block_table, cache_len, indptr, q (or None), rotary (or None), interleaved, out_q (or
// None), req_status, (these two or neither: positions (or None), axes (bytes, or None)), stream
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("paged_kv_append", n, n == 13 ? 13 : 15, [&]() -> PyObject* {
    const bool interleaved = truth(a[9], "interleaved");
    const at::Tensor& k = tensor(a[0], "k");
    if (k.dim() != 3) refuse(ASV_ERR_SHAPE, "k and v must be [N, kv_heads, head_dim]");
    const Paged p = paged(tensor(a[2], "k_cache"), tensor(a[3], "v_cache"), tensor(a[4], "block_table"),
                          tensor(a[5], "cache_len"), tensor(a[6], "indptr"), k.size(0));
    const asv_rows kr = rows(k, "k", p, p.cache.kv_heads), vr = rows(tensor(a[1], "v"), "v", p, p.cache.kv_heads);
    asv_rows qr, oq;
    int heads = 0;
    const bool with_q = a[7] != Py_None;
    if (with_q) {
      const at::Tensor& q = tensor(a[7], "q");
      if (q.dim() != 3) refuse(ASV_ERR_SHAPE, "q must be [N, q_heads, head_dim]");
      if (a[10] == Py_None) refuse(ASV_ERR_NULL, "out.q is missing");
      heads = extent(q.size(1), "q_heads");
      qr = rows(q, "q", p, heads);
      oq = rows(tensor(a[10], "out.q"), "out.q", p, heads);
    }
    asv_rotary rot;
    const bool rotate = a[8] != Py_None;
    if (rotate) {
      const at::Tensor& t = tensor(a[8], "rotary");
      if (t.scalar_type() != at::kFloat || t.dim() != 2 || !t.is_contiguous() || t.device() != p.device)
        refuse(ASV_ERR_SHAPE, "rotary must be a contiguous float32 [max_position, dim] table");
      rot = {static_cast<const float*>(t.data_ptr()), extent(t.size(1), "the rotation's dim"),
             extent(t.size(0), "max_position"), interleaved};
    }
    asv_positions at = {};
    const bool placed = n > 13 && a[12] != Py_None;
    if (placed) {
      const at::Tensor& t = tensor(a[12], "positions");
      if (t.scalar_type() != at::kInt) refuse(ASV_ERR_DTYPE, "positions must be int32");
      if ((t.dim() != 1 && t.dim() != 2) || t.size(-1) != p.batch.N || (t.size(-1) > 1 && t.stride(-1) != 1) ||
          t.device() != p.device)
        refuse(ASV_ERR_SHAPE, "positions must be [axes, %d] or [%d], each axis's contiguous, on the tensors' device", p.batch.N,
               p.batch.N);
      at.at = static_cast<const int32_t*>(t.data_ptr());
      at.axes = t.dim() == 1 ? 1 : extent(t.size(0), "axes");
      at.stride_axis = t.dim() == 1 ? 0 : t.stride(0);
    }
    if (n > 13 && a[13] != Py_None) {
      if (!placed || !rotate) refuse(ASV_ERR_PARAM, "axes go with positions and a rotation");
      if (!PyBytes_Check(a[13]) || PyBytes_GET_SIZE(a[13]) != rot.dim / 2)
        refuse(ASV_ERR_PARAM, "axes must be the axis of each of the rotation's %d pairs", rot.dim / 2);
      at.axis_of_pair = reinterpret_cast<const uint8_t*>(PyBytes_AS_STRING(a[13]));
    } else if (placed && at.axes != 1) {
      refuse(ASV_ERR_PARAM, "positions of several axes need axes=, the axis of each pair");
    }
    uint32_t* status = status_of(tensor(a[11], "req_status"), p);
    const cudaStream_t stream = stream_of(a[n - 1]);
    return result(unlocked([&]() {
                    const asv_rows *qs = with_q ? &qr : nullptr, *os = with_q ? &oq : nullptr;
                    const asv_rotary* turn = rotate ? &rot : nullptr;
                    return placed ? g_append_ex(&p.cache, &p.batch, &kr, &vr, qs, os, heads, turn, &at, status, stream)
                                  : g_append(&p.cache, &p.batch, &kr, &vr, qs, os, heads, turn, status, stream);
                  }),
                  "paged_kv_append");
  });
}

// A tensor of `type` on `device` with `n` entries in a row; None: nullptr.
void* entries(PyObject* o, const char* name, at::ScalarType type, const char* type_name, int64_t n, at::Device device) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type) refuse(ASV_ERR_DTYPE, "%s must be %s", name, type_name);
  if (t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
    refuse(ASV_ERR_SHAPE, "%s must be contiguous, [%lld]", name, (long long)n);
  if (t.device() != device) refuse(ASV_ERR_SHAPE, "the tensors must be on one device");
  return t.data_ptr();
}

// cache_len, new_len, block_table, held, free_pages, free_count, page_size, release (or None), indptr, slots (or None),
// positions (or None), requests (or None), req_status, N, stream
PyObject* py_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("paged_plan", n, 15, [&]() -> PyObject* {
    const at::Tensor& table = tensor(a[2], "block_table");
    if (table.scalar_type() != at::kInt) refuse(ASV_ERR_DTYPE, "block_table must be int32");
    if (table.dim() != 2 || (table.size(1) > 1 && table.stride(1) != 1))
      refuse(ASV_ERR_SHAPE, "block_table must be [B, max_pages], its rows contiguous");
    const at::Device dev = table.device();
    const int64_t B = table.size(0);
    const at::Tensor& pool = tensor(a[4], "free_pages");
    const long long page = whole_number(a[6], "page_size"), rows = whole_number(a[13], "max_tokens");
    if (rows < 0 || rows > 0x7fffffff) refuse(ASV_ERR_SHAPE, "max_tokens must be a whole number of 32 bits, 0 or more");
    if (page < 1 || page > 0x7fffffff) refuse(ASV_ERR_SHAPE, "page_size must be a whole number of 32 bits, 1 or more");
    auto ints = [&](int i, const char* name, int64_t len) {
      return static_cast<int32_t*>(entries(a[i], name, at::kInt, "int32", len, dev));
    };
    auto present = [&](int i, const char* name, int64_t len) {
      int32_t* p = ints(i, name, len);
      if (a[i] == Py_None) refuse(ASV_ERR_NULL, "%s is missing", name);
      return p;
    };
    const asv_page_pool p = {static_cast<int32_t*>(table.data_ptr()),
                             extent(table.size(1), "max_pages"),
                             table.stride(0),
                             int(page),
                             present(3, "held", B),
                             present(4, "free_pages", pool.dim() == 1 ? pool.size(0) : -1),
                             extent(pool.dim() == 1 ? pool.size(0) : 0, "free_pages"),
                             present(5, "free_count", 1)};
    const int32_t* len = present(0, "cache_len", B);
    const int32_t* grow = present(1, "new_len", B);
    const uint8_t* release = static_cast<const uint8_t*>(entries(a[7], "release", at::kBool, "bool", B, dev));
    int32_t* indptr = present(8, "out.indptr", B + 1);
    int64_t* slots = static_cast<int64_t*>(entries(a[9], "out.slots", at::kLong, "int64", rows, dev));
    int32_t* positions = ints(10, "out.positions", rows);
    int32_t* requests = ints(11, "out.requests", rows);
    uint32_t* status = reinterpret_cast<uint32_t*>(present(12, "out.req_status", B));
    const int requests_in = extent(B, "B");
    const cudaStream_t stream = stream_of(a[14]);
    return result(unlocked([&]() {
                    return g_plan(len, grow, requests_in, &p, release, int(rows), indptr, slots, positions, requests, status,
                                  stream);
                  }),
                  "paged_plan");
  });
}

// AsvError, and the addresses of paged_attention, paged_kv_append, asv_status_string, asv_last_cuda_error
PyObject* py_bind(PyObject*, PyObject* args) {
  PyObject* error;
  unsigned long long f[4];
  if (!PyArg_ParseTuple(args, "OKKKK", &error, &f[0], &f[1], &f[2], &f[3])) return nullptr;
  Py_INCREF(error);
  Py_XDECREF(g_error);
  g_error = error;
  g_attention = reinterpret_cast<decltype(g_attention)>(f[0]);
  g_append = reinterpret_cast<decltype(g_append)>(f[1]);
  g_status_string = reinterpret_cast<decltype(g_status_string)>(f[2]);
  g_last_cuda_error = reinterpret_cast<decltype(g_last_cuda_error)>(f[3]);
  Py_RETURN_NONE;
}

// A [B, n] or [B] field (or with V > 0 rows of V: one dimension more) of `type`.
asv_field field(const at::Tensor& t, const char* name, at::ScalarType type, const char* type_name, int64_t dims, int64_t B,
                int64_t n, int64_t V, at::Device device) {
  if (t.scalar_type() != type) refuse(ASV_ERR_DTYPE, "%s must be %s", name, type_name);
  const int64_t d = dims + (V > 0 ? 1 : 0);
  if (t.dim() != d || t.size(0) != B || (dims == 2 && t.size(1) != n) || (V > 0 && t.size(d - 1) != V))
    refuse(ASV_ERR_SHAPE, "%s has the wrong shape: one entry%s for each row of logits", name, V > 0 ? " of the vocabulary" : "");
  if (V > 1 && t.stride(d - 1) != 1) refuse(ASV_ERR_SHAPE, "the last dimension of %s must be contiguous", name);
  if (t.device() != device) refuse(ASV_ERR_SHAPE, "the tensors must be on one device");
  return {t.data_ptr(), t.stride(0), dims == 2 ? t.stride(1) : 0};
}

// A number, or a tensor [B] of its own for each request.
template <class Number>
void parameter(PyObject* o, const char* name, at::ScalarType type, const char* type_name, int64_t B, at::Device device,
               Number* one, const Number** each) {
  if (THPVariable_Check(o)) {
    *each = static_cast<const Number*>(entries(o, name, type, type_name, B, device));
    return;
  }
  if constexpr (std::is_integral_v<Number>) {
    const long long v = whole_number(o, name);
    if (v < 0 || v > 0x7fffffff) refuse(ASV_ERR_PARAM, "%s must be a whole number of 32 bits, 0 or more", name);
    *one = Number(v);
  } else {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      refuse(ASV_ERR_PARAM, "%s must be a number or a tensor", name);
    }
    *one = Number(v);
  }
}

// logits, u, temperature, top_k, top_p, min_p (each a number or a tensor [B]), tokens, logprobs (or None), probs (or
// None), req_status, stream
PyObject* py_sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("sample_tokens", n, 11, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "logits");
    const int64_t dims = x.dim() - 1;
    if (dims != 1 && dims != 2) refuse(ASV_ERR_SHAPE, "logits must be [B, n, V] or [B, V]");
    const at::Device dev = x.device();
    const int64_t B = x.size(0), rows = dims == 2 ? x.size(1) : 1, V = x.size(dims);
    asv_logits l = {};
    if (x.scalar_type() == at::kFloat) l.dtype = ASV_F32;
    else if (x.scalar_type() == at::kBFloat16) l.dtype = ASV_BF16;
    else refuse(ASV_ERR_DTYPE, "logits must be float32 or bfloat16");
    if (V < 1 || (V > 1 && x.stride(dims) != 1)) refuse(ASV_ERR_SHAPE, "the last dimension of logits must be contiguous and not empty");
    l.data = x.data_ptr();
    l.B = extent(B, "B");
    l.n = extent(rows, "n");
    l.V = extent(V, "V");
    l.stride_request = x.stride(0);
    l.stride_position = dims == 2 ? x.stride(1) : 0;
    const asv_field u = field(tensor(a[1], "u"), "u", at::kFloat, "float32", dims, B, rows, 0, dev);
    asv_sampling one = {1.0f, 0, 1.0f, 0.0f};
    asv_sampling_each each = {};
    parameter(a[2], "temperature", at::kFloat, "float32", B, dev, &one.temperature, &each.temperature);
    parameter(a[3], "top_k", at::kInt, "int32", B, dev, &one.top_k, &each.top_k);
    parameter(a[4], "top_p", at::kFloat, "float32", B, dev, &one.top_p, &each.top_p);
    parameter(a[5], "min_p", at::kFloat, "float32", B, dev, &one.min_p, &each.min_p);
    const asv_field tokens = field(tensor(a[6], "out.tokens"), "out.tokens", at::kInt, "int32", dims, B, rows, 0, dev);
    asv_field logprobs = {}, probs = {};
    if (a[7] != Py_None)
      logprobs = field(tensor(a[7], "out.logprobs"), "out.logprobs", at::kFloat, "float32", dims, B, rows, 0, dev);
    if (a[8] != Py_None)
      probs = field(tensor(a[8], "out.probs"), "out.probs", at::kFloat, "float32", dims, B, rows, V, dev);
    if (a[9] == Py_None) refuse(ASV_ERR_NULL, "out.req_status is missing");
    uint32_t* status = static_cast<uint32_t*>(entries(a[9], "out.req_status", at::kInt, "int32", B, dev));
    const bool with_logprobs = a[7] != Py_None, with_probs = a[8] != Py_None;
    const cudaStream_t stream = stream_of(a[10]);
    return result(unlocked([&]() {
                    return g_sample(&l, &u, &one, &each, &tokens, with_logprobs ? &logprobs : nullptr,
                                    with_probs ? &probs : nullptr, status, stream);
                  }),
                  "sample_tokens");
  });
}

// the addresses of paged_kv_append_ex, paged_plan and sample_tokens
PyObject* py_bind_step(PyObject*, PyObject* args) {
  unsigned long long f[3];
  if (!PyArg_ParseTuple(args, "KKK", &f[0], &f[1], &f[2])) return nullptr;
  g_append_ex = reinterpret_cast<decltype(g_append_ex)>(f[0]);
  g_plan = reinterpret_cast<decltype(g_plan)>(f[1]);
  g_sample = reinterpret_cast<decltype(g_sample)>(f[2]);
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"bind", py_bind, METH_VARARGS, nullptr},
    {"bind_step", py_bind_step, METH_VARARGS, nullptr},
    {"sample_tokens", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_sample)), METH_FASTCALL, nullptr},
    {"paged_plan", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_plan)), METH_FASTCALL, nullptr},
    {"paged_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_attention)), METH_FASTCALL, nullptr},
    {"paged_kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_append)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "asv_torch", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_asv_torch() { return PyModule_Create(&kModule); }
