// Python binding of the operators around the attention (module _bind, used by
// _block.py): checks torch tensors, allocates outputs and workspaces, and calls
// the C entries of libra.so.  Written against CPython and torch's C++ API because
// a single token's call is host time: the same checks through ctypes took 10 us
// and more of a call whose kernel runs for 3.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <cstring>
#include <optional>
#include <string>

#include "../../include/ra.h"

namespace {

PyObject* g_error = nullptr;   // RaError(fn, status)
PyObject* g_memory = nullptr;  // torch.OutOfMemoryError

// A Python exception has been set.
struct Raised {};

[[noreturn]] void value_error(const std::string& text) {
  PyErr_SetString(PyExc_ValueError, text.c_str());
  throw Raised{};
}

std::string text_of(c10::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) value_error(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

const at::Tensor& cuda4(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 4 || !t.is_cuda()) value_error(std::string(name) + " must be a four-dimensional CUDA tensor");
  return t;
}

[[noreturn]] void mismatch(const at::Tensor& t, const char* name, const char* kind, at::ScalarType dt,
                           c10::IntArrayRef shape, c10::Device dev) {
  value_error(std::string(name) + " must be a " + kind + c10::toString(dt) + " tensor of shape " + text_of(shape) +
              " on " + dev.str() + ", got " + c10::toString(t.scalar_type()) + ", " + text_of(t.sizes()) +
              ", strides " + text_of(t.strides()) + " on " + t.device().str());
}

// Address of a contiguous tensor of the given type and shape; NULL for None.
void* arg(PyObject* o, const char* name, at::ScalarType dt, c10::IntArrayRef shape, c10::Device dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != dt || t.sizes() != shape || t.device() != dev || !t.is_contiguous())
    mismatch(t, name, "contiguous ", dt, shape, dev);
  return t.data_ptr();
}

// Address and strides of a [B, H, N, D] tensor with contiguous channels.
void* view(const at::Tensor& t, const char* name, at::ScalarType dt, c10::IntArrayRef shape, c10::Device dev,
           ra_strides* st) {
  if (t.scalar_type() != dt || t.sizes() != shape || t.device() != dev) mismatch(t, name, "", dt, shape, dev);
  if (t.stride(3) != 1)
    value_error(std::string(name) + " must have contiguous channels, got strides " + text_of(t.strides()));
  *st = ra_strides{t.stride(0), t.stride(1), t.stride(2)};
  return t.data_ptr();
}

at::Tensor dense(c10::IntArrayRef shape, at::ScalarType dt, c10::Device dev) {
  return at::Tensor(at::detail::empty_cuda(shape, dt, dev, std::nullopt));
}

int dtype_of(const at::Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return RA_DT_BF16;
  if (t.scalar_type() == at::kFloat) return RA_DT_F32;
  value_error("inputs must be bfloat16 or float32");
}

int integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (v < INT_MIN || v > INT_MAX) value_error(std::string(name) + " is out of range");
  return static_cast<int>(v);
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return static_cast<float>(v);
}

float scale_of(PyObject* o, int64_t D) {
  return o == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D))) : number(o);
}

// An extent of a tensor as the C entries take it.
int extent(int64_t v) {
  if (v > INT_MAX) value_error("a tensor's extent is out of range");
  return static_cast<int>(v);
}

bool truth(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw Raised{};
  return r == 1;
}

// Calls a C entry without the interpreter's lock: a launch waits when the stream's queue is full.
template <typename F>
void call(const char* fn, F f) {
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = f();
  Py_END_ALLOW_THREADS
  if (status == RA_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "si", fn, status);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

void* stream_of(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// A C structure held by a bytes object or a ctypes structure.
template <typename T>
T structure(PyObject* o, const char* name) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw Raised{};
  T v;
  const bool fits = b.len == static_cast<Py_ssize_t>(sizeof(T));
  if (fits) std::memcpy(&v, b.buf, sizeof(T));
  PyBuffer_Release(&b);
  if (!fits) value_error(std::string(name) + " is not the structure expected");
  return v;
}

// Runs an entry: no C++ exception leaves it, and a wrong number of arguments is refused.
template <typename F>
PyObject* entry(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const Raised&) {
    return nullptr;
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_memory, e.what_without_backtrace());
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    return nullptr;
  }
}

// An output: the caller's (checked) or a new one.
struct Out {
  at::Tensor t;
  PyObject* given = nullptr;
  void* p = nullptr;
  PyObject* object() const {
    if (given) {
      Py_INCREF(given);
      return given;
    }
    return THPVariable_Wrap(t);
  }
};

Out output(PyObject* o, const char* name, at::ScalarType dt, c10::IntArrayRef shape, c10::Device dev) {
  Out r;
  if (o == Py_None) {
    r.t = dense(shape, dt, dev);
    r.p = r.t.data_ptr();
  } else {
    r.given = o;
    r.p = arg(o, name, dt, shape, dev);
  }
  return r;
}

PyObject* pair(PyObject* a, PyObject* b) {
  if (!a || !b) {
    Py_XDECREF(a);
    Py_XDECREF(b);
    return nullptr;
  }
  PyObject* t = PyTuple_New(2);
  if (!t) {
    Py_DECREF(a);
    Py_DECREF(b);
    return nullptr;
  }
  PyTuple_SET_ITEM(t, 0, a);
  PyTuple_SET_ITEM(t, 1, b);
  return t;
}

PyObject* none() {
  Py_INCREF(Py_None);
  return Py_None;
}

// problem, q, k, table, pos, q_weight, k_weight, q_bias, k_bias, norm, eps, q_out, k_out
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 13, [&]() -> PyObject* {
    const ra_problem p = structure<ra_problem>(a[0], "p");
    const bool has[2] = {a[1] != Py_None, a[2] != Py_None};
    if (!has[0] && !has[1]) value_error("q or k must be given");
    const at::Tensor& some = cuda4(has[0] ? a[1] : a[2], has[0] ? "q" : "k");
    const c10::Device dev = some.device();
    const c10::cuda::OptionalCUDAGuard guard(dev);
    const at::ScalarType dt = some.scalar_type();
    const int in_dtype = dtype_of(some);
    int heads[2] = {p.H, p.H};
    const char* names[2][2] = {{"q", "q_out"}, {"k", "k_out"}};
    void* x[2] = {};
    ra_strides st[2];
    Out out[2];
    for (int i = 0; i < 2; ++i) {
      if (!has[i]) continue;
      const at::Tensor& t = cuda4(a[1 + i], names[i][0]);
      if (i == 1) heads[1] = extent(t.size(1));
      const int64_t shape[4] = {p.B, heads[i], p.N, p.D};
      x[i] = view(t, names[i][0], dt, shape, dev, &st[i]);
      out[i] = output(a[11 + i], names[i][1], at::kBFloat16, shape, dev);
    }
    const int64_t row[1] = {p.D}, pos[2] = {p.N, 3};
    void* tab = nullptr;
    size_t tab_bytes = 0;
    if (a[3] != Py_None) {
      const at::Tensor& t = tensor(a[3], "table");
      const int64_t shape[2] = {t.dim() > 0 ? t.size(0) : 0, 2};
      tab = arg(a[3], "table", at::kFloat, shape, dev);
      tab_bytes = static_cast<size_t>(shape[0]) * 8;
    }
    auto vec = [&](int i, const char* name) {
      return static_cast<const float*>(arg(a[i], name, at::kFloat, row, dev));
    };
    const float *qw = vec(5, "q_weight"), *kw = vec(6, "k_weight"), *qb = vec(7, "q_bias"), *kb = vec(8, "k_bias");
    const int32_t* at_pos = static_cast<const int32_t*>(arg(a[4], "pos", at::kInt, pos, dev));
    const int norm = integer(a[9], "norm");
    const float eps = number(a[10]);
    void* const stream = stream_of(dev);
    call("ra_qk_norm_rope", [&] {
      return ra_qk_norm_rope(&p, heads[1], norm, eps, in_dtype, x[0], has[0] ? &st[0] : nullptr, x[1],
                             has[1] ? &st[1] : nullptr, qw, kw, qb, kb, at_pos, tab, tab_bytes, out[0].p, out[1].p,
                             stream);
    });
    return pair(has[0] ? out[0].object() : none(), has[1] ? out[1].object() : none());
  });
}

// The cache that four tensors hold now.
ra_kv4_cache cache_of(PyObject* const* a) {
  const at::Tensor& k4 = cuda4(a[0], "k4");
  const c10::IntArrayRef codes = k4.sizes(), scales = codes.slice(0, 3);
  const c10::Device dev = k4.device();
  ra_kv4_cache c;
  std::memset(&c, 0, sizeof(c));
  c.num_pages = extent(codes[0]);
  c.Hk = extent(codes[1]);
  c.page_size = extent(codes[2]);
  c.D = extent(2 * codes[3]);
  c.k4 = static_cast<uint8_t*>(arg(a[0], "k4", at::kByte, codes, dev));
  c.sk = static_cast<float*>(arg(a[1], "sk", at::kFloat, scales, dev));
  c.v4 = static_cast<uint8_t*>(arg(a[2], "v4", at::kByte, codes, dev));
  c.sv = static_cast<float*>(arg(a[3], "sv", at::kFloat, scales, dev));
  return c;
}

// A cache as a tuple of its tensors (k4, sk, v4, sv) on `dev`, or as the bytes that kv4_cache made of them.  Tensors
// are looked at in every call: memory that they were moved to or from since the last one is not mistaken for theirs.
ra_kv4_cache cache_arg(PyObject* o, c10::Device dev) {
  if (!PyTuple_Check(o)) return structure<ra_kv4_cache>(o, "cache");
  if (PyTuple_GET_SIZE(o) != 4) value_error("cache is not the four tensors expected");
  PyObject* const t[4] = {PyTuple_GET_ITEM(o, 0), PyTuple_GET_ITEM(o, 1), PyTuple_GET_ITEM(o, 2), PyTuple_GET_ITEM(o, 3)};
  const ra_kv4_cache c = cache_of(t);
  if (THPVariable_Unpack(t[0]).device() != dev) value_error("the cache's tensors have left " + dev.str());
  return c;
}

// k4, sk, v4, sv -> the ra_kv4_cache as bytes
PyObject* kv4_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 4, [&]() -> PyObject* {
    const ra_kv4_cache c = cache_of(a);
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&c), sizeof(c));
  });
}

const int32_t* ints(PyObject* o, const char* name, int64_t B, c10::Device dev) {
  const int64_t shape[1] = {B};
  return static_cast<const int32_t*>(arg(o, name, at::kInt, shape, dev));
}

const int32_t* block_table(PyObject* o, int64_t B, c10::Device dev, int* max_pages) {
  const at::Tensor& t = tensor(o, "block_table");
  if (t.dim() != 2) value_error("block_table must be [B, max_pages]");
  const int64_t shape[2] = {B, t.size(1)};
  *max_pages = extent(shape[1]);
  return static_cast<const int32_t*>(arg(o, "block_table", at::kInt, shape, dev));
}

c10::Device device(PyObject* index) {
  return c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(integer(index, "device")));
}

// cache, device index, k, v, block_table, start, n_new
PyObject* kv4_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 7, [&]() -> PyObject* {
    const c10::Device dev = device(a[1]);
    const ra_kv4_cache c = cache_arg(a[0], dev);
    const c10::cuda::OptionalCUDAGuard guard(dev);
    const at::Tensor& k = cuda4(a[2], "k");
    const at::Tensor& v = cuda4(a[3], "v");
    const int64_t shape[4] = {k.size(0), c.Hk, k.size(2), c.D};
    ra_strides ks, vs;
    const void* kp = view(k, "k", k.scalar_type(), shape, dev, &ks);
    const void* vp = view(v, "v", k.scalar_type(), shape, dev, &vs);
    int pages = 0;
    const int32_t* table = block_table(a[4], shape[0], dev, &pages);
    const int32_t *start = ints(a[5], "start", shape[0], dev), *n_new = ints(a[6], "n_new", shape[0], dev);
    const int in_dtype = dtype_of(k), B = extent(shape[0]), T = extent(shape[2]);
    void* const stream = stream_of(dev);
    call("ra_kv4_append",
         [&] { return ra_kv4_append(&c, in_dtype, B, T, kp, &ks, vp, &vs, table, pages, start, n_new, stream); });
    return none();
  });
}

// cache, device index, block_table, start, T, n, fp32 (truth value), k, v (outputs or None)
PyObject* kv4_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 9, [&]() -> PyObject* {
    const c10::Device dev = device(a[1]);
    const ra_kv4_cache c = cache_arg(a[0], dev);
    const c10::cuda::OptionalCUDAGuard guard(dev);
    const at::Tensor& t = tensor(a[2], "block_table");
    const int64_t B = t.dim() > 0 ? t.size(0) : 0;
    int pages = 0;
    const int32_t* table = block_table(a[2], B, dev, &pages);
    const int T = integer(a[4], "T");
    if (T < 1 || B < 1) value_error("B and T must be at least 1");
    const int64_t shape[4] = {B, c.Hk, T, c.D};
    at::ScalarType dt = truth(a[6]) ? at::kFloat : at::kBFloat16;
    if (a[7] != Py_None) dt = tensor(a[7], "k").scalar_type() == at::kFloat ? at::kFloat : at::kBFloat16;
    const Out k = output(a[7], "k", dt, shape, dev), v = output(a[8], "v", dt, shape, dev);
    const int32_t *start = ints(a[3], "start", B, dev), *n_read = ints(a[5], "n", B, dev);
    const int out_dtype = dt == at::kFloat ? RA_DT_F32 : RA_DT_BF16, nb = extent(B);
    void* const stream = stream_of(dev);
    call("ra_kv4_read",
         [&] { return ra_kv4_read(&c, out_dtype, nb, T, table, pages, start, n_read, k.p, v.p, stream); });
    return pair(k.object(), v.object());
  });
}

// cache, device index, q, block_table, seq_lens, q_lens, causal, scale, max_len, out, lse, workspace
PyObject* attn_kv4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 12, [&]() -> PyObject* {
    const c10::Device dev = device(a[1]);
    const ra_kv4_cache c = cache_arg(a[0], dev);
    const c10::cuda::OptionalCUDAGuard guard(dev);
    const at::Tensor& q = cuda4(a[2], "q");
    const c10::IntArrayRef shape = q.sizes();
    if (shape[3] != c.D)
      value_error("q must have " + std::to_string(c.D) + " channels, got " + std::to_string(shape[3]));
    const void* qp = arg(a[2], "q", at::kBFloat16, shape, dev);
    ra_kv4_attn prob;
    const int32_t* table = block_table(a[3], shape[0], dev, &prob.max_pages);
    prob.B = extent(shape[0]);
    prob.H = extent(shape[1]);
    prob.Nq = extent(shape[2]);
    prob.causal = truth(a[6]);
    prob.scale = scale_of(a[7], shape[3]);
    const int64_t reach = static_cast<int64_t>(prob.max_pages) * c.page_size;
    prob.max_len = a[8] == Py_None ? static_cast<int>(reach < INT_MAX ? reach : INT_MAX) : integer(a[8], "max_len");
    const int32_t* lens = ints(a[4], "seq_lens", shape[0], dev);
    const int32_t* q_lens = ints(a[5], "q_lens", shape[0], dev);
    const Out out = output(a[9], "out", at::kBFloat16, shape, dev);
    float* lse = static_cast<float*>(arg(a[10], "lse", at::kFloat, shape.slice(0, 3), dev));
    at::Tensor made;
    void* ws = nullptr;
    size_t bytes = 0;
    if (a[11] == Py_None) {
      bytes = ra_attn_kv4_workspace_bytes(&c, &prob);
      if (bytes) {
        const int64_t size[1] = {static_cast<int64_t>(bytes)};
        made = dense(size, at::kByte, dev);
        ws = made.data_ptr();
      }
    } else {
      const int64_t size[1] = {tensor(a[11], "workspace").numel()};
      ws = arg(a[11], "workspace", at::kByte, size, dev);
      bytes = static_cast<size_t>(size[0]);
    }
    void* const stream = stream_of(dev);
    call("ra_attn_kv4",
         [&] { return ra_attn_kv4(&c, &prob, qp, table, lens, q_lens, ws, bytes, out.p, lse, stream); });
    return out.object();
  });
}

// q, k, v, kv_lens, scale, out, lse
PyObject* attn_cross(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 7, [&]() -> PyObject* {
    const at::Tensor& q = cuda4(a[0], "q");
    const at::Tensor& k = cuda4(a[1], "k");
    const at::Tensor& v = cuda4(a[2], "v");
    const c10::Device dev = q.device();
    const c10::cuda::OptionalCUDAGuard guard(dev);
    const c10::IntArrayRef shape = q.sizes();
    const int64_t kshape[4] = {shape[0], k.size(1), k.size(2), shape[3]};
    ra_cross_problem p;
    p.B = extent(shape[0]);
    p.H = extent(shape[1]);
    p.Nq = extent(shape[2]);
    p.D = extent(shape[3]);
    p.Hk = extent(kshape[1]);
    p.Nk = extent(kshape[2]);
    p.scale = scale_of(a[4], shape[3]);
    ra_strides qs, ks, vs, os;
    const void* qp = view(q, "q", at::kBFloat16, shape, dev, &qs);
    const void* kp = view(k, "k", at::kBFloat16, kshape, dev, &ks);
    const void* vp = view(v, "v", at::kBFloat16, kshape, dev, &vs);
    const int32_t* lens = ints(a[3], "kv_lens", shape[0], dev);
    float* lse = static_cast<float*>(arg(a[6], "lse", at::kFloat, shape.slice(0, 3), dev));
    Out out;
    if (a[5] == Py_None) {
      out.t = dense(shape, at::kBFloat16, dev);
    } else {
      out.given = a[5];
    }
    void* op = view(out.given ? tensor(out.given, "out") : out.t, "out", at::kBFloat16, shape, dev, &os);
    void* const stream = stream_of(dev);
    call("ra_attn_cross", [&] { return ra_attn_cross(&p, qp, &qs, kp, &ks, vp, &vs, lens, op, &os, lse, stream); });
    return out.object();
  });
}

// RaError, torch.OutOfMemoryError: once, before any other call
PyObject* set_errors(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 2, [&]() -> PyObject* {
    PyObject** to[2] = {&g_error, &g_memory};
    for (int i = 0; i < 2; ++i) {
      Py_INCREF(a[i]);
      Py_XSETREF(*to[i], a[i]);
    }
    return none();
  });
}

#define RA_FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {RA_FAST(qk_norm_rope), RA_FAST(kv4_cache), RA_FAST(kv4_append), RA_FAST(kv4_read),
                         RA_FAST(attn_kv4),     RA_FAST(attn_cross), RA_FAST(set_errors),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
