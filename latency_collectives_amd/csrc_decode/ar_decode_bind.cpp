// The decode operators' calls on torch tensors: addresses, sizes and strides out of the tensors,
// checks of what the C entry points cannot see (place, type, shape), then the C entry point.
//
// These calls sit between short kernels of a decode step, so what they cost on the host decides
// the step's rate: reading a call's tensors through the interpreter (attributes, methods, a packed
// struct) took 5.0 us of a 7.6 us call, reading them here takes 0.4 us.

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <optional>

#include "../../include/ar_decode.h"

namespace {

PyObject* g_error = nullptr;  // ArError(code, message)
PyObject *g_value = nullptr, *g_geometry = nullptr, *g_device = nullptr, *g_cuda_stream = nullptr;

struct Bad {};  // a Python exception is set

[[noreturn]] void bad(const char* name, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
void bad(const char* name, const char* fmt, ...) {
  char why[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(why, sizeof why, fmt, ap);
  va_end(ap);
  PyErr_Format(PyExc_ValueError, "%s: %s", name, why);
  throw Bad();
}

constexpr int kMaxParams = 16;

struct Signature {
  const char* fn;
  int count, required;
  const char* name[kMaxParams];
};

// Positional and keyword arguments in the signature's order; NULL where one is left out or None.
struct Params {
  PyObject* at[kMaxParams] = {};
  Params(const Signature& s, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
    if (n > s.count) {
      PyErr_Format(PyExc_TypeError, "%s() takes at most %d arguments, got %zd", s.fn, s.count, n);
      throw Bad();
    }
    for (Py_ssize_t i = 0; i < n; ++i) at[i] = args[i];
    const Py_ssize_t named = kw == nullptr ? 0 : PyTuple_GET_SIZE(kw);
    for (Py_ssize_t i = 0; i < named; ++i) {
      PyObject* key = PyTuple_GET_ITEM(kw, i);
      int j = 0;
      while (j < s.count && PyUnicode_CompareWithASCIIString(key, s.name[j]) != 0) ++j;
      if (j == s.count || at[j] != nullptr) {
        PyErr_Format(PyExc_TypeError, "%s() got %s argument '%U'", s.fn,
                     j == s.count ? "an unexpected" : "multiple values for", key);
        throw Bad();
      }
      at[j] = args[n + i];
    }
    for (int j = 0; j < s.count; ++j) {
      if (at[j] == nullptr && j < s.required) {
        PyErr_Format(PyExc_TypeError, "%s() misses the argument '%s'", s.fn, s.name[j]);
        throw Bad();
      }
      if (at[j] == Py_None) at[j] = nullptr;
    }
  }
};

// Reads one call's arguments; every tensor has to be on the GPU of the first one.
struct Reader {
  const Signature& s;
  const Params& p;
  int device = -1;

  const at::Tensor& tensor(int j) {
    PyObject* o = p.at[j];
    if (o == nullptr || !THPVariable_Check(o)) bad(s.name[j], "needs a tensor");
    return THPVariable_Unpack(o);
  }
  void* address(int j, const at::Tensor& t) {
    if (t.requires_grad() && at::GradMode::is_enabled())
      bad(s.name[j], "requires a gradient, which this call does not give (torch.no_grad() allows it)");
    if (!t.is_cuda()) bad(s.name[j], "not on the GPU");
    const int d = t.get_device();
    if (device < 0) device = d;
    if (d != device) bad(s.name[j], "on another GPU than the other tensors");
    return t.data_ptr();
  }
  // A contiguous vector of at least n elements.
  template <class T>
  T* vec(int j, at::ScalarType type, int64_t n) {
    const at::Tensor& t = tensor(j);
    if (t.is_cuda() && (t.scalar_type() != type || !t.is_contiguous() || t.numel() < n))
      bad(s.name[j], "needs %lld contiguous elements of %s", (long long)n, c10::toString(type));
    return static_cast<T*>(address(j, t));
  }
  // The block tables: address, row stride, width.
  int32_t* table(int j, int64_t rows, int64_t& stride, int& width) {
    const at::Tensor& t = tensor(j);
    if (t.dim() != 2 || t.scalar_type() != at::kInt || !t.is_cuda() || t.size(0) < rows ||
        (t.size(1) > 1 && t.stride(1) != 1) || t.size(1) > INT32_MAX)
      bad(s.name[j], "needs an int32 [%lld, pages] tensor on the GPU with contiguous rows", (long long)rows);
    width = static_cast<int>(t.size(1));
    stride = t.size(0) > 1 ? t.stride(0) : width;
    return static_cast<int32_t*>(address(j, t));
  }
  // A [tokens, heads, head_dim] tensor with a contiguous last dimension.
  void* heads(int j, at::ScalarType type, int64_t tokens, int64_t n, int64_t dim, int64_t& token,
              int64_t& head) {
    const at::Tensor& t = tensor(j);
    void* a = address(j, t);
    if (t.scalar_type() != type || t.dim() != 3)
      bad(s.name[j], "needs [tokens, heads, head_dim] of %s", c10::toString(type));
    const auto size = t.sizes(), stride = t.strides();
    if (stride[2] != 1 && size[2] != 1) bad(s.name[j], "its last dimension is not contiguous");
    if (size[0] != tokens || size[1] != n || size[2] != dim)
      bad(s.name[j], "needs [%lld, %lld, %lld], got [%lld, %lld, %lld]", (long long)tokens, (long long)n,
          (long long)dim, (long long)size[0], (long long)size[1], (long long)size[2]);
    // a dimension of size one may have any stride
    token = size[0] == 1 ? 0 : stride[0], head = size[1] == 1 ? 0 : stride[1];
    return a;
  }
  // The sizes of the tensor that sets a call's geometry.
  const at::Tensor& shape3(int j, int& dtype, at::ScalarType& type) {
    const at::Tensor& t = tensor(j);
    type = t.scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat)
      bad("dtype", "%s is torch.bfloat16 or torch.float32, got %s", s.name[j], c10::toString(type));
    if (t.dim() != 3) bad(s.name[j], "needs [tokens, heads, head_dim]");
    for (int i = 0; i < 3; ++i)
      if (t.size(i) > INT32_MAX) bad(s.name[j], "too large");
    dtype = type == at::kBFloat16 ? AR_BFLOAT16 : AR_FLOAT32;
    return t;
  }
  int64_t integer(int j, int64_t otherwise) {
    if (p.at[j] == nullptr) return otherwise;
    const long long v = PyLong_AsLongLong(p.at[j]);
    if (v == -1 && PyErr_Occurred()) throw Bad();
    return v;
  }
  int small(int j, int otherwise) {
    const int64_t v = integer(j, otherwise);
    if (v < INT32_MIN || v > INT32_MAX) bad(s.name[j], "out of range");
    return static_cast<int>(v);
  }
  double real(int j, double otherwise) {
    if (p.at[j] == nullptr) return otherwise;
    const double v = PyFloat_AsDouble(p.at[j]);
    if (v == -1.0 && PyErr_Occurred()) throw Bad();
    return v;
  }
  int truth(int j) {
    if (p.at[j] == nullptr) return 0;
    const int v = PyObject_IsTrue(p.at[j]);
    if (v < 0) throw Bad();
    return v;
  }
  // The call's stream: an address, an object with `cuda_stream`, or torch's current one.
  void* stream(int j) {
    PyObject* o = p.at[j];
    if (o == nullptr) return c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(device)).stream();
    PyObject* owned = nullptr;
    if (!PyLong_Check(o)) {
      owned = PyObject_GetAttr(o, g_cuda_stream);
      if (owned == nullptr) throw Bad();
      o = owned;
    }
    void* v = PyLong_AsVoidPtr(o);
    Py_XDECREF(owned);
    if (v == nullptr && PyErr_Occurred()) throw Bad();
    return v;
  }
};

// The GPU of a call's tensors as the current one, for the launch: a stream belongs to its GPU.
struct Here {
  std::optional<c10::DeviceGuard> guard;
  explicit Here(const Reader& r) {
    if (r.device >= 0 && r.device != c10::hip::current_device())
      guard.emplace(c10::Device(c10::DeviceType::CUDA, static_cast<c10::DeviceIndex>(r.device)));
  }
};

struct Handle {
  ar_kv4* h;
  long heads, dim, page, device;
  explicit Handle(PyObject* o) {
    PyObject* v = o == nullptr ? nullptr : PyObject_GetAttr(o, g_value);
    PyObject* g = v == nullptr ? nullptr : PyObject_GetAttr(o, g_geometry);
    PyObject* d = g == nullptr ? nullptr : PyObject_GetAttr(o, g_device);
    if (d == nullptr) {
      Py_XDECREF(v);
      Py_XDECREF(g);
      PyErr_Clear();
      bad("h", "needs a handle of ar_kv4_create");
    }
    device = PyLong_AsLong(d);
    Py_DECREF(d);
    h = v == Py_None ? nullptr : static_cast<ar_kv4*>(PyLong_AsVoidPtr(v));
    long* to[3] = {&heads, &dim, &page};
    for (int i = 0; i < 3; ++i)
      *to[i] = PyTuple_Check(g) && PyTuple_GET_SIZE(g) == 3 ? PyLong_AsLong(PyTuple_GET_ITEM(g, i)) : 0;
    Py_DECREF(v);
    Py_DECREF(g);
    if (PyErr_Occurred()) throw Bad();
  }
  // After the call's tensors are read.
  void check_place(const Reader& r) const {
    if (device >= 0 && r.device >= 0 && r.device != device)
      bad("h", "made on GPU %ld, the tensors are on GPU %d", device, r.device);
  }
};

void cache(Reader& r, int j, const Handle& h, uint8_t*& data, uint8_t*& scales, int64_t& pages) {
  const at::Tensor &d = r.tensor(j), &s = r.tensor(j + 1);
  data = static_cast<uint8_t*>(r.address(j, d));
  scales = static_cast<uint8_t*>(r.address(j + 1, s));
  if (d.scalar_type() != at::kByte || s.scalar_type() != at::kByte || !d.is_contiguous() ||
      !s.is_contiguous() || d.dim() < 1)
    bad("cache", "needs contiguous uint8 tensors");
  pages = d.size(0);
  if (d.numel() != pages * h.heads * h.page * h.dim || s.numel() != pages * h.heads * 2 * h.page * (h.dim / 32))
    bad("cache", "data [pages, %ld, 2, %ld] and scales [pages, %ld, 2, %ld, %ld] are wanted", h.heads,
        h.page * h.dim / 2, h.heads, h.dim / 32, h.page);
}

PyObject* done(int rc) {
  if (rc == AR_OK) Py_RETURN_NONE;
  PyObject* e = PyObject_CallFunction(g_error, "is", rc, ar_last_error());
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

// No C++ exception passes into the interpreter.
template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Bad&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

const Signature kTables = {"ar_page_tables", 13, 12,
                           {"cached_len", "new_len", "pool", "free_pages", "table", "kv_len", "q_start",
                            "slots", "positions", "pool_out", "refused", "page_size", "stream"}};

PyObject* page_tables(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&] {
    const Params p(kTables, args, n, kw);
    Reader r{kTables, p};
    const int64_t b = r.tensor(0).numel(), t = r.tensor(7).numel(), nfree = r.tensor(3).numel();
    if (b > INT32_MAX || t > INT32_MAX || nfree > INT32_MAX) bad("cached_len", "too large");
    ar_page_tables_args a;
    a.table = r.table(4, b, a.table_stride, a.table_width);
    a.cached_len = r.vec<int32_t>(0, at::kInt, b);
    a.new_len = r.vec<int32_t>(1, at::kInt, b);
    a.pool = r.vec<int32_t>(2, at::kInt, 2);
    a.free_pages = r.vec<int32_t>(3, at::kInt, 0);
    a.kv_len = r.vec<int32_t>(5, at::kInt, b);
    a.q_start = r.vec<int32_t>(6, at::kInt, b + 1);
    a.slots = r.vec<int64_t>(7, at::kLong, 0);
    a.positions = r.vec<int32_t>(8, at::kInt, t);
    a.pool_out = r.vec<int32_t>(9, at::kInt, 2);
    a.refused = r.vec<int32_t>(10, at::kInt, b);
    a.nreq = static_cast<int>(b), a.nfree = static_cast<int>(nfree), a.ntokens = static_cast<int>(t);
    a.page_size = r.small(11, 0);
    const Here here(r);
    return done(ar_page_tables(&a, r.stream(12)));
  });
}

// What ar_qk_norm_rope and ar_kv4_norm_rope_append share; j* are the places of their arguments,
// k_out or v negative where a call has none.
void norm_rope(Reader& r, ar_qk_norm_rope_args& a, int q, int k, int v, int q_out, int k_out, int positions,
               int weights) {
  at::ScalarType type;
  const at::Tensor& tq = r.shape3(q, a.dtype, type);
  const at::Tensor& tk = r.tensor(k);
  const int64_t t = tq.size(0), hq = tq.size(1), d = tq.size(2);
  if (tk.dim() != 3 || tk.size(1) > INT32_MAX) bad(r.s.name[k], "needs [tokens, heads, head_dim]");
  const int64_t hkv = tk.size(1);
  a.ntokens = static_cast<int>(t), a.q_heads = static_cast<int>(hq), a.kv_heads = static_cast<int>(hkv);
  a.head_dim = static_cast<int>(d);
  a.q = r.heads(q, type, t, hq, d, a.q_token, a.q_head);
  a.k = r.heads(k, type, t, hkv, d, a.k_token, a.k_head);
  a.q_out = r.heads(q_out, type, t, hq, d, a.qo_token, a.qo_head);
  if (v >= 0) a.v = r.heads(v, type, t, hkv, d, a.v_token, a.v_head);
  if (k_out >= 0) a.k_out = r.heads(k_out, type, t, hkv, d, a.ko_token, a.ko_head);
  if (r.p.at[positions + 1] != nullptr) {
    const at::Tensor& cs = r.tensor(positions + 1);
    if (cs.dim() != 2 || cs.size(0) > INT32_MAX || cs.size(1) > INT32_MAX)
      bad("cos_sin", "needs [rows, rot]");
    a.rows = static_cast<int>(cs.size(0)), a.rot = static_cast<int>(cs.size(1));
    a.cos_sin = r.vec<float>(positions + 1, at::kFloat, 0);
  }
  if (r.p.at[positions] != nullptr) a.positions = r.vec<int32_t>(positions, at::kInt, t);
  else if (a.rot != 0) bad("positions", "a rotation needs them");
  if (r.p.at[weights] != nullptr) a.q_weight = r.vec<void>(weights, type, d);
  if (r.p.at[weights + 1] != nullptr) a.k_weight = r.vec<void>(weights + 1, type, d);
  a.eps = r.real(weights + 2, 1e-6);
  a.interleaved = r.truth(weights + 3);
}

const Signature kRope = {"ar_qk_norm_rope", 11, 4,
                         {"q", "k", "q_out", "k_out", "positions", "cos_sin", "q_weight", "k_weight", "eps",
                          "interleaved", "stream"}};

PyObject* qk_norm_rope(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&] {
    const Params p(kRope, args, n, kw);
    Reader r{kRope, p};
    ar_qk_norm_rope_args a = {};
    norm_rope(r, a, 0, 1, -1, 2, 3, 4, 6);
    const Here here(r);
    return done(ar_qk_norm_rope(&a, r.stream(10)));
  });
}

const Signature kFused = {"ar_kv4_norm_rope_append", 15, 10,
                          {"h", "q", "k", "v", "q_out", "positions", "cos_sin", "slots", "data", "scales",
                           "q_weight", "k_weight", "eps", "interleaved", "stream"}};

PyObject* kv4_norm_rope_append(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&] {
    const Params p(kFused, args, n, kw);
    Reader r{kFused, p};
    const Handle h(p.at[0]);
    ar_qk_norm_rope_args a = {};
    norm_rope(r, a, 1, 2, 3, 4, -1, 5, 10);
    a.slots = r.vec<int64_t>(7, at::kLong, a.ntokens);
    cache(r, 8, h, a.data, a.scales, a.num_pages);
    const Here here(r);
    return done(ar_kv4_norm_rope_append(h.h, &a, r.stream(14)));
  });
}

const Signature kAppend = {"ar_kv4_append", 7, 6, {"h", "k", "v", "slots", "data", "scales", "stream"}};
const Signature kRead = {"ar_kv4_read", 7, 6, {"h", "slots", "data", "scales", "k", "v", "stream"}};

template <int (*CALL)(ar_kv4*, const ar_kv4_rows_args*, void*)>
PyObject* rows(const Signature& s, int k, int slots, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&] {
    const Params p(s, args, n, kw);
    Reader r{s, p};
    const Handle h(p.at[0]);
    ar_kv4_rows_args a = {};
    at::ScalarType type;
    const int64_t t = r.shape3(k, a.dtype, type).size(0);
    a.ntokens = static_cast<int>(t);
    a.k = r.heads(k, type, t, h.heads, h.dim, a.k_token, a.k_head);
    a.v = r.heads(k + 1, type, t, h.heads, h.dim, a.v_token, a.v_head);
    a.slots = r.vec<int64_t>(slots, at::kLong, t);
    cache(r, slots + 1, h, a.data, a.scales, a.num_pages);
    const Here here(r);
    return done(CALL(h.h, &a, r.stream(6)));
  });
}
PyObject* kv4_append(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return rows<ar_kv4_append>(kAppend, 1, 3, args, n, kw);
}
PyObject* kv4_read(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return rows<ar_kv4_read>(kRead, 4, 1, args, n, kw);
}

const Signature kAttention = {"ar_kv4_attention", 12, 8,
                              {"h", "q", "data", "scales", "table", "kv_len", "q_start", "out", "lse",
                               "scale", "window", "stream"}};

PyObject* kv4_attention(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&] {
    const Params p(kAttention, args, n, kw);
    Reader r{kAttention, p};
    const Handle h(p.at[0]);
    ar_kv4_attention_args a = {};
    at::ScalarType type;
    const at::Tensor& q = r.shape3(1, a.dtype, type);
    const int64_t t = q.size(0), hq = q.size(1), d = q.size(2), b = r.tensor(5).numel();
    if (d != h.dim) bad("q", "the handle is for head_dim %ld, got %lld", h.dim, (long long)d);
    if (b > INT32_MAX) bad("kv_len", "too large");
    a.ntokens = static_cast<int>(t), a.q_heads = static_cast<int>(hq), a.nreq = static_cast<int>(b);
    a.table = r.table(4, b, a.table_stride, a.table_width);
    a.q = r.heads(1, type, t, hq, d, a.q_token, a.q_head);
    a.out = r.heads(7, type, t, hq, d, a.o_token, a.o_head);
    if (p.at[8] != nullptr) a.lse = r.vec<float>(8, at::kFloat, t * hq);
    uint8_t *data, *scales;
    cache(r, 2, h, data, scales, a.num_pages);
    a.data = data, a.scales = scales;
    a.kv_len = r.vec<int32_t>(5, at::kInt, b);
    a.q_start = r.vec<int32_t>(6, at::kInt, b + 1);
    a.scale = r.real(9, 1.0 / std::sqrt(static_cast<double>(d)));
    a.window = r.small(10, 0);
    h.check_place(r);
    const Here here(r);
    return done(ar_kv4_attention(h.h, &a, r.stream(11)));
  });
}

// The class of the error that a failing call raises.
PyObject* setup(PyObject*, PyObject* error) {
  Py_INCREF(error);
  Py_XDECREF(g_error);
  g_error = error;
  Py_RETURN_NONE;
}

#define ARD_METHOD(NAME, DOC) \
  {"ar_" #NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(NAME)), METH_FASTCALL | METH_KEYWORDS, "ar_" #NAME DOC}
PyMethodDef kMethods[] = {
    ARD_METHOD(page_tables,
               "(cached_len, new_len, pool, free_pages, table, kv_len, q_start, slots, positions, pool_out, "
               "refused, page_size, stream=None)\n--\n\nBlock tables, slots and positions of a step."),
    ARD_METHOD(qk_norm_rope,
               "(q, k, q_out, k_out, positions=None, cos_sin=None, q_weight=None, k_weight=None, eps=1e-06, "
               "interleaved=False, stream=None)\n--\n\nPer-head norm of q and k with the position rotation."),
    ARD_METHOD(kv4_append, "(h, k, v, slots, data, scales, stream=None)\n--\n\nRows into the 4-bit cache."),
    ARD_METHOD(kv4_read, "(h, slots, data, scales, k, v, stream=None)\n--\n\nRows of the 4-bit cache as values."),
    ARD_METHOD(kv4_norm_rope_append,
               "(h, q, k, v, q_out, positions, cos_sin, slots, data, scales, q_weight=None, k_weight=None, "
               "eps=1e-06, interleaved=False, stream=None)\n--\n\nNorm, rotation and the cache's new rows."),
    ARD_METHOD(kv4_attention,
               "(h, q, data, scales, table, kv_len, q_start, out, lse=None, scale=None, window=0, "
               "stream=None)\n--\n\nAttention over the 4-bit cache."),
    {"_setup", setup, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_decode_calls", nullptr, -1, kMethods, nullptr, nullptr,
                       nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode_calls() {
  g_value = PyUnicode_InternFromString("value");
  g_geometry = PyUnicode_InternFromString("geometry");
  g_device = PyUnicode_InternFromString("device");
  g_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  if (g_value == nullptr || g_geometry == nullptr || g_device == nullptr || g_cuda_stream == nullptr) return nullptr;
  return PyModule_Create(&kModule);
}
