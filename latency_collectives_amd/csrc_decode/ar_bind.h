// What the compiled bindings share: a call's arguments in its signature's order, tensors read and checked,
// handles, and no C++ exception past the interpreter's border. Included once by each module.
#pragma once

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

// A handle's address and GPU, and its geometry: `count` numbers, by which the kinds of handles differ.
struct AnyHandle {
  void* address = nullptr;
  long geometry[4] = {}, device = -1;
  AnyHandle(PyObject* o, int count, const char* maker) {
    PyObject* v = o == nullptr ? nullptr : PyObject_GetAttr(o, g_value);
    PyObject* g = v == nullptr ? nullptr : PyObject_GetAttr(o, g_geometry);
    PyObject* d = g == nullptr ? nullptr : PyObject_GetAttr(o, g_device);
    if (d == nullptr || !PyTuple_Check(g) || PyTuple_GET_SIZE(g) != count) {
      Py_XDECREF(v);
      Py_XDECREF(g);
      Py_XDECREF(d);
      PyErr_Clear();
      bad("h", "needs a handle of %s", maker);
    }
    device = PyLong_AsLong(d);
    Py_DECREF(d);
    address = v == Py_None ? nullptr : PyLong_AsVoidPtr(v);
    for (int i = 0; i < count; ++i) geometry[i] = PyLong_AsLong(PyTuple_GET_ITEM(g, i));
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

// What ar_qk_norm_rope and the norm_rope_append of the caches share; j* are the places of their arguments,
// k_out or v negative where a call has none.
[[maybe_unused]] void norm_rope(Reader& r, ar_qk_norm_rope_args& a, int q, int k, int v, int q_out, int k_out, int positions,
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

// The class of the error that a failing call raises.
PyObject* setup(PyObject*, PyObject* error) {
  Py_INCREF(error);
  Py_XDECREF(g_error);
  g_error = error;
  Py_RETURN_NONE;
}

bool intern_names() {
  g_value = PyUnicode_InternFromString("value");
  g_geometry = PyUnicode_InternFromString("geometry");
  g_device = PyUnicode_InternFromString("device");
  g_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  return g_value != nullptr && g_geometry != nullptr && g_device != nullptr && g_cuda_stream != nullptr;
}

#define ARD_METHOD(NAME, DOC) \
  {"ar_" #NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(NAME)), METH_FASTCALL | METH_KEYWORDS, "ar_" #NAME DOC}

}  // namespace
