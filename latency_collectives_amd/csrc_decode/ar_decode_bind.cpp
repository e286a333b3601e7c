// The decode operators' calls on torch tensors: addresses, sizes and strides out of the tensors,
// checks of what the C entry points cannot see (place, type, shape), then the C entry point.
//
// These calls sit between short kernels of a decode step, so what they cost on the host decides
// the step's rate: reading a call's tensors through the interpreter (attributes, methods, a packed
// struct) took 5.0 us of a 7.6 us call, reading them here takes 0.4 us.

#include "ar_bind.h"

namespace {

struct Handle : AnyHandle {
  ar_kv4* h;
  long heads, dim, page;
  explicit Handle(PyObject* o)
      : AnyHandle(o, 3, "ar_kv4_create"), h(static_cast<ar_kv4*>(address)), heads(geometry[0]), dim(geometry[1]), page(geometry[2]) {}
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
  if (!intern_names()) return nullptr;
  return PyModule_Create(&kModule);
}
