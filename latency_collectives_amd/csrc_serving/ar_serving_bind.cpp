// The serving operators' calls on torch tensors, as ar_decode_bind.cpp has those of the decode operators.

#include "../csrc_decode/ar_bind.h"

#include <vector>

#include "../../include/ar_serving.h"

namespace {

struct Handle8 : AnyHandle {  // (kv_heads, head_dim, page_size, bits)
  ar_kv8* h;
  long heads, dim, page;
  explicit Handle8(PyObject* o)
      : AnyHandle(o, 4, "ar_kv8_create"), h(static_cast<ar_kv8*>(address)), heads(geometry[0]), dim(geometry[1]), page(geometry[2]) {}
};

void cache8(Reader& r, int j, const Handle8& h, uint8_t*& data, uint8_t*& scales, int64_t& pages) {
  const at::Tensor &d = r.tensor(j), &s = r.tensor(j + 1);
  data = static_cast<uint8_t*>(r.address(j, d));
  scales = static_cast<uint8_t*>(r.address(j + 1, s));
  if (d.scalar_type() != at::kByte || s.scalar_type() != at::kByte || !d.is_contiguous() || !s.is_contiguous() || d.dim() < 1)
    bad("cache", "needs contiguous uint8 tensors");
  pages = d.size(0);
  if (d.numel() != pages * h.heads * 2 * h.page * h.dim || s.numel() != pages * h.heads * 2 * (h.page / 16))
    bad("cache", "data [pages, %ld, 2, %ld] and scales [pages, %ld, %ld, 2] are wanted", h.heads, h.page * h.dim, h.heads, h.page / 16);
}

const Signature kAppend = {"ar_kv8_append", 7, 6, {"h", "k", "v", "slots", "data", "scales", "stream"}};
const Signature kRead = {"ar_kv8_read", 7, 6, {"h", "slots", "data", "scales", "k", "v", "stream"}};

template <int (*CALL)(ar_kv8*, const ar_kv8_rows_args*, void*)>
PyObject* rows8(const Signature& s, int k, int slots, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&] {
    const Params p(s, args, n, kw);
    Reader r{s, p};
    const Handle8 h(p.at[0]);
    ar_kv8_rows_args a = {};
    at::ScalarType type;
    const int64_t t = r.shape3(k, a.dtype, type).size(0);
    a.ntokens = static_cast<int>(t);
    a.k = r.heads(k, type, t, h.heads, h.dim, a.k_token, a.k_head);
    a.v = r.heads(k + 1, type, t, h.heads, h.dim, a.v_token, a.v_head);
    a.slots = r.vec<int64_t>(slots, at::kLong, t);
    cache8(r, slots + 1, h, a.data, a.scales, a.num_pages);
    const Here here(r);
    return done(CALL(h.h, &a, r.stream(6)));
  });
}
PyObject* kv8_append(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return rows8<ar_kv8_append>(kAppend, 1, 3, args, n, kw);
}
PyObject* kv8_read(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return rows8<ar_kv8_read>(kRead, 4, 1, args, n, kw);
}

const Signature kFused = {"ar_kv8_norm_rope_append", 15, 10,
                          {"h", "q", "k", "v", "q_out", "positions", "cos_sin", "slots", "data", "scales",
                           "q_weight", "k_weight", "eps", "interleaved", "stream"}};

PyObject* kv8_norm_rope_append(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&] {
    const Params p(kFused, args, n, kw);
    Reader r{kFused, p};
    const Handle8 h(p.at[0]);
    ar_qk_norm_rope_args a = {};
    norm_rope(r, a, 1, 2, 3, 4, -1, 5, 10);
    a.slots = r.vec<int64_t>(7, at::kLong, a.ntokens);
    cache8(r, 8, h, a.data, a.scales, a.num_pages);
    const Here here(r);
    return done(ar_kv8_norm_rope_append(h.h, &a, r.stream(14)));
  });
}

const Signature kAttention = {"ar_kv8_attention", 12, 8,
                              {"h", "q", "data", "scales", "table", "kv_len", "q_start", "out", "lse",
                               "scale", "window", "stream"}};

PyObject* kv8_attention(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&] {
    const Params p(kAttention, args, n, kw);
    Reader r{kAttention, p};
    const Handle8 h(p.at[0]);
    ar_kv8_attention_args a = {};
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
    cache8(r, 2, h, data, scales, a.num_pages);
    a.data = data, a.scales = scales;
    a.kv_len = r.vec<int32_t>(5, at::kInt, b);
    a.q_start = r.vec<int32_t>(6, at::kInt, b + 1);
    a.scale = r.real(9, 1.0 / std::sqrt(static_cast<double>(d)));
    a.window = r.small(10, 0);
    h.check_place(r);
    const Here here(r);
    return done(ar_kv8_attention(h.h, &a, r.stream(11)));
  });
}

const Signature kPrompt = {"ar_prompt_attention", 10, 6,
                           {"h", "q", "k", "v", "q_start", "out", "lse", "scale", "window", "stream"}};

PyObject* prompt_attention(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&] {
    const Params p(kPrompt, args, n, kw);
    Reader r{kPrompt, p};
    const AnyHandle h(p.at[0], 2, "ar_prompt_create");  // (kv_heads, head_dim)
    ar_prompt_attention_args a = {};
    at::ScalarType type;
    const at::Tensor& q = r.shape3(1, a.dtype, type);
    const int64_t t = q.size(0), hq = q.size(1), d = q.size(2), hkv = h.geometry[0];
    if (d != h.geometry[1]) bad("q", "the handle is for head_dim %ld, got %lld", h.geometry[1], (long long)d);
    a.ntokens = static_cast<int>(t), a.q_heads = static_cast<int>(hq);
    a.q = r.heads(1, type, t, hq, d, a.q_token, a.q_head);
    a.k = r.heads(2, type, t, hkv, d, a.k_token, a.k_head);
    a.v = r.heads(3, type, t, hkv, d, a.v_token, a.v_head);
    const int64_t starts = r.tensor(4).numel();
    if (starts < 1 || starts > INT32_MAX) bad("q_start", "needs a start for each request and the end");
    a.q_start = r.vec<int32_t>(4, at::kInt, starts);
    a.nreq = static_cast<int>(starts - 1);
    a.out = r.heads(5, type, t, hq, d, a.o_token, a.o_head);
    if (p.at[6] != nullptr) a.lse = r.vec<float>(6, at::kFloat, t * hq);
    a.scale = r.real(7, 1.0 / std::sqrt(static_cast<double>(d)));
    a.window = r.small(8, 0);
    h.check_place(r);
    const Here here(r);
    return done(ar_prompt_attention(static_cast<ar_prompt*>(h.address), &a, r.stream(9)));
  });
}

// A vector's length as an int.
int length(Reader& r, int j) {
  const int64_t n = r.tensor(j).numel();
  if (n > INT32_MAX) bad(r.s.name[j], "too large");
  return static_cast<int>(n);
}

const Signature kFork = {"ar_pages_fork", 14, 13,
                         {"src", "dst", "kv_len", "table", "shares", "pool", "free_pages", "kv_len_out", "pool_out",
                          "copy_src", "copy_dst", "refused", "page_size", "stream"}};

PyObject* pages_fork(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&] {
    const Params p(kFork, args, n, kw);
    Reader r{kFork, p};
    ar_pages_fork_args a = {};
    a.count = length(r, 0), a.nreq = length(r, 2), a.num_pages = length(r, 4), a.nfree = length(r, 6);
    a.table = r.table(3, a.nreq, a.table_stride, a.table_width);
    a.src = r.vec<int32_t>(0, at::kInt, a.count);
    a.dst = r.vec<int32_t>(1, at::kInt, a.count);
    a.kv_len = r.vec<int32_t>(2, at::kInt, a.nreq);
    a.shares = r.vec<int32_t>(4, at::kInt, 1);
    a.pool = r.vec<int32_t>(5, at::kInt, 2);
    a.free_pages = r.vec<int32_t>(6, at::kInt, 0);
    a.kv_len_out = r.vec<int32_t>(7, at::kInt, a.nreq);
    a.pool_out = r.vec<int32_t>(8, at::kInt, 2);
    a.copy_src = r.vec<int32_t>(9, at::kInt, a.count);
    a.copy_dst = r.vec<int32_t>(10, at::kInt, a.count);
    a.refused = r.vec<int32_t>(11, at::kInt, a.count);
    a.page_size = r.small(12, 0);
    const Here here(r);
    return done(ar_pages_fork(&a, r.stream(13)));
  });
}

const Signature kFree = {"ar_pages_free", 11, 10,
                         {"requests", "kv_len", "table", "shares", "pool", "free_pages", "kv_len_out", "pool_out",
                          "scratch", "page_size", "stream"}};

PyObject* pages_free(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&] {
    const Params p(kFree, args, n, kw);
    Reader r{kFree, p};
    ar_pages_free_args a = {};
    a.count = length(r, 0), a.nreq = length(r, 1), a.num_pages = length(r, 3), a.nfree = length(r, 5);
    a.table = r.table(2, a.nreq, a.table_stride, a.table_width);
    a.requests = r.vec<int32_t>(0, at::kInt, a.count);
    a.kv_len = r.vec<int32_t>(1, at::kInt, a.nreq);
    a.shares = r.vec<int32_t>(3, at::kInt, 1);
    a.pool = r.vec<int32_t>(4, at::kInt, 2);
    a.free_pages = r.vec<int32_t>(5, at::kInt, 0);
    a.kv_len_out = r.vec<int32_t>(6, at::kInt, a.nreq);
    a.pool_out = r.vec<int32_t>(7, at::kInt, 2);
    a.scratch = r.vec<uint32_t>(8, at::kInt, (static_cast<int64_t>(a.num_pages) + 31) / 32 + 1);
    a.page_size = r.small(9, 0);
    const Here here(r);
    return done(ar_pages_free(&a, r.stream(10)));
  });
}

const Signature kCompact = {"ar_pages_compact", 12, 11,
                            {"kv_len", "table", "shares", "table_out", "shares_out", "free_pages", "pool_out",
                             "move_src", "move_dst", "scratch", "page_size", "stream"}};

PyObject* pages_compact(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&] {
    const Params p(kCompact, args, n, kw);
    Reader r{kCompact, p};
    ar_pages_compact_args a = {};
    a.nreq = length(r, 0), a.num_pages = length(r, 2), a.nfree = length(r, 5), a.nmoves = length(r, 7);
    a.table = r.table(1, a.nreq, a.table_stride, a.table_width);
    int width;
    a.table_out = r.table(3, a.nreq, a.out_stride, width);
    if (width != a.table_width) bad("table_out", "needs %d pages a row, got %d", a.table_width, width);
    a.kv_len = r.vec<int32_t>(0, at::kInt, a.nreq);
    a.shares = r.vec<int32_t>(2, at::kInt, 1);
    a.shares_out = r.vec<int32_t>(4, at::kInt, a.num_pages);
    a.free_pages = r.vec<int32_t>(5, at::kInt, a.num_pages);
    a.pool_out = r.vec<int32_t>(6, at::kInt, 2);
    a.move_src = r.vec<int32_t>(7, at::kInt, a.num_pages / 2);
    a.move_dst = r.vec<int32_t>(8, at::kInt, a.nmoves);
    a.scratch = r.vec<uint32_t>(9, at::kInt, (static_cast<int64_t>(a.num_pages) + 31) / 32 + 1);
    a.page_size = r.small(10, 0);
    const Here here(r);
    return done(ar_pages_compact(&a, r.stream(11)));
  });
}

const Signature kCopy = {"ar_pages_copy", 4, 3, {"buffers", "src", "dst", "stream"}};

PyObject* pages_copy(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    const Params p(kCopy, args, n, kw);
    Reader r{kCopy, p};
    PyObject* list = p.at[0];
    if (list == nullptr || !(PyList_Check(list) || PyTuple_Check(list))) bad("buffers", "needs a list or a tuple of tensors");
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(list);
    if (count > INT32_MAX) bad("buffers", "too large");
    std::vector<void*> address(count);
    std::vector<int64_t> bytes(count);
    ar_pages_copy_args a = {};
    for (Py_ssize_t i = 0; i < count; ++i) {
      PyObject* o = PySequence_Fast_GET_ITEM(list, i);
      if (!THPVariable_Check(o)) bad("buffers", "needs tensors");
      const at::Tensor& t = THPVariable_Unpack(o);
      address[i] = r.address(0, t);
      if (t.dim() < 1 || !t.is_contiguous()) bad("buffers", "needs contiguous tensors [pages, ...]");
      const int64_t pages = t.size(0);
      if (pages > INT32_MAX) bad("buffers", "too large");
      if (i == 0) a.num_pages = static_cast<int>(pages);
      if (pages != a.num_pages) bad("buffers", "need the same number of pages, got %d and %lld", a.num_pages, (long long)pages);
      bytes[i] = pages == 0 ? 0 : static_cast<int64_t>(t.nbytes()) / pages;
    }
    a.buffers = address.data(), a.page_bytes = bytes.data(), a.nbuffers = static_cast<int>(count);
    a.count = length(r, 1);
    a.src = r.vec<int32_t>(1, at::kInt, a.count);
    a.dst = r.vec<int32_t>(2, at::kInt, a.count);
    const Here here(r);
    return done(ar_pages_copy(&a, r.stream(3)));
  });
}

PyMethodDef kMethods[] = {
    ARD_METHOD(kv8_append, "(h, k, v, slots, data, scales, stream=None)\n--\n\nRows into the 8-bit cache."),
    ARD_METHOD(kv8_read, "(h, slots, data, scales, k, v, stream=None)\n--\n\nRows of the 8-bit cache as values."),
    ARD_METHOD(kv8_norm_rope_append,
               "(h, q, k, v, q_out, positions, cos_sin, slots, data, scales, q_weight=None, k_weight=None, "
               "eps=1e-06, interleaved=False, stream=None)\n--\n\nNorm, rotation and the 8-bit cache's new rows."),
    ARD_METHOD(kv8_attention,
               "(h, q, data, scales, table, kv_len, q_start, out, lse=None, scale=None, window=0, "
               "stream=None)\n--\n\nAttention over the 8-bit cache."),
    ARD_METHOD(pages_fork,
               "(src, dst, kv_len, table, shares, pool, free_pages, kv_len_out, pool_out, copy_src, copy_dst, "
               "refused, page_size, stream=None)\n--\n\nRequests that share another's pages."),
    ARD_METHOD(pages_copy, "(buffers, src, dst, stream=None)\n--\n\nPages of a list, in every buffer."),
    ARD_METHOD(pages_free,
               "(requests, kv_len, table, shares, pool, free_pages, kv_len_out, pool_out, scratch, page_size, "
               "stream=None)\n--\n\nRequests' pages back to the free list."),
    ARD_METHOD(pages_compact,
               "(kv_len, table, shares, table_out, shares_out, free_pages, pool_out, move_src, move_dst, scratch, "
               "page_size, stream=None)\n--\n\nThe pages in use to the lowest ids."),
    ARD_METHOD(prompt_attention,
               "(h, q, k, v, q_start, out, lse=None, scale=None, window=0, stream=None)\n--\n\n"
               "Causal attention over packed prompts."),
    {"_setup", setup, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_serving_calls", nullptr, -1, kMethods, nullptr, nullptr,
                       nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving_calls() {
  if (!intern_names()) return nullptr;
  return PyModule_Create(&kModule);
}
