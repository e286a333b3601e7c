/*
 * ar_decode.h -- C ABI of the decode operators: what one tensor-parallel rank computes between two
 * AllReduces (ar.h) of a decode step, over its own heads, on one MI355X (gfx950).
 *
 *   ar_page_tables           block tables, slots, positions of a step from the requests' lengths
 *   ar_qk_norm_rope          per-head RMS norm of q and k with the position rotation, one pass
 *   ar_kv4_append            keys and values into a paged cache held in 4 bits
 *   ar_kv4_norm_rope_append  the two above in one launch (the form of a decode step)
 *   ar_kv4_read              rows of the cache as values
 *   ar_kv4_attention         attention over the cache, from one new token a request to prompt chunks
 *
 * Conventions are those of ar.h: device pointers from any HIP allocator, `stream` a hipStream_t,
 * AR_OK or a negative AR_E* code with a message in ar_last_error(). Every call only enqueues one
 * launch on `stream` and can be captured into a graph. Arguments are checked before anything is
 * launched; what lies in device memory (lengths, page ids, slots, positions) is bounded by the
 * kernels themselves, as each entry point says. Strides are in elements; the last dimension is
 * contiguous. Types are AR_FLOAT32 and AR_BFLOAT16.
 */
#ifndef LATENCY_COLLECTIVES_AR_DECODE_H
#define LATENCY_COLLECTIVES_AR_DECODE_H

#include "ar.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * ar_page_tables: a step's block tables and slots. Request b holds cached_len[b] tokens and brings
 * new_len[b]; its tokens live in pages of page_size tokens, table[b * table_stride + j] the page of
 * tokens j * page_size and on. Requests take the pages they lack from the free list in order:
 *   need[b] = ceil((cached + new) / page_size) - ceil(cached / page_size)
 * pages, the entries free_pages[pool[0] + need[0] + .. + need[b-1]] and on, where need is 0 for a
 * request refused for its lengths, its row or its places, but not for one that finds too few pages:
 * those after it that need any find too few as well. Written are
 *   table                 the new entries only
 *   kv_len[b]             cached_len[b] + new_len[b]
 *   q_start[0..nreq]      where each request's new tokens start among the step's tokens
 *   slots[i]              page * page_size + offset of new token i
 *   positions[i]          its position in its request
 *   pool_out[0..1]        pool[0] (at least 0) + pages taken, pool[1]
 *   refused[b]            0, or 1 for a request that got nothing: the free list has too few pages
 *                         left, its row of the table or the step's ntokens are too short, or a
 *                         length is negative. Its kv_len stays cached_len[b] (at least 0), its
 *                         tokens keep their places (slots and positions -1), its table row stays.
 * Tokens from q_start[nreq] to ntokens are padding: slots and positions -1. What the calls below
 * give for tokens without a position means nothing: ar_kv4_norm_rope_append leaves their rows of
 * q_out, and ar_kv4_attention attends with those for a refused request, whose tokens q_start still
 * counts. A caller masks them by their positions. pool and the lengths are read only, so a call can
 * be repeated; pool_out and kv_len must be other buffers. The free list is entries
 * [pool[0], min(pool[1], nfree)). A negative page id gives slots -1.
 */
typedef struct {
  const int32_t* cached_len; /* [nreq] */
  const int32_t* new_len;    /* [nreq] */
  const int32_t* pool;       /* [2] first and end of the free pages within free_pages */
  const int32_t* free_pages; /* [nfree] */
  int32_t* table;            /* [nreq][table_stride] */
  int32_t* kv_len;           /* [nreq] */
  int32_t* q_start;          /* [nreq + 1] */
  int64_t* slots;            /* [ntokens] */
  int32_t* positions;        /* [ntokens] */
  int32_t* pool_out;         /* [2] */
  int32_t* refused;          /* [nreq] */
  int64_t table_stride;
  int nreq;        /* 0..4096 */
  int table_width; /* pages a row holds */
  int nfree;
  int ntokens; /* places for new tokens */
  int page_size;
} ar_page_tables_args;
int ar_page_tables(const ar_page_tables_args* a, void* stream);

/*
 * ar_qk_norm_rope: for every token t and head, with x its head_dim values,
 *   y = x / sqrt(mean(x^2) + eps) * weight          (where the weight is given)
 *   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)   over the first `rot` elements
 * with pairs (i, i + rot/2), or (2i, 2i+1) with `interleaved`; cos and sin of pair i are
 * cos_sin[p][i] and cos_sin[p][rot/2 + i] of the token's position p. Computed in 64 bits, rounded
 * to binary32 and, for AR_BFLOAT16, from there. head_dim a multiple of 8 up to 256, rot a multiple of 8 up to head_dim, 0 for none (then
 * positions and cos_sin may be NULL). A token of negative position is padding: nothing is written
 * for it. A position at or beyond `rows` gives NaN. q_out may be q and k_out k (in place, equal
 * strides). q_heads or kv_heads may be 0. Addresses and strides are multiples of 4 elements.
 */
typedef struct {
  const void* q;
  const void* k;
  const void* v; /* ar_kv4_norm_rope_append only */
  void* q_out;
  void* k_out; /* ar_qk_norm_rope only */
  const int32_t* positions; /* [ntokens] */
  const float* cos_sin;     /* [rows][rot] */
  const void* q_weight;     /* [head_dim] of the tensors' type, or NULL */
  const void* k_weight;
  const int64_t* slots; /* [ntokens], ar_kv4_norm_rope_append only */
  uint8_t* data;        /* the cache, ar_kv4_norm_rope_append only */
  uint8_t* scales;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;
  int64_t qo_token, qo_head, ko_token, ko_head;
  int64_t num_pages; /* ar_kv4_norm_rope_append only */
  double eps;
  int dtype, ntokens, q_heads, kv_heads, head_dim, rot, rows, interleaved;
} ar_qk_norm_rope_args;
int ar_qk_norm_rope(const ar_qk_norm_rope_args* a, void* stream);

/*
 * The paged cache in 4 bits. For every page and kv head: K and V of page_size tokens, a code of 4
 * bits an element (e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign) and a scale byte for every 32
 * elements of a row (s stands for 2^(s - 127); above 252: the 32 elements are NaN).
 *   data   uint8 [num_pages][kv_heads][2][page_size * head_dim / 2]      0: K, 1: V
 *          K: [token][head_dim / 2], element 2i in the low half of byte i
 *          V: [token / 4][head_dim / 8][token % 4][4]: eight elements of four tokens side by side,
 *             so that the operand of the attention's second product is one 16-byte load
 *   scales uint8 [num_pages][kv_heads][2][head_dim / 32][page_size]
 * The scale of a group is the smallest power of two, 2^-126 to 2^125, of which no element is over
 * six times; codes are the nearest, ties to the even code. A group with a NaN or an infinity
 * becomes NaN.
 *
 * ar_kv4_create: a handle for caches of one geometry: kv_heads 1..1024, head_dim 64, 96, 128, 192
 * or 256, page_size a power of two, 16..1024. It owns the attention's workspace (35 to 70 MB); the
 * caches themselves are the caller's, one handle serves every layer. As with ar_create, calls on
 * one handle are issued in order on one stream (only ar_kv4_attention uses the workspace).
 * It belongs to the GPU that is current when it is created, where ar_kv4_attention has to be
 * called; AR_EINVAL elsewhere. Synchronous. NULL on error. On a machine without a GPU the handle has
 * no workspace: its calls check their arguments and then return AR_EHIP.
 */
typedef struct ar_kv4 ar_kv4;
ar_kv4* ar_kv4_create(int kv_heads, int head_dim, int page_size);
void ar_kv4_destroy(ar_kv4* h);

/*
 * ar_kv4_append: token t's rows k and v to slot slots[t] (page * page_size + offset); a slot
 * outside the cache, as -1, is skipped. Two tokens with one slot leave it undefined.
 * ar_kv4_read: the rows at `slots` as values of `dtype` in k and v (zeros for a slot outside).
 * dtype is that of k and v. Addresses and strides are multiples of 4 elements.
 */
typedef struct {
  void* k;
  void* v;
  const int64_t* slots;
  uint8_t* data;
  uint8_t* scales;
  int64_t k_token, k_head, v_token, v_head;
  int64_t num_pages;
  int dtype, ntokens;
} ar_kv4_rows_args;
int ar_kv4_append(ar_kv4* h, const ar_kv4_rows_args* a, void* stream);
int ar_kv4_read(ar_kv4* h, const ar_kv4_rows_args* a, void* stream);

/*
 * ar_kv4_norm_rope_append: ar_qk_norm_rope with the rotated keys, rounded to dtype, and the values
 * going straight into the cache: what ar_qk_norm_rope and ar_kv4_append give, in one launch.
 * kv_heads and head_dim must be the handle's. Padding tokens (negative position) write nothing.
 */
int ar_kv4_norm_rope_append(ar_kv4* h, const ar_qk_norm_rope_args* a, void* stream);

/*
 * ar_kv4_attention: with request b's tokens q_start[b] .. q_start[b+1]-1 the last ones of its
 * kv_len[b], token i of m at position p = kv_len - m + i,
 *   out[i] = sum_t softmax_t(scale * q[i] . k[t]) v[t]  over 0 <= t <= p, t < kv_len, and with
 * window > 0 also t > p - window. q has q_heads = kv_heads * group heads, head h reads kv head
 * h / group. A row that sees nothing (p < 0), or scores of minus infinity alone, gives zeros and
 * lse = -inf; one with a score that is NaN or plus infinity NaN for both. lse [ntokens][q_heads], or
 * NULL, is the natural logarithm of the row's sum of exponentials. Statistics and sums are
 * binary32; probabilities are rounded to bfloat16 for AR_BFLOAT16 (their products with the values,
 * which 4 bits hold exactly, are summed in binary32), kept to 24 bits for AR_FLOAT32; queries and
 * keys enter their products as they are. Which parts a row's sums are joined from depends on the
 * whole call's lengths, so a request's last bits may change with the others'.
 * Masked places do not reach a result whatever they hold. Page ids outside [0, num_pages) and
 * tokens beyond table_width * page_size count as masked. table_width is also what the host knows of
 * the lengths when it chooses between kernels: the width that the step needs serves better than the
 * buffer's. Lengths and starts must not change while a call runs: it stays inside its buffers, but
 * its results and those of the handle's later calls may be wrong; a new handle is needed then.
 * Tokens that no request covers keep their rows of out. q and out 16-byte aligned, their strides
 * multiples of 16 bytes.
 */
typedef struct {
  const void* q;
  void* out;
  float* lse;
  const uint8_t* data;
  const uint8_t* scales;
  const int32_t* table;   /* [nreq][table_stride] */
  const int32_t* kv_len;  /* [nreq] */
  const int32_t* q_start; /* [nreq + 1] */
  int64_t q_token, q_head, o_token, o_head;
  int64_t table_stride;
  int64_t num_pages;
  double scale;
  int dtype, ntokens, q_heads, nreq, table_width, window;
} ar_kv4_attention_args;
int ar_kv4_attention(ar_kv4* h, const ar_kv4_attention_args* a, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LATENCY_COLLECTIVES_AR_DECODE_H */
