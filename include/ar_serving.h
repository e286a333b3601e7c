/*
 * ar_serving.h -- C ABI of the serving operators beside those of ar_decode.h: a paged cache held in
 * 8 bits with the attention that reads it, the life of a cache's pages after ar_page_tables has
 * given them out, and attention over prompts that are not in a cache.
 *
 *   ar_kv8_append            keys and values into a paged cache held in 8 bits
 *   ar_kv8_norm_rope_append  norm, rotation and append in one launch (the form of a decode step)
 *   ar_kv8_read              rows of the cache as values
 *   ar_kv8_attention         attention over the cache, from one new token a request to prompt chunks
 *   ar_pages_fork            requests that share another's pages
 *   ar_pages_copy            pages of a list, in any number of caches
 *   ar_pages_free            requests' pages back to the free list
 *   ar_pages_compact         the pages in use to the lowest ids
 *   ar_prompt_attention      causal attention over packed prompts of different lengths
 *
 * Conventions are those of ar_decode.h: device pointers, `stream` a hipStream_t, AR_OK or a negative
 * AR_E* code with a message in ar_last_error(). Calls only enqueue work on `stream` and can be
 * captured into a graph. Arguments are checked before anything is launched; what lies in device
 * memory (lengths, page ids, slots, request numbers) is bounded by the kernels. Strides are in
 * elements; the last dimension is contiguous. Types are AR_FLOAT32 and AR_BFLOAT16.
 */
#ifndef LATENCY_COLLECTIVES_AR_SERVING_H
#define LATENCY_COLLECTIVES_AR_SERVING_H

#include "ar_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The paged cache in 8 bits. For every page and kv head: K and V of page_size tokens, a code of 8
 * bits an element (e4m3: a sign, four exponent bits, three mantissa bits; 448 the largest, 0x7F NaN),
 * and for every block of 16 tokens a scale byte for K and one for V (s stands for 2^(s - 127)).
 *   data   uint8 [num_pages][kv_heads][2][page_size * head_dim]      0: K, 1: V
 *          K: [token][head_dim]
 *          V: [token / 4][head_dim][token % 4]: an element of four tokens side by side, as the operand
 *             of the attention's second product wants them
 *   scales uint8 [num_pages][kv_heads][page_size / 16][2]            0: K, 1: V
 * The scale that rows need is the smallest power of two, 2^-100 to 2^119, of which no finite element
 * is over 448 times; codes are the nearest, ties to the even code. Elements beyond 448 * 2^119 become
 * that, infinities and NaN become NaN (that element alone). A reader takes scales outside 2^-100 to
 * 2^119 as the nearer of the two.
 *
 * ar_kv8_create: a handle for caches of one geometry, with the conditions and rules of ar_kv4_create. Its
 * workspace is 69 to 102 MB.
 */
typedef struct ar_kv8 ar_kv8;
ar_kv8* ar_kv8_create(int kv_heads, int head_dim, int page_size);
void ar_kv8_destroy(ar_kv8* h);

/*
 * ar_kv8_append: token t's rows k and v to slot slots[t] (page * page_size + offset); a slot outside
 * the cache, as -1, is skipped. The tokens of one block of 16 whose slots keep step with their places in the
 * call (slots[t] - t the same) are a run, skipped tokens between them or not. A run that holds the block's first
 * token starts the block afresh: what the block held is void. Any other run keeps the block's scale, or
 * raises it to what its rows need; the block's other tokens are then rounded to the new scale. So a
 * block's tokens may come one by one or all at once, in the order of their positions. Two runs of one
 * call in one block, as of tokens in another order, leave that block undefined (and nothing else).
 * ar_kv8_read: the rows at `slots` as values of `dtype` in k and v (zeros for a slot outside).
 * dtype is that of k and v. Addresses and strides are multiples of 4 elements.
 */
typedef ar_kv4_rows_args ar_kv8_rows_args;
int ar_kv8_append(ar_kv8* h, const ar_kv8_rows_args* a, void* stream);
int ar_kv8_read(ar_kv8* h, const ar_kv8_rows_args* a, void* stream);

/*
 * ar_kv8_norm_rope_append: what ar_qk_norm_rope gives for q, and ar_kv8_append of the rotated keys,
 * rounded to dtype, and the values, in one launch. kv_heads and head_dim must be the handle's.
 * Padding tokens (negative position) write nothing.
 */
int ar_kv8_norm_rope_append(ar_kv8* h, const ar_qk_norm_rope_args* a, void* stream);

/*
 * ar_kv8_attention: as ar_kv4_attention in every respect, over the 8-bit cache. A NaN element of a
 * value reaches that element of the rows that see it, a NaN element of a key those rows whole.
 */
typedef ar_kv4_attention_args ar_kv8_attention_args;
int ar_kv8_attention(ar_kv8* h, const ar_kv8_attention_args* a, void* stream);

/*
 * Pages that several requests hold. `shares` [num_pages] counts the holders of a page beyond the
 * first: 0 for a page that one request holds, or none. ar_page_tables hands out pages of count 0 and
 * needs no change. The free list is as there: entries [pool[0], min(pool[1], nfree)) of free_pages,
 * taken from the front; pages that come back go in front of it, where the taken ones stood. Lengths
 * and the pool go from one buffer to another, as in ar_page_tables; the outputs must not be the inputs.
 * Requests are numbered by their rows of the table, of which pages_for(kv_len) entries count, at
 * most table_width. Page ids outside [0, num_pages) are held and freed by nobody.
 *
 * ar_pages_fork: for each i, request dst[i], which holds nothing, becomes a copy of src[i]: its row gets
 * src's whole pages, shared from now on, and, where src's last page is partly filled, a page of its
 * own from the free list; copy_src[i] and copy_dst[i] are then that last page and its copy, for
 * ar_pages_copy in every cache, otherwise -1. Written too:
 *   kv_len_out[nreq]   the lengths, of the copies their sources'
 *   pool_out           pool[0] (at least 0) + pages taken, pool[1]
 *   refused[i]         1 for a fork that got nothing: a number outside [0, nreq), src[i] == dst[i], a dst[i]
 *                      whose length is not 0 or that stands earlier in the list, a src of negative length or
 *                      longer than its row, no page left for the last one (later forks that need one
 *                      find none either). 0 otherwise
 * A src that is another fork's dst holds nothing, and so does its copy. shares and table change in
 * place (table only in the rows of dst).
 *
 * ar_pages_free: the requests listed (numbers outside [0, nreq) count as nothing, twice is once) give their
 * pages back: each holder is counted off, and the pages that nobody holds any more are put in front of
 * the free list in ascending order, entries pool_out[0] .. pool[0]-1 where pool_out[0] = pool[0] - pages
 * freed. Should more pages come back than were taken (pool[0] of them), the lowest ids are lost.
 * kv_len_out is 0 for the listed, kv_len for the others; pool_out[1] = pool[1]. Table rows stay as they are.
 *
 * ar_pages_compact: the pages that requests hold move to the ids below their number: with n pages held,
 * the k-th held page at or above n goes to the k-th id below n that nobody holds, in ascending order,
 *   move_src[k], move_dst[k]   for ar_pages_copy in every cache; the rest of the lists is -1
 *   table_out          the table with the new ids, entries past a request's pages -1
 *   shares_out         the counts at the new ids, 0 for pages that nobody holds
 *   free_pages[i] = i  and pool_out = {n, num_pages}: the free list is the pages from n on
 * The table has to hold every page in use: all others are free afterwards. The lists take num_pages / 2
 * entries at least, free_pages num_pages. No copy's source is another's destination.
 *
 * scratch: (num_pages + 31) / 32 + 1 words, zero before the first call that uses them and left so by
 * every call. Calls with one scratch buffer are issued in order on one stream.
 */
typedef struct {
  const int32_t* src; /* [count] */
  const int32_t* dst; /* [count] */
  const int32_t* kv_len; /* [nreq] */
  int32_t* table;        /* [nreq][table_stride] */
  int32_t* shares;       /* [num_pages] */
  const int32_t* pool;   /* [2] */
  const int32_t* free_pages; /* [nfree] */
  int32_t* kv_len_out;   /* [nreq] */
  int32_t* pool_out;     /* [2] */
  int32_t* copy_src;     /* [count] */
  int32_t* copy_dst;     /* [count] */
  int32_t* refused;      /* [count] */
  int64_t table_stride;
  int count; /* 0..4096 */
  int nreq;  /* 0..4096 */
  int table_width;
  int num_pages;
  int nfree;
  int page_size;
} ar_pages_fork_args;
int ar_pages_fork(const ar_pages_fork_args* a, void* stream);

typedef struct {
  const int32_t* requests; /* [count] */
  const int32_t* kv_len;   /* [nreq] */
  const int32_t* table;    /* [nreq][table_stride] */
  int32_t* shares;         /* [num_pages] */
  const int32_t* pool;     /* [2] */
  int32_t* free_pages;     /* [nfree] */
  int32_t* kv_len_out;     /* [nreq] */
  int32_t* pool_out;       /* [2] */
  uint32_t* scratch;       /* [(num_pages + 31) / 32 + 1] */
  int64_t table_stride;
  int count; /* 0..4096 */
  int nreq;  /* 0..4096 */
  int table_width;
  int num_pages; /* 1..2^19 */
  int nfree;
  int page_size;
} ar_pages_free_args;
int ar_pages_free(const ar_pages_free_args* a, void* stream);

typedef struct {
  const int32_t* kv_len; /* [nreq] */
  const int32_t* table;  /* [nreq][table_stride] */
  const int32_t* shares; /* [num_pages] */
  int32_t* table_out;    /* [nreq][out_stride] */
  int32_t* shares_out;   /* [num_pages] */
  int32_t* free_pages;   /* [nfree] */
  int32_t* pool_out;     /* [2] */
  int32_t* move_src;     /* [nmoves] */
  int32_t* move_dst;     /* [nmoves] */
  uint32_t* scratch;     /* [(num_pages + 31) / 32 + 1] */
  int64_t table_stride;
  int64_t out_stride;
  int nreq; /* 0..4096 */
  int table_width;
  int num_pages; /* 1..2^19 */
  int nfree;     /* num_pages at least */
  int nmoves;    /* num_pages / 2 at least */
  int page_size;
} ar_pages_compact_args;
int ar_pages_compact(const ar_pages_compact_args* a, void* stream);

/*
 * ar_pages_copy: page src[i] over page dst[i] of every buffer, buffer b of num_pages pages of
 * page_bytes[b] bytes each. Pairs with an id outside [0, num_pages), as -1, are skipped, and so are those
 * with one id twice. Two pairs with one dst, or a dst that is another pair's src, leave those pages
 * undefined. `buffers` and `page_bytes` are host arrays, read before the call returns. Up to 64
 * buffers are one launch. page_bytes may be any number of bytes; buffers and pages of multiples of 16 are fastest.
 */
typedef struct {
  void* const* buffers;      /* host [nbuffers] */
  const int64_t* page_bytes; /* host [nbuffers] */
  const int32_t* src;        /* [count] */
  const int32_t* dst;        /* [count] */
  int nbuffers;
  int count;
  int num_pages;
} ar_pages_copy_args;
int ar_pages_copy(const ar_pages_copy_args* a, void* stream);

/*
 * ar_prompt_attention: prompts packed one after the other, request b's tokens q_start[b] ..
 * q_start[b+1]-1. Token i of them
 *   out[i] = sum_t softmax_t(scale * q[i] . k[t]) v[t]  over 0 <= t <= i, and with window > 0 also
 * t > i - window, t counted from the request's first token. q has q_heads = kv_heads * group heads,
 * head h reads kv head h / group. lse, types, statistics and special values are as in
 * ar_kv4_attention: probabilities are rounded to bfloat16 for AR_BFLOAT16; AR_FLOAT32 calls multiply in
 * binary32. A NaN or infinity of a masked place does not reach a result; a value's infinity that a row sees may be NaN
 * there if its probability is zero in binary32. Starts are taken between 0 and
 * ntokens; tokens that no request covers keep their rows of out and lse, those of requests that overlap are
 * undefined and the others' are not (but overlaps that make 256 times the tokens, or 2^31 units of a tile's rows and
 * 32 tokens, may leave every row as it was). q, k, v and out are 16-byte aligned, their strides multiples of
 * 16 bytes, those of tokens of k and v 2^23 bytes at most.
 *
 * ar_prompt_create: a handle with the workspace (partial results, 69 to 102 MB), for kv_heads 1..1024 and head_dim 64,
 * 96, 128, 192 or 256. Calls on one handle are issued in order on one stream, on the GPU that was
 * current when it was created.
 */
typedef struct ar_prompt ar_prompt;
ar_prompt* ar_prompt_create(int kv_heads, int head_dim);
void ar_prompt_destroy(ar_prompt* h);

typedef struct {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;             /* [ntokens][q_heads], or NULL */
  const int32_t* q_start; /* [nreq + 1] */
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, o_token, o_head;
  double scale;
  int dtype, ntokens, q_heads, nreq, window;
} ar_prompt_attention_args;
int ar_prompt_attention(ar_prompt* h, const ar_prompt_attention_args* a, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LATENCY_COLLECTIVES_AR_SERVING_H */
