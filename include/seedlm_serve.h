/*
 * seedlm_serve.h -- what a serving step needs around the packed projections of
 * seedlm.h: page tables and slots of a paged key-value cache, rotary positions
 * with the cache write, attention of new tokens over the cache, and low-rank
 * adapters of many requests beside a shared projection.
 *
 * Conventions are those of seedlm.h: status codes, dtype codes, streams passed
 * as void*, device pointers of the current device, asynchronous launches, no
 * C++ exception across the boundary.  Argument structs are host memory that is
 * read during the call only.  No call synchronises or copies to the host, so
 * each can be captured into a HIP graph; a call that uses scratch follows the
 * scratch rules of seedlm_gemv (per device and stream, allocated by the first
 * call that needs it, freed by seedlm_scratch_release; a replay of a captured
 * graph must not overlap a call on the stream that it was captured on, nor a
 * replay of another graph captured there).
 *
 * The paged cache.  Keys and values live in two fp16 pools of `pages` pages of
 * `page_size` tokens.  Element (page, token, head, d) of either pool sits at
 *   page * page_stride + token * token_stride + head * head_stride + d
 * elements from its base, the strides being the same for both pools; any order
 * of heads and tokens within a page fits.  A request's token at position p is
 * token p % page_size of page table[request][p / page_size]; its slot is
 * page * page_size + p % page_size.  A page number outside [0, pages) holds no
 * tokens: nothing is read or written through it.
 */
#ifndef SEEDLM_SERVE_H
#define SEEDLM_SERVE_H

#include "seedlm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most requests of one seedlm_cache_plan call and queries of a seedlm_cache_attend. */
#define SEEDLM_MAX_REQUESTS 4096
/* Largest adapter rank. */
#define SEEDLM_MAX_RANK 256

/*
 * seedlm_cache_plan -- one serving step's bookkeeping, from request lengths:
 * pages for the new tokens, pages of finished requests back to the pool, and
 * the row, position and slot of every new token.
 *
 *   requests    n, in [1, SEEDLM_MAX_REQUESTS]
 *   page_size   tokens of a page, >= 1
 *   max_pages   columns of table (a request holds at most max_pages pages)
 *   pool        entries of ring: the number of pages of the cache
 *   tokens      T, entries of rows, positions and slots (0: they may be NULL)
 *   lens        int32 [n]: tokens each request has in the cache
 *   fresh       int32 [n]: new tokens of each request; negative: the request
 *               is finished and gives its pages back
 *   table       int32 [n][max_pages], row stride table_stride; in and out
 *   ring        int32 [pool]: free pages, a queue; in and out
 *   ring_state  int32 [2]: index of the queue's first entry, entries in it
 *   lens_out    int32 [n]; may be lens
 *   ring_state_out int32 [2]; may be ring_state
 *   offsets     int32 [n+1]: where each request's new tokens start among all
 *               new tokens, which lie request after request (sums stop at
 *               2^31 - 1)
 *   rows, positions, slots  int32 [T]: request, position and slot of each new
 *               token; past the last one -1, 0, -1
 *   spans       int32 [T] or NULL: the tokens that each new token attends to,
 *               position + 1, itself among them; 0 where its slot is -1
 *   ok          int32 [n]: 1 or 0
 * A request's step is granted (ok = 1) if its tokens fit its table row, they and
 * those of all requests before it fit the T entries, and the queue holds its new
 * pages after those that requests before it asked for: its new pages come from the queue's front into its table row and
 * its length grows.  Otherwise (ok = 0) it gets no pages, its length stays and
 * its tokens' slots are -1.  A finished request has ok = 1 and length 0; its
 * pages join the queue's end (for later calls) and its table row keeps its
 * contents.  Lengths are taken into [0, max_pages * page_size].  Other
 * overlaps among the arrays than the two named are not allowed.
 * One launch (two when lens_out or ring_state_out is the input and the call
 * needs several workgroups: then 4 (n + 2) bytes of stream scratch are used).
 * Errors: SEEDLM_E_INVALID (null, range, overlap of lens and lens_out),
 * SEEDLM_E_UNSUPPORTED (max_pages * page_size + tokens or pool * page_size of
 * 2^31 or more, tokens or pool above 2^30), SEEDLM_E_NOMEM, SEEDLM_E_DEVICE.
 */
typedef struct seedlm_cache_plan_args {
  const int32_t* lens;
  const int32_t* fresh;
  int32_t* table;
  int32_t* ring;
  const int32_t* ring_state;
  int32_t* lens_out;
  int32_t* ring_state_out;
  int32_t* offsets;
  int32_t* rows;
  int32_t* positions;
  int32_t* slots;
  int32_t* ok;
  int32_t* spans;
  int64_t table_stride;
  int32_t requests, page_size, max_pages, pool, tokens;
} seedlm_cache_plan_args;
SEEDLM_API int seedlm_cache_plan(const seedlm_cache_plan_args* args, void* stream);

/* The two pools of a paged cache (fp16 device memory). */
typedef struct seedlm_cache_t {
  void* k;
  void* v;
  int64_t pages;
  int64_t page_stride, token_stride, head_stride; /* elements */
  int32_t page_size, kv_heads, head_dim;
} seedlm_cache_t;

/*
 * seedlm_cache_append -- rotate q and k by their positions, write q_out, and
 * write k and v into their cache slots.
 *   q      [tokens][heads][head_dim], row stride q_stride elements
 *   k, v   [tokens][kv_heads][head_dim], row strides k_stride, v_stride
 *   q_out  as q, row stride q_out_stride; may be q
 *          all four of x_dtype (SEEDLM_F32 or SEEDLM_F16); heads of a row are
 *          head_dim apart
 *   cos, sin  fp32 [table_len][rot / 2], contiguous: position p turns pair i
 *          by the angle whose cosine and sine are cos[p][i], sin[p][i]:
 *          (a, b) -> (a cos - b sin, b cos + a sin), in fp32, rounded once
 *   rot    rotated elements of a head, even, in [0, head_dim]; pair i is
 *          elements (i, i + rot/2), or (2i, 2i + 1) when interleaved; the
 *          other elements are copied
 *   positions, slots  int32 [tokens]
 * A token whose slot lies outside [0, pages * page_size) is a padding row:
 * nothing is written to the cache for it.  A token whose position lies outside
 * [0, table_len) is one too, and its q_out row is zero.  Two tokens of one call
 * must not share a slot.  fp32 k and v are rounded to fp16 (nearest even).
 * One launch, no scratch.  tokens = 0 is a no-op.
 * Errors: SEEDLM_E_INVALID (null, range, a stride smaller than what it spans),
 * SEEDLM_E_UNSUPPORTED (dtype, odd rot or head_dim, head_dim above 512,
 * more than 16384 heads, tokens of 2^24 or more, pages * page_size of 2^31 or
 * more), SEEDLM_E_DEVICE.
 */
typedef struct seedlm_cache_append_args {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  const float* cos;
  const float* sin;
  const int32_t* positions;
  const int32_t* slots;
  seedlm_cache_t cache;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  int32_t tokens, heads, rot, table_len, interleaved, x_dtype;
} seedlm_cache_append_args;
SEEDLM_API int seedlm_cache_append(const seedlm_cache_append_args* args, void* stream);

/*
 * seedlm_cache_attend -- attention of query tokens over their requests' pages of
 * the cache, one token per request or several: out = sum_t softmax_t(scale *
 * q . k_t) v_t for every head, head h reading cache head h / (heads / kv_heads).
 *   q      [queries][heads][head_dim], row stride q_stride elements
 *   out    as q, row stride out_stride; may be q
 *          both of x_dtype (SEEDLM_F32 or SEEDLM_F16)
 *   table  int32 [table_rows][max_pages], row stride table_stride
 *   rows   int32 [queries]: each query's row of table, or NULL: its own number
 *          (then table_rows >= queries).  A row outside [0, table_rows) has no
 *          tokens
 *   lens   int32 [queries]: tokens each query attends to, its own among them;
 *          taken into [0, min(max_len, max_pages * page_size)].  With one token
 *          per request that is the requests' lengths after seedlm_cache_plan, with
 *          rows of a plan its spans (several tokens of a request then see one
 *          another as their positions allow)
 *   max_len  bound on lens that the host knows (the work is split by the
 *          lengths themselves, which only the GPU reads)
 *   scale  finite
 * head_dim 64, 128 or 256; heads a multiple of kv_heads, at most 16384; queries
 * at least 1 and at most SEEDLM_MAX_REQUESTS.  A query of no tokens (length 0, no row, or no
 * valid page) gets zeros.  What lies in the cache beyond a query's length, NaN
 * and infinities included, does not reach its output.  An infinity among the
 * values that it does attend to makes the output elements that it enters infinite
 * or NaN.  With fp32 queries one among the keys may make a head's output NaN where
 * the formula gives the token a weight of 0.  Products of fp16 keys are exact;
 * scores, softmax statistics and sums are fp32, and the softmax weights enter
 * the matrix cores as the sum of two fp16 numbers (22 bits), as do fp32 queries.
 * The cache's base addresses are 16-byte aligned and its strides multiples of
 * 8 elements; a pool spans less than 2^35 elements.  fp16 q is 16-byte aligned with
 * a q_stride that is a multiple of 8; fp32 q likewise, of 4.
 * Scratch: seedlm_cache_attend_scratch_bytes, on the stream.
 * Results are the same for the same arguments; the split, and with it the
 * order of sums, depends on all lengths of the call.
 * Errors: SEEDLM_E_INVALID (null, range), SEEDLM_E_UNSUPPORTED (dtype,
 * head_dim, alignment, size), SEEDLM_E_NOMEM, SEEDLM_E_DEVICE.
 */
typedef struct seedlm_cache_attend_args {
  const void* q;
  void* out;
  const int32_t* table;
  const int32_t* rows;
  const int32_t* lens;
  seedlm_cache_t cache;
  int64_t q_stride, out_stride, table_stride;
  int32_t queries, table_rows, heads, max_pages, max_len, x_dtype;
  float scale;
} seedlm_cache_attend_args;
SEEDLM_API int seedlm_cache_attend(const seedlm_cache_attend_args* args, void* stream);

/* seedlm_cache_attend_scratch_bytes -- stream scratch that seedlm_cache_attend
 * uses for these arguments on the current device.  Errors as there. */
SEEDLM_API int seedlm_cache_attend_scratch_bytes(const seedlm_cache_attend_args* args,
                                                 size_t* bytes);

/*
 * seedlm_lora_many -- low-rank adapters of many requests beside shared
 * projections: for every site i and activation row t with adapter a = adapter[t],
 *   y_i[t] = base_i[t] + scales[a] * B_i[a] (A_i[a] x_i[t]).
 * base_i is what the shared projection gave (seedlm_gemv_many, seedlm_gemm).
 *   x      device [tokens][cols] of x_dtype, contiguous
 *   A      device fp16 [adapters][rank][cols], contiguous
 *   B      device fp16 [adapters][rows][rank], contiguous
 *   base   device [tokens][rows] of y_dtype, contiguous
 *   y      as base; may be base (only rows with an adapter are then written);
 *          otherwise no y overlaps another array of the call
 *   adapter  device int32 [tokens], in any order; a value outside
 *          [0, adapters) means none: y_i[t] = base_i[t]
 *   scales device fp32 [adapters]
 * rank in [1, SEEDLM_MAX_RANK] per site; n sites, up to 8 consecutive ones
 * sharing their launches: one for few rows with a small A, two, or three for
 * many rows.  x_dtype and y_dtype are SEEDLM_F32 or SEEDLM_F16.
 * A row's result depends on its own adapter alone: NaN or infinities in other
 * adapters do not reach it.  Infinities in its own give the infinity or NaN that
 * the formula does, whatever the number of rows.  A x is held in fp32; the sum is
 * rounded once.  Calls with fp16 x and y, many rows and ranks and sizes that are
 * multiples of 8 run on the matrix cores, A x entering the second product as the
 * sum of two fp16 numbers (22 bits).
 * Scratch: seedlm_lora_scratch_bytes, on the stream.  tokens = 0 and n = 0 are
 * no-ops.
 * Errors: SEEDLM_E_INVALID (null, range, a pointer not aligned to its type),
 * SEEDLM_E_UNSUPPORTED (dtype; rows or cols of 2^24, tokens of 2^20 or more),
 * SEEDLM_E_NOMEM, SEEDLM_E_DEVICE.
 */
typedef struct seedlm_lora_site {
  const void* x;
  const void* A;
  const void* B;
  const void* base;
  void* y;
  int64_t rows, cols;
  int32_t rank;
} seedlm_lora_site;
SEEDLM_API int seedlm_lora_many(const seedlm_lora_site* sites, int n, const int32_t* adapter,
                                const float* scales, int64_t tokens, int adapters, int x_dtype,
                                int y_dtype, void* stream);

/* seedlm_lora_scratch_bytes -- stream scratch that seedlm_lora_many uses for
 * these sites (only their sizes and alignment count).  Errors as there. */
SEEDLM_API int seedlm_lora_scratch_bytes(const seedlm_lora_site* sites, int n, int64_t tokens,
                                         int adapters, int x_dtype, int y_dtype, size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* SEEDLM_SERVE_H */
