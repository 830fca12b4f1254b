/*
 * cosa_kv.h - C ABI of libcosa_kv: what stands around the sparse prefill of cosa.h on GB300 (sm_103a).
 *
 * The prefill calls take queries and paged keys and values as attention wants them and write the
 * attention of a whole prompt.  These calls make that input, keep the context in 4 bits afterwards,
 * and decode on it:
 *
 *   cosa_qk_norm_rope    RMS norm of every query and key head and the position rotation in one pass;
 *                        keys and values go into the bf16 pages that the prefill reads, or keys to rows.
 *   cosa_kv4_store       K and V rounded into a paged 4-bit cache, from rows or from bf16 pages.
 *   cosa_kv4_load        the 4-bit cache back into bf16 pages (for the next prefill over the context).
 *   cosa_kv4_attention   attention of the newest tokens of each request over the 4-bit cache, which can
 *                        also add up the attention weight that every cache slot receives.
 *   cosa_kv4_evict       per request and kv head, the slots with the largest accumulated weights (and
 *                        the first and the most recent ones) moved in order into other pages.
 *
 * Conventions (as in cosa.h, whose status codes are used)
 *   - Every pointer is DEVICE memory owned by the caller, except `p` (host).  The library allocates
 *     nothing, keeps no pointer after a call returns, and enqueues all work on `stream`.  A call may be
 *     captured into a CUDA graph.  A workspace belongs to one call at a time: two calls, or two graphs,
 *     that can run at the same time need two workspaces.
 *   - Return value: COSA_OK, or a negative status for an error found on the host before anything is
 *     enqueued, or COSA_ERR_CUDA for a failed launch.  Lengths that contradict `p` are found on the
 *     device: *device_status (an int32 the caller zeroes; may be NULL) becomes COSA_ERR_BAD_INPUT.  The
 *     attention, the eviction and the calls from pages to pages then treat the request concerned as empty;
 *     cosa_qk_norm_rope and cosa_kv4_store from rows leave out (write nothing of) the tokens of no request
 *     and those whose slot is negative or, where a cache is written, not below max_seqlen; the other tokens of
 *     the request are written.  A wait inside the attention kernel that runs out after 2 s gives
 *     COSA_ERR_DEVICE_TIMEOUT; the kernel ends once the copies in flight have landed, after 2 s more at the
 *     latest, and the outputs are then undefined.
 *   - Requests are packed by cu_seqlens int32 [num_reqs + 1] (cu_seqlens[0] = 0, non-decreasing, last
 *     entry <= total_tokens); rows behind the last request are neither read nor written.
 *   - A cache slot is a token's place in its request: slot s of request b is row s % P of logical page
 *     s / P of row b of its page table.  A page-table entry outside its cache means the page does not
 *     exist: nothing is written for its slots, and they take part in nothing.  No page may stand in
 *     a table twice where a call writes it.
 *   - Tensors (bf16 unless noted; d = head_dim, P = page_size):
 *       q            [total_tokens, Hq, d], tokens q_stride elements apart (0: dense)
 *       k, v         [total_tokens, Hkv, d], tokens k_stride / v_stride elements apart (0: dense)
 *       k_cache, v_cache  [num_pages, P, Hkv, d] dense (the pages of cosa.h)
 *       kv4_cache    uint8 [num_kv4_pages, Hkv, P * 9d/8] dense
 *       page tables  int32 [num_reqs, max_pages_per_req]
 *     q, k, v and the caches are 16-byte aligned, strides are multiples of 8 elements.
 *
 * The 4-bit cache.  32 neighbouring values of a head share a scale s, the bf16 nearest to max|x| / 7;
 * a value x is held as c = clamp(rint(x / s), -7, 7) (ties to even; c = 0 if s = 0) and stands for c * s.
 * A group with a value that is not finite gets a NaN scale: all of it stands for NaN.  With bf16 input
 * both roundings are exact decisions (the quotients of 8-bit significands cannot come nearer to a
 * border than fp32 resolves without lying on it).  A page of one kv head is P/16 tiles of 16 tokens,
 * each 18 d bytes:
 *       K codes   [16][d/2]    token t is row t;  the 32-bit word w = c * (d/32) + g (0 <= c < 4) holds
 *                              values 32 g + 8 c .. + 7, one to a nibble, lowest first
 *       V codes   [16][d/2]    token t is row (t % 2) * 8 + t / 2;  the 16-bit word w = i * (d/32) + g
 *                              (0 <= i < 8) holds values 32 g + 4 i .. + 3, one to a nibble, lowest first
 *       K scales  bf16 [16][d/32]
 *       V scales  bf16 [16][d/32]
 * Of the four nibbles of each 16 bits, nibble n holds |c| of its value in the three low bits and, in the high
 * bit, the sign of the value of nibble n ^ 2.  Signs and word orders are laid out for the attention's matrix
 * instructions: a lane's codes are one load, and two codes become two bf16 operands by a shift and a mask.
 */
#ifndef COSA_KV_H_
#define COSA_KV_H_

#include <stddef.h>
#include <stdint.h>

#include "cosa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* cosa_kv_params.flags.  Flags and fields that a call has no use for are ignored by it: one set of parameters serves all. */
#define COSA_KV_FLAG_INTERLEAVED 1 /* rotation pairs are (2i, 2i+1); default (i, i + rotary_dim/2) */
/* Test hook for the bounded waits of cosa_kv4_attention: no copy of the cache is issued, so every wait in the kernel runs
   out after its 2 s budget, the kernel ends, *device_status becomes COSA_ERR_DEVICE_TIMEOUT and out is undefined. */
#define COSA_KV_FLAG_TEST_STALL 4

typedef struct cosa_kv_params {
  int32_t num_reqs;          /* B >= 1                                                          */
  int32_t num_q_heads;       /* Hq >= 1                                                         */
  int32_t num_kv_heads;      /* Hkv >= 1, Hq % Hkv == 0                                         */
  int32_t head_dim;          /* d: 64 or 128                                                    */
  int32_t page_size;         /* P: 16, 32, 64 or 128                                            */
  int32_t total_tokens;      /* rows of q / k / v                                               */
  int32_t max_seqlen;        /* >= every context length; row pitch of the weights               */
  int32_t num_pages;         /* pages of the bf16 caches                                        */
  int32_t num_kv4_pages;     /* pages of the 4-bit cache                                        */
  int32_t max_pages_per_req; /* row pitch of the page tables, >= ceil(max_seqlen / P)           */
  int32_t rotary_dim;        /* rotated values per head: a multiple of 16, <= d                 */
  int32_t max_new_tokens;    /* attention: query tokens per request to tile for (any value >= 1
                                is right; the largest request's is fastest)                     */
  int32_t budget;            /* evict: slots kept per request and kv head                       */
  int32_t sink;              /* evict: first slots always kept                                  */
  int32_t recent;            /* evict: last slots always kept, sink + recent <= budget          */
  int32_t max_dst_pages;     /* evict: row pitch of dst_page_table, >= ceil(budget / P)         */
  int32_t flags;             /* COSA_KV_FLAG_*                                                  */
  int32_t reserved;          /* 0                                                               */
  int64_t q_stride;          /* elements between tokens of q, k, v; 0 for dense rows            */
  int64_t k_stride;
  int64_t v_stride;
  double sm_scale;           /* attention: logit scale, normally 1/sqrt(d); 2^-100 to 2^60      */
  double norm_eps;           /* norm: added to the mean square; 0, or 2^-126 to 2^126           */
} cosa_kv_params;

/* Library version, (major << 16) | minor. */
int cosa_kv_version(void);

/*
 * Norm and rotation of q and k, and the cache write of the prefill.  Per token and head
 *     y = x / sqrt(mean(x^2) + norm_eps) * weight          (skipped where the weight is NULL)
 *     (y_a, y_b) <- (y_a cos t - y_b sin t, y_b cos t + y_a sin t),   t = position * inv_freq[i]
 * for the rotary_dim / 2 pairs (a, b) of the head; the other values stay.  Angles are formed and
 * reduced in 64 bits, everything else in fp32, and each value is rounded once, to bf16.
 *
 *   q_weight, k_weight   bf16 [d], 16-byte aligned, or NULL for no norm of that side
 *   inv_freq   float64 [rotary_dim / 2]
 *   positions  int32 [total_tokens], or NULL: a token's position is its slot
 *   start      int32 [num_reqs], slot of each request's first token, or NULL for 0
 *   q_out      bf16 [total_tokens, Hq, d] dense; may be q itself where q is dense
 *   k_out      bf16 [total_tokens, Hkv, d] dense, or NULL; may be k itself where k is dense
 *   k_cache, v_cache, page_table   or all NULL: k and v of the token at slot s go to the pages' slot s.
 * At least one of k_out and k_cache is given; v is read only for the caches.
 * Slots of the caches are below max_seqlen.
 */
int cosa_qk_norm_rope(const cosa_kv_params* p, const void* q, const void* k, const void* v, const void* q_weight,
                      const void* k_weight, const double* inv_freq, const int32_t* positions,
                      const int32_t* cu_seqlens, const int32_t* start, void* q_out, void* k_out, void* k_cache,
                      void* v_cache, const int32_t* page_table, int32_t* device_status, void* stream);

/*
 * Rounds K and V into the 4-bit cache, either
 *   rows    (src_page_table NULL)  k, v [total_tokens, Hkv, d] packed by cu_seqlens; token i of request b goes
 *           to slot start[b] + i (start NULL: 0); kv_len is not read;
 *   pages   (src_page_table given)  k, v are k_cache, v_cache [num_pages, P, Hkv, d]; slots start[b] ..
 *           kv_len[b] - 1 are copied to the same slots; cu_seqlens is not read.  A slot whose source page
 *           does not exist is left as it is.
 * Other slots of the cache, of the same pages too, are left as they are.
 */
int cosa_kv4_store(const cosa_kv_params* p, const void* k, const void* v, const int32_t* cu_seqlens,
                   const int32_t* src_page_table, const int32_t* start, const int32_t* kv_len, void* kv4_cache,
                   const int32_t* page_table, int32_t* device_status, void* stream);

/*
 * Writes slots start[b] .. kv_len[b] - 1 (start NULL: from 0) of the 4-bit cache to the same slots of
 * the bf16 caches through dst_page_table (values c * s, rounded to bf16).
 */
int cosa_kv4_load(const cosa_kv_params* p, const void* kv4_cache, const int32_t* page_table, const int32_t* start,
                  const int32_t* kv_len, void* k_cache, void* v_cache, const int32_t* dst_page_table,
                  int32_t* device_status, void* stream);

/*
 * Attention over the 4-bit cache.  Request b has n = cu_seqlens[b+1] - cu_seqlens[b] query tokens, the
 * last n of its kv_len[b] cache slots: token i attends to slots 0 .. kv_len[b] - n + i that exist.
 * A row that sees nothing gives 0.  Query head h reads kv head h / (Hq / Hkv).
 *   q, out    bf16 [total_tokens, Hq, d], both dense; out is not q itself
 *   weights   float32 [num_reqs, Hkv, max_seqlen], or NULL: weights[b, j, s] += the sum, over the request's
 *             query tokens and the heads of kv head j, of the softmax weight of slot s (s < kv_len[b]).
 *   workspace at least cosa_kv4_attention_workspace_size(p, weights != NULL) bytes, 256-byte aligned;
 *             its content on entry does not matter.  The size is 0 where the call refuses p.
 * Logits, softmax and sums are fp32; q and the codes enter the products exactly, and p * s is rounded
 * to bf16 for the second one.  |q| and the scales are below 2^31 (beyond, the result is not finite), and values
 * smaller than 2^-90 lose precision.  Results do not depend on the run; another max_seqlen, max_new_tokens or batch may
 * round differently.
 */
size_t cosa_kv4_attention_workspace_size(const cosa_kv_params* p, int with_weights);
int cosa_kv4_attention(const cosa_kv_params* p, const void* q, const int32_t* cu_seqlens, const void* kv4_cache,
                       const int32_t* page_table, const int32_t* kv_len, void* out, float* weights,
                       void* workspace, size_t workspace_bytes, int32_t* device_status, void* stream);

/*
 * Keeps min(budget, existing slots) slots of every (request, kv head): the existing ones among the first
 * `sink` and the last `recent` slots, then those with the largest weights (ties and equal zeros: the
 * lowest slot; NaN counts as the smallest).  The kept slots, in ascending order, become slots 0, 1, ...
 * of dst_page_table in the same cache.  The source pages are not changed, and no destination page may
 * be a source page of the call.
 *   weights      float32 [num_reqs, Hkv, max_seqlen]
 *   new_len      out: int32 [num_reqs], slots kept (equal for all kv heads of a request); not `kv_len` itself
 *   kept         out: int32 [num_reqs, Hkv, budget], the old slot of every new one, then -1
 *   weights_out  out, or NULL: float32 [num_reqs, Hkv, max_seqlen], the kept slots' weights, then 0;
 *                not `weights` itself
 */
int cosa_kv4_evict(const cosa_kv_params* p, void* kv4_cache, const int32_t* page_table, const int32_t* kv_len,
                   const float* weights, const int32_t* dst_page_table, int32_t* new_len, int32_t* kept,
                   float* weights_out, int32_t* device_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* COSA_KV_H_ */
