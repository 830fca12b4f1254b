/*
 * cosa_attn.h - C ABI of libcosa_attn: dense attention beside the sparse prefill of cosa.h on GB300 (sm_103a), for
 * trees of drafted tokens and for latent attention.
 *
 *   cosa_tree_attention     attention of each request's newest tokens, a tree of drafted ones or plain successors, over
 *                           the bf16 pages that the prefill reads.
 *   cosa_tree_commit        after the check: the accepted path of each tree moved to the slots behind its context.
 *   cosa_latent_rope        latent attention's norm and rotation: one latent vector and one rotated key part per token,
 *                           into pages of latent vectors and into rows; the rotated parts of the queries.
 *   cosa_latent_attention   attention of each request's newest tokens over the pages of latent vectors (absorbed form).
 *   cosa_latent_prefill     causal attention of whole prompts, keys and values expanded per head (expanded form).
 *
 * Latent attention keeps one vector c of latent_dim values and one rotated key part r of 64 values per token for all heads.
 * Head h has the key (c Wk_h, r), the value c Wv_h and the query (u, w), w rotated.  Expanded: the caller forms k = c Wk_h and
 * v = c Wv_h by matrix products and calls cosa_latent_prefill.  Absorbed: u . (c Wk_h) = (u Wk_h^T) . c, so the caller
 * forms u Wk_h^T, calls cosa_latent_attention, which returns sum p c, and multiplies by Wv_h.
 *
 * Conventions (as in cosa_kv.h; status codes of cosa.h)
 *   - Every pointer is DEVICE memory owned by the caller, except `p` (host).  The library allocates
 *     nothing, keeps no pointer after a call returns, and enqueues all work on `stream`.  A call may be
 *     captured into a CUDA graph.  A workspace belongs to one call at a time: two calls, or two graphs,
 *     that can run at the same time need two workspaces.
 *   - Return value: COSA_OK, or a negative status for an error found on the host before anything is
 *     enqueued, or COSA_ERR_CUDA for a failed launch.  Lengths that contradict `p` or each other are found on the
 *     device: *device_status (an int32 the caller zeroes; may be NULL) becomes COSA_ERR_BAD_INPUT.  The
 *     attentions then treat the request concerned as one that has no keys (rows of cu_seqlens ranges that do not fit
 *     total_tokens are not written; a cu_seqlens that falls may leave all rows unwritten), the commit leaves its slots as they are, and cosa_latent_rope leaves out (writes nothing
 *     of) the tokens of no request and those whose slot is negative or, where a cache is written, not below max_seqlen.
 *     A wait inside an attention kernel that runs out after 2 s gives COSA_ERR_DEVICE_TIMEOUT; the kernel ends
 *     once the copies in flight have landed, after 2 s more at the latest, and the outputs are then undefined.  CTAs that
 *     start after that see it in *device_status and do nothing; a status that is not zeroed after it leaves the outputs of
 *     later attentions undefined too.  Without device_status, or where it holds another error already, every wave of
 *     CTAs takes that long.
 *   - Requests are packed by cu_seqlens int32 [num_reqs + 1] (cu_seqlens[0] = 0, non-decreasing, last
 *     entry <= total_tokens); rows behind the last request are neither read nor written.
 *   - A cache slot is a token's place in its request: slot s of request b is row s % P of logical page
 *     s / P of row b of its page table.  A page-table entry outside its cache means the page does not
 *     exist: nothing is written for its slots, and they take part in nothing.  No page may stand in
 *     a table twice where a call writes it.  Slots from kv_len on may hold anything.
 *   - Request b of the attentions over pages has n = cu_seqlens[b+1] - cu_seqlens[b] query tokens, the last n of its
 *     kv_len[b] slots (their keys and values are in the cache).  All of them see the kv_len[b] - n slots of the context.
 *     Without tree_mask token i also sees tokens 0 .. i.  With it, int64 [total_tokens], token i sees token j where bit j
 *     of its mask is set (itself only if bit i is), and n is at most 64; bits from n on are ignored.
 *     A row that sees nothing gives 0, and -inf for its lse.  What a row does not see, infinities and NaN among it, does
 *     not change it.
 *     A batch whose tiles of 128 slots, by max_seqlen, times row tiles pass 31 bits is refused; so is one of the expanded form
 *     whose (total_tokens / 128 + num_reqs) * Hq do.
 *   - lse, float32 [total_tokens, Hq] or NULL: the natural logarithm of the sum of exp(logit) over what the row sees.
 *   - Tensors are bf16 unless noted, 16-byte aligned.  Strides are in elements, multiples of 8, and 0 for dense; heads lie
 *     within a token or tokens within a head, without overlap.
 *       k_cache, v_cache  [num_pages, P, Hkv, d] dense (the pages of cosa.h)
 *       latent_cache      [num_pages, P, latent_dim + 64] dense: c, then r
 *       page tables       int32 [num_reqs, max_pages_per_req]
 *   - Logits, softmax and sums are fp32; exp(logit - reference) is rounded to bf16 as an operand of the second product,
 *     not in the sum that divides it.  The reference is at most 8 binary orders below the row's maximum.  Results do
 *     not depend on the run; another max_new_tokens or batch may round differently.
 */
#ifndef COSA_ATTN_H_
#define COSA_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#include "cosa.h"

#ifdef __cplusplus
extern "C" {
#endif

#define COSA_ATTN_ROPE_DIM 64  /* rotated values of a latent key and of a query head */
#define COSA_ATTN_MAX_TREE 64  /* tokens of a tree */

/* cosa_attn_params.flags */
#define COSA_ATTN_FLAG_INTERLEAVED 1 /* rotation pairs are (2i, 2i+1); default (i, i + 32) */
/* Test hook for the bounded waits of the attentions: no copy is issued, so every wait in the kernel runs out after its
   2 s budget, the kernel ends, *device_status becomes COSA_ERR_DEVICE_TIMEOUT and the outputs are undefined. */
#define COSA_ATTN_FLAG_TEST_STALL 4

/* Every call checks num_reqs, num_q_heads, total_tokens, flags and reserved, the three attentions max_new_tokens too; other fields that
   a call has no use for are ignored by it. */
typedef struct cosa_attn_params {
  int32_t num_reqs;          /* B >= 1                                                          */
  int32_t num_q_heads;       /* Hq >= 1                                                         */
  int32_t num_kv_heads;      /* Hkv >= 1, Hq % Hkv == 0 (tree attention)                        */
  int32_t head_dim;          /* d: 64 or 128 (tree attention; prefill: values of k_nope and v)  */
  int32_t latent_dim;        /* values of a latent vector: 256 or 512                           */
  int32_t page_size;         /* P: 16, 32, 64 or 128                                            */
  int32_t total_tokens;      /* query rows                                                      */
  int32_t total_kv_tokens;   /* prefill: key rows                                               */
  int32_t max_seqlen;        /* >= every context length                                         */
  int32_t num_pages;         /* pages of each cache                                             */
  int32_t max_pages_per_req; /* row pitch of the page table, >= ceil(max_seqlen / P)            */
  int32_t max_new_tokens;    /* attentions over pages: query tokens per request to tile for (any
                                value >= 1 is right; the largest request's is fastest; the
                                expanded form, >= 1 too, does not use it); commit: row pitch of
                                path, at most 64                                                */
  int32_t flags;             /* COSA_ATTN_FLAG_*                                                */
  int32_t reserved;          /* 0                                                               */
  int64_t q_stride;          /* between tokens of q (tree), q_latent, q_nope                    */
  int64_t q_head_stride;     /* between heads of them                                           */
  int64_t q_rope_stride;     /* between tokens of q_rope                                        */
  int64_t q_rope_head_stride;/* between heads of q_rope                                         */
  int64_t k_stride;          /* between tokens of k_nope; of kv (rope)                          */
  int64_t k_head_stride;     /* between heads of k_nope                                         */
  int64_t k_rope_stride;     /* between tokens of k_rope                                        */
  int64_t v_stride;          /* between tokens of v                                             */
  int64_t v_head_stride;     /* between heads of v                                              */
  double sm_scale;           /* logit scale; 2^-100 to 2^60                                     */
  double norm_eps;           /* rope: added to the mean square; 0, or 2^-126 to 2^126           */
} cosa_attn_params;

/* Library version, (major << 16) | minor. */
int cosa_attn_version(void);

/*
 * Attention over the bf16 pages.  Query head h reads kv head h / (Hq / Hkv).
 *   q          [total_tokens, Hq, d], tokens q_stride and heads q_head_stride apart
 *   tree_mask  int64 [total_tokens], or NULL
 *   out        [total_tokens, Hq, d] dense, not q itself
 *   workspace  at least cosa_tree_attention_workspace_size(p) bytes, 256-byte aligned; its content on entry does
 *              not matter.  The size is 0 where the call refuses p.
 */
size_t cosa_tree_attention_workspace_size(const cosa_attn_params* p);
int cosa_tree_attention(const cosa_attn_params* p, const void* q, const int32_t* cu_seqlens, const void* k_cache,
                        const void* v_cache, const int32_t* page_table, const int32_t* kv_len, const int64_t* tree_mask,
                        void* out, float* lse, void* workspace, size_t workspace_bytes, int32_t* device_status, void* stream);

/*
 * Keeps the accepted path of each tree: with n tokens of request b in the last n of its kv_len[b] slots, the rows of
 * tokens path[b, 0] < path[b, 1] < ... (path_len[b] of them, each in 0 .. n - 1) move, in the same pages, to
 * slots kv_len[b] - n, kv_len[b] - n + 1, ...  Other slots are left as they are; a slot whose page does not exist is
 * neither source nor destination.
 *   cache_a, cache_b  [num_pages, P, row_elems] dense; cache_b may be NULL (a latent cache).  row_elems is a multiple
 *                     of 8: Hkv * d, or latent_dim + 64.
 *   cu_seqlens        of the trees' tokens: only its differences are used
 *   path              int32 [num_reqs, max_new_tokens]
 *   path_len          int32 [num_reqs], 0 .. min(n, max_new_tokens)
 *   new_len           out: int32 [num_reqs], kv_len[b] - n + path_len[b], or kv_len[b] for a request that contradicts
 *                     itself; none of the inputs
 */
int cosa_tree_commit(const cosa_attn_params* p, void* cache_a, void* cache_b, int32_t row_elems, const int32_t* cu_seqlens,
                     const int32_t* page_table, const int32_t* kv_len, const int32_t* path, const int32_t* path_len,
                     int32_t* new_len, int32_t* device_status, void* stream);

/*
 * Norm and rotation of latent attention.  Per token, with kv its row (c, r):
 *     c <- c / sqrt(mean(c^2) + norm_eps) * weight         (skipped where weight is NULL)
 *     (r_a, r_b) <- (r_a cos t - r_b sin t, r_b cos t + r_a sin t),   t = position * inv_freq[i]
 * for the 32 pairs (a, b), and the same rotation for the 64 values q of every head.  Angles are formed and reduced in
 * 64 bits, everything else in fp32, and each value is rounded once, to bf16.
 *   kv         [total_tokens, latent_dim + 64], tokens k_stride apart
 *   q          [total_tokens, Hq, 64], tokens q_rope_stride and heads q_rope_head_stride apart, or NULL
 *   weight     bf16 [latent_dim], or NULL
 *   inv_freq   float64 [32]
 *   positions  int32 [total_tokens], or NULL: a token's position is its slot
 *   start      int32 [num_reqs], slot of each request's first token, or NULL for 0
 *   q_out      [total_tokens, Hq, 64] dense; may be q itself where q is dense; given with q
 *   c_out, k_out   [total_tokens, latent_dim] and [total_tokens, 64] dense, or both NULL
 *   latent_cache, page_table   or both NULL: the token at slot s goes to the pages' slot s, below max_seqlen
 * At least one of c_out and latent_cache is given.
 */
int cosa_latent_rope(const cosa_attn_params* p, const void* kv, const void* q, const void* weight, const double* inv_freq,
                     const int32_t* positions, const int32_t* cu_seqlens, const int32_t* start, void* q_out, void* c_out,
                     void* k_out, void* latent_cache, const int32_t* page_table, int32_t* device_status, void* stream);

/*
 * Attention over the pages of latent vectors: logits (q_latent . c + q_rope . r) * sm_scale, output sum p c.
 *   q_latent   [total_tokens, Hq, latent_dim], tokens q_stride and heads q_head_stride apart
 *   q_rope     [total_tokens, Hq, 64], tokens q_rope_stride and heads q_rope_head_stride apart
 *   tree_mask  int64 [total_tokens], or NULL
 *   out        [total_tokens, Hq, latent_dim] dense, neither q_latent nor q_rope itself
 *   workspace  at least cosa_latent_attention_workspace_size(p) bytes, as above
 */
size_t cosa_latent_attention_workspace_size(const cosa_attn_params* p);
int cosa_latent_attention(const cosa_attn_params* p, const void* q_latent, const void* q_rope, const int32_t* cu_seqlens,
                          const void* latent_cache, const int32_t* page_table, const int32_t* kv_len,
                          const int64_t* tree_mask, void* out, float* lse, void* workspace, size_t workspace_bytes,
                          int32_t* device_status, void* stream);

/*
 * Causal attention of packed prompts: logits (q_nope . k_nope + q_rope . k_rope) * sm_scale, output sum p v.  Request b has
 * n query rows and m = cu_kv[b+1] - cu_kv[b] >= n key rows, the last n of them its own: row i sees keys 0 .. m - n + i.
 *   q_nope, k_nope, v   [tokens, Hq, d], tokens and heads apart by their strides
 *   q_rope              [total_tokens, Hq, 64], tokens and heads apart by its strides
 *   k_rope              [total_kv_tokens, 64], tokens k_rope_stride apart: shared by the heads
 *   cu_kv               int32 [num_reqs + 1], or NULL: cu_seqlens (and total_kv_tokens rows)
 *   out                 [total_tokens, Hq, d] dense, none of the inputs
 */
int cosa_latent_prefill(const cosa_attn_params* p, const void* q_nope, const void* q_rope, const void* k_nope,
                        const void* k_rope, const void* v, const int32_t* cu_seqlens, const int32_t* cu_kv, void* out,
                        float* lse, int32_t* device_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* COSA_ATTN_H_ */
