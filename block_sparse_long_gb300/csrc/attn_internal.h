// Host-side declarations of libcosa_attn: launch records shared by the C-ABI layer (attn_api.cu) and the kernel files.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "cosa_attn.h"

namespace cosa_attn {

struct RopeLaunch {
  const uint16_t *kv, *q, *weight;
  const double* inv_freq;
  const int32_t *positions, *cu_seqlens, *start, *page_table;
  uint16_t *q_out, *c_out, *k_out, *cache;
  int32_t* status;
  int64_t kv_stride, q_stride, q_head_stride;
  int num_reqs, num_q_heads, latent_dim, page_shift, total_tokens, max_seqlen, num_pages, max_pages_per_req;
  int interleaved;
  float eps;
};
cudaError_t launch_rope(const RopeLaunch& L, cudaStream_t stream);

struct CommitLaunch {
  uint16_t *cache_a, *cache_b;
  const int32_t *cu_seqlens, *page_table, *kv_len, *path, *path_len;
  int32_t *new_len, *status;
  int num_reqs, row_elems, page_shift, max_seqlen, num_pages, max_pages_per_req, path_pitch;
};
cudaError_t launch_commit(const CommitLaunch& L, cudaStream_t stream);

// Attention over pages: k_cache and v_cache of the tree attention, or the latent vectors in k_cache alone.
struct PagedLaunch {
  const uint16_t *q, *q_rope, *k_cache, *v_cache;
  const int32_t *cu_seqlens, *page_table, *kv_len;
  const int64_t* tree_mask;
  uint16_t* out;
  float* lse;
  void* workspace;
  int32_t* status;
  int64_t q_stride, q_head_stride, q_rope_stride, q_rope_head_stride;
  int num_reqs, num_q_heads, num_kv_heads, head_dim, latent_dim;      // latent_dim 0: the tree attention
  int page_size, page_shift, total_tokens, max_seqlen, num_pages, max_pages_per_req, max_new_tokens;
  float scale_log2;      // sm_scale * log2(e)
  bool stall;            // COSA_ATTN_FLAG_TEST_STALL
};
bool paged_fits(const PagedLaunch& L);      // its tiles are numbered in 31 bits
size_t paged_workspace_bytes(const PagedLaunch& L);
cudaError_t launch_paged(const PagedLaunch& L, cudaStream_t stream);

struct PrefillLaunch {
  const uint16_t *q, *q_rope, *k, *k_rope, *v;
  const int32_t *cu_seqlens, *cu_kv;
  uint16_t* out;
  float* lse;
  int32_t* status;
  int64_t q_stride, q_head_stride, q_rope_stride, q_rope_head_stride, k_stride, k_head_stride, k_rope_stride, v_stride, v_head_stride;
  int num_reqs, num_heads, head_dim, total_tokens, total_kv_tokens;
  float scale_log2;
  bool stall;
};
bool prefill_fits(int total_tokens, int num_reqs, int num_heads);      // its CTAs are numbered in 31 bits
cudaError_t launch_prefill(const PrefillLaunch& L, cudaStream_t stream);

}  // namespace cosa_attn
