// Host-side declarations of libcosa_kv: launch records shared by the C-ABI layer (kv_api.cu) and the
// kernel files.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "cosa_kv.h"

namespace cosa_kv {

// Launch of a kernel that begins with wait_for_stream() (kv_layout.cuh), in clusters of `cluster` CTAs where it is not 1.
template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream, int cluster,
                         const Args&... args) {
  cudaLaunchAttribute attrs[2]{};
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(static_cast<unsigned>(threads));
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  c.attrs = attrs;
  c.numAttrs = cluster == 1 ? 1 : 2;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

struct RopeLaunch {
  const uint16_t *q, *k, *v, *q_weight, *k_weight;
  const double* inv_freq;
  const int32_t *positions, *cu_seqlens, *start, *page_table;
  uint16_t *q_out, *k_out, *k_cache, *v_cache;
  int32_t* status;
  int64_t q_stride, k_stride, v_stride;
  int num_reqs, num_q_heads, num_kv_heads, head_dim, page_size, total_tokens, max_seqlen, num_pages, max_pages_per_req;
  int rotary_dim, interleaved;
  int page_shift;        // log2(page_size)
  float eps;
};
cudaError_t launch_rope(const RopeLaunch& L, cudaStream_t stream);

struct ConvertLaunch {
  // store: k, v are the source (rows or pages); load: k_cache, v_cache the destination
  const uint16_t *k, *v;
  uint16_t *k_cache, *v_cache;
  uint8_t* cache;
  const int32_t *page_table, *other_table, *cu_seqlens, *start, *kv_len;
  int32_t* status;
  int64_t k_stride, v_stride;
  int num_reqs, num_kv_heads, head_dim, page_size, total_tokens, max_seqlen, num_pages, num_kv4_pages, max_pages_per_req;
  int page_shift;        // log2(page_size)
};
cudaError_t launch_store_rows(const ConvertLaunch& L, cudaStream_t stream);
cudaError_t launch_store_pages(const ConvertLaunch& L, cudaStream_t stream);
cudaError_t launch_load(const ConvertLaunch& L, cudaStream_t stream);

struct AttnLaunch {
  const uint16_t* q;
  const int32_t *cu_seqlens, *page_table, *kv_len;
  const uint8_t* cache;
  uint16_t* out;
  float* weights;
  void* workspace;
  int32_t* status;
  int num_reqs, num_q_heads, num_kv_heads, head_dim, page_size, total_tokens, max_seqlen, num_kv4_pages, max_pages_per_req;
  int max_new_tokens;
  float scale_log2;      // sm_scale * log2(e)
  bool stall;            // COSA_KV_FLAG_TEST_STALL
};
size_t attn_workspace_bytes(int num_q_heads, int head_dim, int total_tokens, int max_seqlen, bool with_weights);
cudaError_t launch_attention(const AttnLaunch& L, cudaStream_t stream);

struct EvictLaunch {
  uint8_t* cache;
  const int32_t *page_table, *kv_len, *dst_page_table;
  const float* weights;
  int32_t *new_len, *kept;
  float* weights_out;
  int32_t* status;
  int num_reqs, num_kv_heads, head_dim, page_size, max_seqlen, num_kv4_pages, max_pages_per_req, max_dst_pages;
  int budget, sink, recent;
  int page_shift;        // log2(page_size)
};
cudaError_t launch_evict(const EvictLaunch& L, cudaStream_t stream);

}  // namespace cosa_kv
