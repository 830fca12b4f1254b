// Attention of each request's newest tokens over pages: the tree attention's keys and values, or latent vectors.
//
// A warp has a query row (token, head) and walks the slots, 32-bit sums in registers, with the running maximum and sum of the
// softmax.
#include <cstdint>

#include "attn_internal.h"
#include "kv_internal.h"
#include "kv_layout.cuh"

namespace cosa_attn {
namespace {

constexpr int kThreads = 128;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float value(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }

template <int DK, int DV, bool kLatent>
__global__ void __launch_bounds__(kThreads) row_kernel(const PagedLaunch L) {
  cosa_kv::wait_for_stream();
  const int lane = threadIdx.x % 32;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / 32;
  const int64_t t = row / L.num_q_heads;
  const int h = static_cast<int>(row % L.num_q_heads);
  if (t >= L.total_tokens) return;
  int b = 0;
  while (b < L.num_reqs && L.cu_seqlens[b + 1] <= t) ++b;
  if (b == L.num_reqs) return;
  const int first = L.cu_seqlens[b], n = L.cu_seqlens[b + 1] - first, i = static_cast<int>(t) - first;
  if (i < 0 || first < 0 || L.cu_seqlens[b + 1] > L.total_tokens) {
    cosa::report_status(L.status, cosa::kStatusBadInput);
    return;
  }
  int len = L.kv_len[b];
  if (len < n || len > L.max_seqlen || (L.tree_mask && n > COSA_ATTN_MAX_TREE)) {
    cosa::report_status(L.status, cosa::kStatusBadInput);
    len = 0;
  }
  const uint64_t mask = L.tree_mask ? static_cast<uint64_t>(L.tree_mask[t]) : 0;
  float q[DK / 32];
#pragma unroll
  for (int e = 0; e < DK / 32; ++e) {
    const int d = e * 32 + lane;
    if (kLatent && d >= DV)
      q[e] = value(L.q_rope + t * L.q_rope_stride + h * (DK - DV) + d - DV);
    else
      q[e] = value(L.q + t * L.q_stride + h * DV + d);
  }
  float o[DV / 32] = {}, m = -INFINITY, l = 0.f;
  const int kvh = h / (L.num_q_heads / L.num_kv_heads);
  for (int s = 0; s < len; ++s) {
    const int j = s - (len - n);
    if (j >= 0 && (L.tree_mask ? !(mask >> j & 1) : j > i)) continue;
    const int phys = L.page_table[static_cast<size_t>(b) * L.max_pages_per_req + (s >> L.page_shift)];
    if (phys < 0 || phys >= L.num_pages) continue;
    const int64_t place = (static_cast<int64_t>(phys) << L.page_shift) + (s & (L.page_size - 1));
    const uint16_t* k = L.k_cache + (kLatent ? place : place * L.num_kv_heads + kvh) * DK;
    const uint16_t* v = kLatent ? k : L.v_cache + (place * L.num_kv_heads + kvh) * DV;
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < DK / 32; ++e) x = fmaf(q[e], value(k + e * 32 + lane), x);
#pragma unroll
    for (int w = 1; w < 32; w *= 2) x += __shfl_xor_sync(kAll, x, w);
    x *= L.scale_log2;
    const float top = fmaxf(m, x), keep = m == top ? 1.f : exp2f(m - top), p = exp2f(x - top);
    m = top;
    l = l * keep + p;
#pragma unroll
    for (int e = 0; e < DV / 32; ++e) o[e] = o[e] * keep + p * value(v + e * 32 + lane);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < DV / 32; ++e)
    L.out[(t * L.num_q_heads + h) * DV + e * 32 + lane] = static_cast<uint16_t>(cosa::pack_bf16x2(o[e] * inv, 0.f));
  if (L.lse && lane == 0) L.lse[t * L.num_q_heads + h] = (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

size_t paged_workspace_bytes(const PagedLaunch&) { return 256; }

cudaError_t launch_paged(const PagedLaunch& L, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(L.total_tokens) * L.num_q_heads;
  const unsigned grid = static_cast<unsigned>((rows * 32 + kThreads - 1) / kThreads);
  auto* kernel = L.latent_dim == 512   ? row_kernel<576, 512, true>
                 : L.latent_dim == 256 ? row_kernel<320, 256, true>
                 : L.head_dim == 128   ? row_kernel<128, 128, false>
                                       : row_kernel<64, 64, false>;
  return cosa_kv::launch_after(kernel, dim3(grid), kThreads, 0, stream, 1, L);
}

}  // namespace cosa_attn
