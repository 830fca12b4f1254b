// Causal attention of packed prompts in the expanded form of latent attention.
//
// A warp has a query row (token, head) and walks its keys, 32-bit sums in registers, with the running maximum and sum of the
// softmax.
#include <cstdint>

#include "attn_internal.h"
#include "kv_internal.h"
#include "kv_layout.cuh"

namespace cosa_attn {
namespace {

constexpr int kThreads = 128;
constexpr int kRot = COSA_ATTN_ROPE_DIM;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float value(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }

template <int D>
__global__ void __launch_bounds__(kThreads) row_kernel(const PrefillLaunch L) {
  cosa_kv::wait_for_stream();
  const int lane = threadIdx.x % 32;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / 32;
  const int64_t t = row / L.num_heads;
  const int h = static_cast<int>(row % L.num_heads);
  if (t >= L.total_tokens) return;
  int b = 0;
  while (b < L.num_reqs && L.cu_seqlens[b + 1] <= t) ++b;
  if (b == L.num_reqs) return;
  const int32_t* cu_kv = L.cu_kv ? L.cu_kv : L.cu_seqlens;
  const int first = L.cu_seqlens[b], n = L.cu_seqlens[b + 1] - first, i = static_cast<int>(t) - first;
  if (i < 0 || first < 0 || L.cu_seqlens[b + 1] > L.total_tokens) {
    cosa::report_status(L.status, cosa::kStatusBadInput);
    return;
  }
  const int64_t from = cu_kv[b];
  int64_t len = cu_kv[b + 1] - from;
  if (from < 0 || len < n || from + len > L.total_kv_tokens) {
    cosa::report_status(L.status, cosa::kStatusBadInput);
    len = 0;
  }
  float q[D / 32], qr[kRot / 32], o[D / 32] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) q[e] = value(L.q + t * L.q_stride + h * L.q_head_stride + e * 32 + lane);
#pragma unroll
  for (int e = 0; e < kRot / 32; ++e) qr[e] = value(L.q_rope + t * L.q_rope_stride + h * L.q_rope_head_stride + e * 32 + lane);
  for (int64_t s = from; s < from + len - n + i + 1 && len; ++s) {
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) x = fmaf(q[e], value(L.k + s * L.k_stride + h * L.k_head_stride + e * 32 + lane), x);
#pragma unroll
    for (int e = 0; e < kRot / 32; ++e) x = fmaf(qr[e], value(L.k_rope + s * L.k_rope_stride + e * 32 + lane), x);
#pragma unroll
    for (int w = 1; w < 32; w *= 2) x += __shfl_xor_sync(kAll, x, w);
    x *= L.scale_log2;
    const float top = fmaxf(m, x), keep = m == top ? 1.f : exp2f(m - top), p = exp2f(x - top);
    m = top;
    l = l * keep + p;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] = o[e] * keep + p * value(L.v + s * L.v_stride + h * L.v_head_stride + e * 32 + lane);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) L.out[(t * L.num_heads + h) * D + e * 32 + lane] = static_cast<uint16_t>(cosa::pack_bf16x2(o[e] * inv, 0.f));
  if (L.lse && lane == 0) L.lse[t * L.num_heads + h] = (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

cudaError_t launch_prefill(const PrefillLaunch& L, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(L.total_tokens) * L.num_heads;
  const unsigned grid = static_cast<unsigned>((rows * 32 + kThreads - 1) / kThreads);
  return cosa_kv::launch_after(L.head_dim == 128 ? row_kernel<128> : row_kernel<64>, dim3(grid), kThreads, 0, stream, 1, L);
}

}  // namespace cosa_attn
