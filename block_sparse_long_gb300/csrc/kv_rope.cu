// RMS norm of each query and key head, position rotation, and the bf16 cache write, in one pass.
//
// Per head x of d values:  y = x * rsqrt(mean(x^2) + eps) * w, then for each of the rotary_dim / 2
// pairs (a, b):  (y_a cos t - y_b sin t, y_b cos t + y_a sin t) with t = position * inv_freq[i].
// A value is read once and written once (4 bytes per value), for about ten operations: memory bound.
#include <cstdint>

#include "cosa_kv.h"
#include "kv_internal.h"
#include "kv_layout.cuh"

namespace cosa_kv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;   // tokens of a CTA

// A row (token, head) is D / 16 lanes of 16 values in two chunks of eight.  Lane l's chunks are chosen so
// that both halves of every rotation pair are in one lane: chunks l and l + rotary_dim / 16 of the
// rotated part, then what is left of the head two by two.  (Interleaved pairs are neighbours: any choice.)
template <int D>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeLaunch L, const int tokens_per_cta) {
  constexpr int kLanes = D / 16;
  constexpr int kRowsPerPass = kThreads / kLanes;
  __shared__ float2 s_rot[kMaxTokens][D / 2];   // cos, sin
  __shared__ int s_slot[kMaxTokens];            // cache slot, -1: the token is left out
  __shared__ int s_phys[kMaxTokens];            // physical page of the slot, -1: none
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * tokens_per_cta;
  const int last = L.cu_seqlens[L.num_reqs];
  if (blockIdx.x == 0 && tid == 0 && (L.cu_seqlens[0] != 0 || last > L.total_tokens))
    cosa::report_status(L.status, cosa::kStatusBadInput);
  const int ntok = min(tokens_per_cta, min(last, L.total_tokens) - t0);
  if (ntok <= 0) return;

  // a warp per token: its request is the number of requests that end at or before it
  if (tid / 32 < ntok) {
    const int t = t0 + tid / 32, lane = tid % 32;
    int b = 0;
    for (int i = lane; i < L.num_reqs; i += 32) b += L.cu_seqlens[i + 1] <= t;
    b = __reduce_add_sync(0xffffffffu, b);
    if (lane == 0) {
      const int off = b < L.num_reqs ? t - L.cu_seqlens[b] : -1;
      const int64_t slot = off < 0 ? -1 : static_cast<int64_t>(off) + (L.start ? L.start[b] : 0);
      const bool fits = slot >= 0 && (!L.k_cache || slot < L.max_seqlen);
      if (!fits) cosa::report_status(L.status, cosa::kStatusBadInput);
      s_slot[tid / 32] = fits ? static_cast<int>(min(slot, static_cast<int64_t>(INT32_MAX))) : -1;
      int phys = -1;
      if (fits && L.k_cache) {
        phys = L.page_table[static_cast<size_t>(b) * L.max_pages_per_req + slot / L.page_size];
        if (phys >= L.num_pages) phys = -1;
      }
      s_phys[tid / 32] = phys;
    }
  }
  __syncthreads();
  // The angle in turns, in 64 bits, less its whole turns; the rest is at most half a turn, which fp32
  // holds to 2^-25 of a turn.  (Far positions have angles of 10^5 and more: fp32 would lose them.)
  const int half = L.rotary_dim / 2;
  for (int i = tid; i < ntok * half; i += kThreads) {
    const int j = i / half, f = i - j * half;
    const int pos = L.positions ? L.positions[t0 + j] : s_slot[j];
    constexpr double kInvTwoPi = 0.15915494309189533577;
    const double turns = static_cast<double>(pos) * L.inv_freq[f] * kInvTwoPi;
    float sn, cs;
    sincospif(2.0f * static_cast<float>(turns - rint(turns)), &sn, &cs);
    s_rot[j][f] = make_float2(cs, sn);
  }
  __syncthreads();

  const int lane = tid % kLanes;
  const int rot_chunks = L.rotary_dim / 8;        // chunks of eight rotated values
  const bool turned = lane < rot_chunks / 2;      // this lane's chunks are rotated (both or neither)
  const int c0 = turned ? lane : 2 * lane;
  const int c1 = turned ? lane + rot_chunks / 2 : 2 * lane + 1;
  const int rows = L.num_q_heads + L.num_kv_heads + (L.k_cache ? L.num_kv_heads : 0);
  for (int r0 = 0; r0 < ntok * rows; r0 += kRowsPerPass) {   // uniform over the CTA: the shuffles need every lane
    const int r = r0 + tid / kLanes;
    const bool in = r < ntok * rows;
    const int j = in ? r / rows : 0;
    const int head = in ? r - j * rows : 0;
    const int slot = s_slot[j];
    const int64_t t = t0 + j;
    const uint16_t *src, *w = nullptr;
    uint16_t *dst = nullptr, *dst2 = nullptr;
    const size_t page = (static_cast<size_t>(max(s_phys[j], 0)) * L.page_size + max(slot, 0) % L.page_size) * L.num_kv_heads;
    const bool paged = s_phys[j] >= 0;
    if (head < L.num_q_heads) {
      src = L.q + t * L.q_stride + static_cast<int64_t>(head) * D;
      dst = L.q_out + (t * L.num_q_heads + head) * D;
      w = L.q_weight;
    } else if (head < L.num_q_heads + L.num_kv_heads) {
      const int h = head - L.num_q_heads;
      src = L.k + t * L.k_stride + static_cast<int64_t>(h) * D;
      if (L.k_out) dst = L.k_out + (t * L.num_kv_heads + h) * D;
      if (paged) dst2 = L.k_cache + (page + h) * D;
      w = L.k_weight;
    } else {
      const int h = head - L.num_q_heads - L.num_kv_heads;
      src = L.v + t * L.v_stride + static_cast<int64_t>(h) * D;
      if (paged) dst2 = L.v_cache + (page + h) * D;
    }
    const bool value = head >= L.num_q_heads + L.num_kv_heads;
    uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
    if (in) {
      u0 = *reinterpret_cast<const uint4*>(src + 8 * c0);
      u1 = *reinterpret_cast<const uint4*>(src + 8 * c1);
    }
    float a[8], b[8];
    unpack8(u0, a);
    unpack8(u1, b);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
#pragma unroll
    for (int m = 1; m < kLanes; m *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    if (!in || slot < 0) continue;
    if (!value) {
      if (w) {
        const float inv = rsqrtf(ss * (1.0f / D) + L.eps);
        float wa[8], wb[8];
        unpack8(*reinterpret_cast<const uint4*>(w + 8 * c0), wa);
        unpack8(*reinterpret_cast<const uint4*>(w + 8 * c1), wb);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[i] = a[i] * inv * wa[i];
          b[i] = b[i] * inv * wb[i];
        }
      }
      if (turned) {
        if (L.interleaved) {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float2 ra = s_rot[j][4 * c0 + i / 2], rb = s_rot[j][4 * c1 + i / 2];
            const float x = a[i], y = b[i];
            a[i] = x * ra.x - a[i + 1] * ra.y;
            a[i + 1] = a[i + 1] * ra.x + x * ra.y;
            b[i] = y * rb.x - b[i + 1] * rb.y;
            b[i + 1] = b[i + 1] * rb.x + y * rb.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 rt = s_rot[j][8 * c0 + i];
            const float x = a[i];
            a[i] = x * rt.x - b[i] * rt.y;
            b[i] = b[i] * rt.x + x * rt.y;
          }
        }
      }
      u0 = pack8(a);
      u1 = pack8(b);
    }
    if (dst) {
      *reinterpret_cast<uint4*>(dst + 8 * c0) = u0;
      *reinterpret_cast<uint4*>(dst + 8 * c1) = u1;
    }
    if (dst2) {
      *reinterpret_cast<uint4*>(dst2 + 8 * c0) = u0;
      *reinterpret_cast<uint4*>(dst2 + 8 * c1) = u1;
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch& L, cudaStream_t stream) {
  const int per = L.total_tokens >= 8 * 152 ? kMaxTokens : 1;
  const unsigned grid = static_cast<unsigned>((L.total_tokens + per - 1) / per);
  if (L.head_dim == 128)
    rope_kernel<128><<<grid, kThreads, 0, stream>>>(L, per);
  else
    rope_kernel<64><<<grid, kThreads, 0, stream>>>(L, per);
  return cudaGetLastError();
}

}  // namespace cosa_kv
