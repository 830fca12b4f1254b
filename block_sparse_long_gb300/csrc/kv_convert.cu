// K and V into the 4-bit cache and back (layout: include/cosa_kv.h).
//
// Per group of 32 values:  s = bf16(max|x| / 7),  c = clamp(rint(x / s), -7, 7).  Eight values of a
// token's head are a lane's work: lane (g, c) of the D / 8 lanes of a row holds values 32 g + 8 c .. + 7,
// which are one 32-bit word of the K layout and two 16-bit words of the V layout; the four lanes of a group
// share their largest magnitude by two shuffles.  Both directions are memory bound: 4 d bytes of bf16
// and 9/8 d bytes of cache per token and kv head.
#include <cstdint>

#include "cosa_kv.h"
#include "kv_internal.h"
#include "kv_layout.cuh"

namespace cosa_kv {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 8;     // tokens of a CTA

// Codes of a lane's eight values, lowest nibble first, and the bits of their group's scale.  Nibble n of each
// half has the magnitude of value n, and the sign of value n ^ 2 in its high bit.  Every lane of the warp calls it.
__device__ __forceinline__ uint32_t quantise8(const uint4& u, uint32_t& scale_bits) {
  float x[8];
  unpack8(u, x);
  // the magnitudes as integers keep their order, with infinities and NaN above every number
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  if (m >= 0x7F800000u) {
    scale_bits = 0x7FC0u;
    return 0u;
  }
  const float s = __uint_as_float(cosa::pack_bf16x2(0.f, __uint_as_float(m) / 7.0f) & 0xFFFF0000u);
  scale_bits = __float_as_uint(s) >> 16;
  if (s == 0.f) return 0u;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = static_cast<int>(fminf(fmaxf(rintf(x[i] / s), -7.f), 7.f));
    w |= static_cast<uint32_t>(abs(c)) << (4 * i);
    w |= c < 0 ? 8u << (4 * (i ^ 2)) : 0u;
  }
  return w;
}

// Eight values from their codes: the products are exact in fp32 and rounded once.
__device__ __forceinline__ uint4 dequantise8(uint32_t w, float s) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float m = static_cast<float>((w >> (4 * i)) & 7u) * s;
    x[i] = (w >> (4 * (i ^ 2))) & 8u ? -m : m;
  }
  return pack8(x);
}

template <int D>
__device__ __forceinline__ void put(uint8_t* tile, int t, int lane, uint32_t kw, uint32_t ks, uint32_t vw, uint32_t vs) {
  using T = Tile<D>;
  const int g = lane / 4, c = lane % 4;
  *reinterpret_cast<uint32_t*>(tile + t * T::kRow + (c * T::G + g) * 4) = kw;
  uint16_t* v = reinterpret_cast<uint16_t*>(tile + T::kVCodes + v_row(t) * T::kRow);
  v[(2 * c) * T::G + g] = static_cast<uint16_t>(vw);
  v[(2 * c + 1) * T::G + g] = static_cast<uint16_t>(vw >> 16);
  if (c == 0) {
    *reinterpret_cast<uint16_t*>(tile + T::kKScales + (t * T::G + g) * 2) = static_cast<uint16_t>(ks);
    *reinterpret_cast<uint16_t*>(tile + T::kVScales + (t * T::G + g) * 2) = static_cast<uint16_t>(vs);
  }
}

// Slots first .. end - 1 of request b; a contradiction gives an empty range and the status.
__device__ __forceinline__ Range slots_of(const ConvertLaunch& L, int b, int len, int from) {
  Range r{from, len, true};
  if (from < 0 || len < 0 || len > L.max_seqlen) r = Range{0, 0, false};
  return r;
}

__device__ __forceinline__ int page_of(const int32_t* table, const ConvertLaunch& L, int b, int slot, int pages) {
  const int phys = table[static_cast<size_t>(b) * L.max_pages_per_req + slot / L.page_size];
  return phys >= 0 && phys < pages ? phys : -1;
}

// Rows packed by cu_seqlens; a CTA takes kTokens tokens of the batch.
template <int D>
__global__ void __launch_bounds__(kThreads) store_rows_kernel(const ConvertLaunch L) {
  constexpr int kLanes = D / 8;
  __shared__ int s_slot[kTokens], s_phys[kTokens];
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * kTokens;
  const int last = L.cu_seqlens[L.num_reqs];
  if (blockIdx.x == 0 && tid == 0 && (L.cu_seqlens[0] != 0 || last > L.total_tokens))
    cosa::report_status(L.status, cosa::kStatusBadInput);
  const int ntok = min(kTokens, min(last, L.total_tokens) - t0);
  if (ntok <= 0) return;
  if (tid / 32 < ntok) {
    const int t = t0 + tid / 32, lane = tid % 32;
    int b = 0;
    for (int i = lane; i < L.num_reqs; i += 32) b += L.cu_seqlens[i + 1] <= t;
    b = __reduce_add_sync(0xffffffffu, b);
    if (lane == 0) {
      const int off = b < L.num_reqs ? t - L.cu_seqlens[b] : -1;
      const int64_t slot = off < 0 ? -1 : static_cast<int64_t>(off) + (L.start ? L.start[b] : 0);
      const bool fits = slot >= 0 && slot < L.max_seqlen;
      if (!fits) cosa::report_status(L.status, cosa::kStatusBadInput);
      s_slot[tid / 32] = fits ? static_cast<int>(slot) : 0;
      s_phys[tid / 32] = fits ? page_of(L.page_table, L, b, static_cast<int>(slot), L.num_kv4_pages) : -1;
    }
  }
  __syncthreads();
  const int lane = tid % kLanes;
  const int rows = ntok * L.num_kv_heads;
  for (int r0 = 0; r0 < rows; r0 += kThreads / kLanes) {     // uniform: the shuffles need every lane
    const int r = r0 + tid / kLanes;
    const bool in = r < rows;
    const int j = in ? r / L.num_kv_heads : 0;
    const int h = in ? r - j * L.num_kv_heads : 0;
    const int64_t t = t0 + j;
    uint4 ku = make_uint4(0, 0, 0, 0), vu = ku;
    if (in) {
      ku = *reinterpret_cast<const uint4*>(L.k + t * L.k_stride + static_cast<int64_t>(h) * D + 8 * lane);
      vu = *reinterpret_cast<const uint4*>(L.v + t * L.v_stride + static_cast<int64_t>(h) * D + 8 * lane);
    }
    uint32_t ks, vs;
    const uint32_t kw = quantise8(ku, ks), vw = quantise8(vu, vs);
    if (in && s_phys[j] >= 0)
      put<D>(L.cache + tile_offset<D>(s_phys[j], h, s_slot[j], L.num_kv_heads, L.page_size), s_slot[j] % kTile, lane, kw,
             ks, vw, vs);
  }
}

// Pages to pages; a CTA takes kTokens slots of request blockIdx.y.  LOAD: from the cache to bf16 pages.
template <int D, bool LOAD>
__global__ void __launch_bounds__(kThreads) pages_kernel(const ConvertLaunch L) {
  using T = Tile<D>;
  constexpr int kLanes = D / 8;
  const int tid = threadIdx.x;
  const int b = blockIdx.y;
  const Range range = slots_of(L, b, L.kv_len[b], L.start ? L.start[b] : 0);
  if (!range.ok && blockIdx.x == 0 && tid == 0) cosa::report_status(L.status, cosa::kStatusBadInput);
  // from the tile boundary at or before the first slot
  const int64_t s0 = static_cast<int64_t>(range.first / kTile * kTile) + static_cast<int64_t>(blockIdx.x) * kTokens;
  if (s0 >= range.end) return;
  const int slot0 = static_cast<int>(s0);
  // kTokens divides 16, so the slots of a CTA share their pages
  const int p4 = page_of(L.page_table, L, b, slot0, L.num_kv4_pages);
  const int p16 = page_of(L.other_table, L, b, slot0, L.num_pages);
  if (p4 < 0 || p16 < 0) return;
  const int lane = tid % kLanes;
  const int rows = kTokens * L.num_kv_heads;
  for (int r0 = 0; r0 < rows; r0 += kThreads / kLanes) {     // uniform: the shuffles need every lane
    const int r = r0 + tid / kLanes;
    const int j = r < rows ? r / L.num_kv_heads : 0;
    const int h = r < rows ? r - j * L.num_kv_heads : 0;
    const int slot = slot0 + j;
    const bool in = r < rows && slot >= range.first && slot < range.end;
    const size_t at = ((static_cast<size_t>(p16) * L.page_size + slot % L.page_size) * L.num_kv_heads + h) * D + 8 * lane;
    uint8_t* tile = L.cache + tile_offset<D>(p4, h, slot, L.num_kv_heads, L.page_size);
    const int t = slot % kTile;
    if (LOAD) {
      if (!in) continue;
      const int g = lane / 4, c = lane % 4;
      const uint32_t kw = *reinterpret_cast<const uint32_t*>(tile + t * T::kRow + (c * T::G + g) * 4);
      const uint16_t* v = reinterpret_cast<const uint16_t*>(tile + T::kVCodes + v_row(t) * T::kRow);
      const uint32_t vw = v[(2 * c) * T::G + g] | (static_cast<uint32_t>(v[(2 * c + 1) * T::G + g]) << 16);
      const float ks = bf16_lo(*reinterpret_cast<const uint16_t*>(tile + T::kKScales + (t * T::G + g) * 2));
      const float vs = bf16_lo(*reinterpret_cast<const uint16_t*>(tile + T::kVScales + (t * T::G + g) * 2));
      *reinterpret_cast<uint4*>(L.k_cache + at) = dequantise8(kw, ks);
      *reinterpret_cast<uint4*>(L.v_cache + at) = dequantise8(vw, vs);
    } else {
      uint4 ku = make_uint4(0, 0, 0, 0), vu = ku;
      if (in) {
        ku = *reinterpret_cast<const uint4*>(L.k + at);
        vu = *reinterpret_cast<const uint4*>(L.v + at);
      }
      uint32_t ks, vs;
      const uint32_t kw = quantise8(ku, ks), vw = quantise8(vu, vs);
      if (in) put<D>(tile, t, lane, kw, ks, vw, vs);
    }
  }
}

}  // namespace

cudaError_t launch_store_rows(const ConvertLaunch& L, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((L.total_tokens + kTokens - 1) / kTokens);
  if (L.head_dim == 128)
    store_rows_kernel<128><<<grid, kThreads, 0, stream>>>(L);
  else
    store_rows_kernel<64><<<grid, kThreads, 0, stream>>>(L);
  return cudaGetLastError();
}

cudaError_t launch_store_pages(const ConvertLaunch& L, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(L.max_seqlen) + kTokens - 1) / kTokens), static_cast<unsigned>(L.num_reqs));
  if (L.head_dim == 128)
    pages_kernel<128, false><<<grid, kThreads, 0, stream>>>(L);
  else
    pages_kernel<64, false><<<grid, kThreads, 0, stream>>>(L);
  return cudaGetLastError();
}

cudaError_t launch_load(const ConvertLaunch& L, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(L.max_seqlen) + kTokens - 1) / kTokens), static_cast<unsigned>(L.num_reqs));
  if (L.head_dim == 128)
    pages_kernel<128, true><<<grid, kThreads, 0, stream>>>(L);
  else
    pages_kernel<64, true><<<grid, kThreads, 0, stream>>>(L);
  return cudaGetLastError();
}

}  // namespace cosa_kv
