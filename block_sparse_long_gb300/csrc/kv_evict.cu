// Eviction by accumulated attention weight.
//
// Per (request, kv head): of the slots that exist, the first `sink` and last `recent` ones, then those with the
// largest weights (ties: the lowest slot), `budget` in all; kept slots move in order into other pages.
//
// A slot's weight becomes a 32-bit key that sorts as the weight does (missing pages 0, NaN 1, kept in any
// case the largest), so the K-th largest key is found by a radix select and everything above it is
// kept, with the lowest slots among the equal ones.  The move copies whole rows of codes and scales.
// Work: 4 bytes per slot and 9/4 d bytes per kept slot, memory bound.
#include <cstdint>

#include "cosa_kv.h"
#include "kv_internal.h"
#include "kv_layout.cuh"

namespace cosa_kv {
namespace {

constexpr int kSelectThreads = 1024;
constexpr uint32_t kMissing = 0u, kNan = 1u, kAlways = 0xFFFFFFFFu;

__device__ __forceinline__ uint32_t key_of(float w) {
  if (isnan(w)) return kNan;
  const uint32_t u = __float_as_uint(w + 0.0f);       // -0 as 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int length_of(const EvictLaunch& L, int b) {
  const int n = L.kv_len[b];
  return n < 0 || n > L.max_seqlen ? 0 : n;
}

__device__ __forceinline__ int page_of(const int32_t* table, int pitch, const EvictLaunch& L, int b, int slot) {
  const int phys = table[static_cast<size_t>(b) * pitch + slot / L.page_size];
  return phys >= 0 && phys < L.num_kv4_pages ? phys : -1;
}

// Exclusive prefix of a flag over the CTA and the CTA's total.
__device__ __forceinline__ int block_prefix(bool flag, int* s_warp, int& total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const unsigned m = __ballot_sync(0xffffffffu, flag);
  __syncthreads();
  if (lane == 0) s_warp[warp] = __popc(m);
  __syncthreads();
  int v = s_warp[lane];          // kSelectThreads / 32 = 32 warps
  const int own = v;
#pragma unroll
  for (int k = 1; k < 32; k *= 2) {
    const int x = __shfl_up_sync(0xffffffffu, v, k);
    if (lane >= k) v += x;
  }
  total = __shfl_sync(0xffffffffu, v, 31);
  return __shfl_sync(0xffffffffu, v - own, warp) + __popc(m & ((1u << lane) - 1u));
}

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const EvictLaunch L) {
  __shared__ int s_hist[256];
  __shared__ int s_warp[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_want, s_keep;
  const int tid = threadIdx.x;
  const int b = blockIdx.x / L.num_kv_heads, h = blockIdx.x % L.num_kv_heads;
  const int n = length_of(L, b);
  if (tid == 0 && h == 0 && n != L.kv_len[b]) cosa::report_status(L.status, cosa::kStatusBadInput);
  const size_t row = static_cast<size_t>(b) * L.num_kv_heads + h;
  const float* w = L.weights + row * L.max_seqlen;
  auto key = [&](int s) -> uint32_t {
    if (page_of(L.page_table, L.max_pages_per_req, L, b, s) < 0) return kMissing;
    if (s < L.sink || s >= n - L.recent) return kAlways;
    return key_of(w[s]);
  };

  // the K-th largest key, eight bits at a time from the top
  uint32_t prefix = 0;
  int want = 0, keep = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) s_hist[tid] = 0;
    __syncthreads();
    for (int s = tid; s < n; s += kSelectThreads) {
      const uint32_t k = key(s);
      if (k != kMissing && (shift == 24 || (k >> (shift + 8)) == prefix)) atomicAdd(&s_hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (tid < 32) {          // lane l has bins 255 - 8 l down to 248 - 8 l
      int mine = 0;
      for (int j = 0; j < 8; ++j) mine += s_hist[255 - 8 * tid - j];
      int end = mine;
#pragma unroll
      for (int k = 1; k < 32; k *= 2) {
        const int x = __shfl_up_sync(0xffffffffu, end, k);
        if (tid >= k) end += x;
      }
      if (shift == 24) {
        keep = min(L.budget, __shfl_sync(0xffffffffu, end, 31));
        want = keep;
        if (tid == 0) s_keep = keep;
      }
      const unsigned past = __ballot_sync(0xffffffffu, end >= want);
      if (want > 0 && tid == __ffs(past) - 1) {
        int before = end - mine, j = 0;
        while (before + s_hist[255 - 8 * tid - j] < want) before += s_hist[255 - 8 * tid - j++];
        s_prefix = (prefix << 8) | static_cast<uint32_t>(255 - 8 * tid - j);
        s_want = want - before;
      }
    }
    __syncthreads();
    keep = s_keep;
    if (keep == 0) break;    // uniform: nothing exists
    prefix = s_prefix;
    want = s_want;
  }

  // kept slots in ascending order
  int32_t* kept = L.kept + row * L.budget;
  int out = 0, ties = 0;
  for (int s0 = 0; keep > 0 && s0 < n; s0 += kSelectThreads) {
    const int s = s0 + tid;
    const uint32_t k = s < n ? key(s) : kMissing;
    int total;
    const int tie = ties + block_prefix(k == prefix && k != kMissing, s_warp, total);
    ties += total;
    const bool in = k != kMissing && (k > prefix || (k == prefix && tie < want));
    const int at = out + block_prefix(in, s_warp, total);
    out += total;
    if (in) kept[at] = s;
  }
  for (int j = keep + tid; j < L.budget; j += kSelectThreads) kept[j] = -1;
  if (tid == 0 && h == 0) L.new_len[b] = keep;
  if (L.weights_out) {
    __syncthreads();
    float* o = L.weights_out + row * L.max_seqlen;
    for (int j = tid; j < L.max_seqlen; j += kSelectThreads) o[j] = j < keep ? w[kept[j]] : 0.f;
  }
}

// One destination tile of 16 slots per CTA.
template <int D>
__global__ void __launch_bounds__(128) move_kernel(const EvictLaunch L) {
  using T = Tile<D>;
  const int tid = threadIdx.x;
  const int b = blockIdx.z, h = blockIdx.y, slot0 = blockIdx.x * kTile;
  const int rows = min(kTile, L.new_len[b] - slot0);
  if (rows <= 0) return;
  const int dst_phys = page_of(L.dst_page_table, L.max_dst_pages, L, b, slot0);
  if (dst_phys < 0) return;
  __shared__ const uint8_t* s_src[kTile];
  __shared__ int s_row[kTile];
  if (tid < rows) {
    const int s = L.kept[(static_cast<size_t>(b) * L.num_kv_heads + h) * L.budget + slot0 + tid];
    s_src[tid] = L.cache + tile_offset<D>(page_of(L.page_table, L.max_pages_per_req, L, b, s), h, s, L.num_kv_heads, L.page_size);
    s_row[tid] = s % kTile;
  }
  __syncthreads();
  uint8_t* dst = L.cache + tile_offset<D>(dst_phys, h, slot0, L.num_kv_heads, L.page_size);
  constexpr int kChunks = T::kRow / 16;      // 16-byte pieces of a row of codes
  for (int k = tid; k < rows * (2 * kChunks + 2); k += 128) {
    const int t = k / (2 * kChunks + 2), j = k % (2 * kChunks + 2);
    const uint8_t* src = s_src[t];
    const int from = s_row[t];
    if (j < kChunks) {
      *reinterpret_cast<uint4*>(dst + t * T::kRow + 16 * j) = *reinterpret_cast<const uint4*>(src + from * T::kRow + 16 * j);
    } else if (j < 2 * kChunks) {
      const int x = 16 * (j - kChunks);
      *reinterpret_cast<uint4*>(dst + T::kVCodes + v_row(t) * T::kRow + x) =
          *reinterpret_cast<const uint4*>(src + T::kVCodes + v_row(from) * T::kRow + x);
    } else {
      const int base = j == 2 * kChunks ? T::kKScales : T::kVScales;
      if constexpr (T::G == 4)
        *reinterpret_cast<uint2*>(dst + base + t * 8) = *reinterpret_cast<const uint2*>(src + base + from * 8);
      else
        *reinterpret_cast<uint32_t*>(dst + base + t * 4) = *reinterpret_cast<const uint32_t*>(src + base + from * 4);
    }
  }
}

}  // namespace

cudaError_t launch_evict(const EvictLaunch& L, cudaStream_t stream) {
  select_kernel<<<static_cast<unsigned>(L.num_reqs * L.num_kv_heads), kSelectThreads, 0, stream>>>(L);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(L.budget) + kTile - 1) / kTile), static_cast<unsigned>(L.num_kv_heads),
                  static_cast<unsigned>(L.num_reqs));
  if (L.head_dim == 128)
    move_kernel<128><<<grid, 128, 0, stream>>>(L);
  else
    move_kernel<64><<<grid, 128, 0, stream>>>(L);
  return cudaGetLastError();
}

}  // namespace cosa_kv
