// Eviction by accumulated attention weight.
//
// Per (request, kv head): of the slots that exist, the first `sink` and last `recent` ones, then those with the
// largest weights (ties: the lowest slot), `budget` in all; kept slots move in order into other pages.
//
// A slot's weight becomes a 32-bit key that sorts as the weight does (missing pages 0, NaN 1, kept in any case the
// largest).  A cluster of one to sixteen CTAs has the slots of one (request, kv head), a run each, their keys in shared
// memory.  The K-th largest key is found by a radix select, 11 bits at a time from the top: every CTA counts its
// keys' digits, sums its share of the bins over the cluster through distributed shared memory, and looks the
// digit up among the sums.  Everything above the K-th key is kept, and the lowest slots among the equal ones; the
// numbers of both in the earlier CTAs and warps, and votes within 32 neighbouring keys, give each kept slot its place.  The
// move then copies whole rows of codes and scales.
//
// Work: 8 bytes per slot and 9/4 d bytes per kept slot.  Measured, 131072 slots of 8 heads of 128 to 16384: 28 us, of which the
// select takes about 16, bound by the latency of its chain of loads, counts and barriers (sixteen CTAs a head), and the move 13
// for 38 MB, of which the scattered rows make 50 MB of reads.  24 requests of 16000 to 4000: 76 us, 221 MB moved; the
// select's 25 us are a CTA a head, two on some SMs.  A run of keys per thread instead of per warp took 33 and 90 us; one CTA
// a head, from global memory, 400 us.
#include <algorithm>
#include <cstdint>

#include <cooperative_groups.h>

#include "cosa_kv.h"
#include "kv_internal.h"
#include "kv_layout.cuh"

namespace cosa_kv {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelectThreads = 512;
constexpr int kWarps = kSelectThreads / 32;
constexpr int kCluster = 16;            // CTAs of a cluster at most
constexpr int kBins = 2048;
constexpr int kMaxKeys = 16384;         // keys that a CTA holds; longer runs are formed again for each pass
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
  const int phys = table[static_cast<size_t>(b) * pitch + (slot >> L.page_shift)];
  return phys >= 0 && phys < L.num_kv4_pages ? phys : -1;
}

// Inclusive sum over a warp's lanes.
__device__ __forceinline__ int warp_scan(int v) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int k = 1; k < 32; k *= 2) {
    const int x = __shfl_up_sync(0xffffffffu, v, k);
    if (lane >= k) v += x;
  }
  return v;
}

// Exclusive sum over the CTA's threads, and the CTA's total.  Ends with the CTA synchronised.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int end = warp_scan(v);
  if (lane == 31) s_warp[warp] = end;
  __syncthreads();
  const int w = lane < kWarps ? s_warp[lane] : 0;
  const int sums = warp_scan(w);
  total = __shfl_sync(0xffffffffu, sums, kWarps - 1);
  const int before = __shfl_sync(0xffffffffu, sums - w, warp);
  __syncthreads();
  return before + end - v;
}

struct SelectSmem {
  int hist[kBins];                // this CTA's digits
  alignas(16) int sums[kBins];    // this CTA's share of the bins over the cluster, from the top: kBins / ctas of them
  int share_total;                // their total
  int counts[2];                  // keep and want of the passes
  int mine[2];                    // this CTA's keys above the K-th, and equal to it
  int warp[32];
  uint32_t digit;
};

// Slots in flight per thread while the keys are formed; the keys' number is rounded up to whole steps (with kMissing).
constexpr int kDeep = 8;
__host__ __device__ constexpr int whole_steps(int run) {
  constexpr int kStep = kDeep * kSelectThreads;
  return (run + kStep - 1) / kStep * kStep;
}
static_assert(kMaxKeys == whole_steps(kMaxKeys), "held keys");

// HELD: the run's keys fit in shared memory.
template <bool HELD>
__global__ void __launch_bounds__(kSelectThreads, 3) select_kernel(const EvictLaunch L) {
  extern __shared__ uint32_t s_keys[];
  __shared__ SelectSmem sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x;
  const int item = static_cast<int>(blockIdx.x) / ctas;
  const int b = item / L.num_kv_heads, h = item % L.num_kv_heads;
  wait_for_stream();
  let_next_start();
  const int n = length_of(L, b);
  if (tid == 0 && rank == 0 && h == 0 && n != L.kv_len[b]) cosa::report_status(L.status, cosa::kStatusBadInput);
  const size_t row = static_cast<size_t>(b) * L.num_kv_heads + h;
  const float* w = L.weights + row * L.max_seqlen;
  // this CTA's run of slots
  const int run = (n + ctas - 1) / ctas;
  const int lo = min(n, rank * run), len = min(n, lo + run) - lo;

  const int32_t* table = L.page_table + static_cast<size_t>(b) * L.max_pages_per_req;
  auto form = [&](int s, int phys, float weight) -> uint32_t {
    if (phys < 0 || phys >= L.num_kv4_pages) return kMissing;
    return s < L.sink || s >= n - L.recent ? kAlways : key_of(weight);
  };
  // key of slot lo + i; kMissing behind the run
  auto key = [&](int i) -> uint32_t {
    if (HELD) return s_keys[i];
    return i < len ? form(lo + i, table[(lo + i) >> L.page_shift], w[lo + i]) : kMissing;
  };
  for (int i = tid; i < kBins; i += kSelectThreads) sm.hist[i] = 0;
  __syncthreads();
  if (HELD) {                         // the first pass counts the keys as they are formed
    for (int i0 = tid; i0 - tid < len; i0 += kDeep * kSelectThreads) {
      float weight[kDeep];
      int phys[kDeep];
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        const int i = i0 + k * kSelectThreads;
        weight[k] = i < len ? w[lo + i] : 0.f;
        phys[k] = i < len ? table[(lo + i) >> L.page_shift] : -1;
      }
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        const int i = i0 + k * kSelectThreads;
        const uint32_t x = form(lo + i, phys[k], weight[k]);
        s_keys[i] = x;
        if (x != kMissing) atomicAdd(&sm.hist[x >> 21], 1);
      }
    }
  }

  const int share = kBins / ctas;
  uint32_t prefix = 0;              // the digits found so far
  int want = 0, keep = 0;           // how many keys with this prefix are kept; how many keys in all
  int used = 0;                     // bits of the prefix
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass == 2 ? 10 : 11, shift = 32 - used - bits;
    if (pass > 0) {
      for (int i = tid; i < kBins; i += kSelectThreads) sm.hist[i] = 0;
      __syncthreads();
    }
    if (!HELD || pass > 0) {
      constexpr int kBatch = 4;       // keys asked for together: a count could be to their address, for all the compiler knows
      for (int i0 = tid; i0 - tid < len; i0 += kBatch * kSelectThreads) {
        uint32_t x[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) x[k] = key(i0 + k * kSelectThreads);
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (x[k] != kMissing && (pass == 0 || (x[k] >> (shift + bits)) == prefix))
            atomicAdd(&sm.hist[(x[k] >> shift) & ((1u << bits) - 1u)], 1);
      }
    }
    cluster.sync();
    if (ctas > 1) {                 // (the cluster has read the sums of the pass before; a CTA alone takes its own bins)
      for (int i = tid; i < share; i += kSelectThreads) sm.sums[i] = 0;
      __syncthreads();
      // This CTA's share of the bins, summed over the cluster: a thread per bin and per four CTAs, whose loads go together.
      for (int i = tid; i < share * ((ctas + 3) / 4); i += kSelectThreads) {
        const int bin = i & (share - 1), r0 = i / share * 4;
        int v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = r0 + k < ctas ? cluster.map_shared_rank(sm.hist, r0 + k)[rank * share + bin] : 0;
        atomicAdd(&sm.sums[share - 1 - bin], (v[0] + v[1]) + (v[2] + v[3]));
      }
      __syncthreads();
    }
    // then, from the top bin down, the number of keys in the bins so far; a thread has up to four neighbouring bins
    {
      const int each = max(1, share / kSelectThreads);
      int v[kBins / kSelectThreads], own = 0, total;
#pragma unroll
      for (int k = 0; k < kBins / kSelectThreads; ++k) {
        const int i = tid * each + k;
        v[k] = k < each && tid * each < share ? (ctas > 1 ? sm.sums[i] : sm.hist[kBins - 1 - i]) : 0;
        own += v[k];
      }
      int upto = block_scan(own, sm.warp, total);
#pragma unroll
      for (int k = 0; k < kBins / kSelectThreads; ++k) {
        upto += v[k];
        if (k < each && tid * each < share) sm.sums[tid * each + k] = upto;
      }
      if (tid == 0) sm.share_total = total;
    }
    cluster.sync();
    // The digit: shares from the top, then the bins of the share that has it (a warp, in every CTA alike).
    if (tid < 32) {
      const int r = ctas - 1 - tid;                   // lane 0 has the top share
      const int mine = r >= 0 ? *cluster.map_shared_rank(&sm.share_total, r) : 0;
      const int end = warp_scan(mine);
      if (pass == 0) want = keep = min(L.budget, __shfl_sync(0xffffffffu, end, 31));
      const int at = __ffs(__ballot_sync(0xffffffffu, end >= want)) - 1;      // want <= the total: there is one
      const int owner = max(ctas - 1 - at, 0);
      int before = __shfl_sync(0xffffffffu, end - mine, at);
      // the bins above the digit are those with which the sum stays below `want`
      const int4* sums = reinterpret_cast<const int4*>(cluster.map_shared_rank(sm.sums, owner));
      int above = 0, most = 0;
#pragma unroll 4
      for (int i = tid; i < share / 4; i += 32) {
        const int4 v = sums[i];
        above += (before + v.x < want) + (before + v.y < want) + (before + v.z < want) + (before + v.w < want);
        most = max(most, max(max(before + v.x < want ? v.x : 0, before + v.y < want ? v.y : 0),
                             max(before + v.z < want ? v.z : 0, before + v.w < want ? v.w : 0)));
      }
      above = min(__reduce_add_sync(0xffffffffu, above), share - 1);
      before += __reduce_max_sync(0xffffffffu, most);
      const uint32_t digit = static_cast<uint32_t>(owner * share + share - 1 - above);
      if (tid == 0) {
        sm.digit = digit;
        sm.counts[0] = keep;
        sm.counts[1] = want - before;
      }
    }
    __syncthreads();
    keep = sm.counts[0];
    want = sm.counts[1];
    prefix = (prefix << bits) | sm.digit;
    used += bits;
    if (keep == 0) break;           // the same in the whole cluster: no slot exists
  }
  // here `prefix` is the K-th largest key and `want` the number of its equals that are kept

  int32_t* kept = L.kept + row * L.budget;
  if (keep > 0) {
    // Neighbouring keys to neighbouring lanes, a run of them to every warp: within 32 keys the places come from votes.
    const int lane = tid % 32, warp = tid / 32;
    const int per = (len + kSelectThreads - 1) / kSelectThreads * 32;
    const int first = warp * per, last = min(len, first + per);
    int above = 0, equal = 0;
#pragma unroll 4
    for (int i = first + lane; i - lane < last; i += 32) {
      const uint32_t x = key(i);
      above += x > prefix;
      equal += x == prefix;           // (the K-th key is a slot's: not kMissing)
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
      sm.warp[warp] = above;
      sm.warp[kWarps + warp] = equal;
    }
    __syncthreads();
    above = lane < kWarps ? sm.warp[lane] : 0;
    equal = lane < kWarps ? sm.warp[kWarps + lane] : 0;
    const int total_above = __reduce_add_sync(0xffffffffu, above), total_equal = __reduce_add_sync(0xffffffffu, equal);
    above = __reduce_add_sync(0xffffffffu, lane < warp ? above : 0);
    equal = __reduce_add_sync(0xffffffffu, lane < warp ? equal : 0);
    if (tid == 0) {
      sm.mine[0] = total_above;
      sm.mine[1] = total_equal;
    }
    cluster.sync();
    // what the CTAs before this one have: a lane for each
    int before_above = 0, before_equal = 0;
    if (lane < rank) {
      const int* c = cluster.map_shared_rank(sm.mine, lane);
      before_above = c[0];
      before_equal = c[1];
    }
    above += __reduce_add_sync(0xffffffffu, before_above);
    equal += __reduce_add_sync(0xffffffffu, before_equal);
    cluster.barrier_arrive();       // this thread reads no other CTA's shared memory any more
    const unsigned before = (1u << lane) - 1u;
#pragma unroll 4
    for (int i = first + lane; i - lane < last; i += 32) {
      const uint32_t x = key(i);
      const unsigned a = __ballot_sync(0xffffffffu, x > prefix), e = __ballot_sync(0xffffffffu, x == prefix);
      const int place = equal + __popc(e & before);
      if (x > prefix || (x == prefix && place < want)) kept[above + __popc(a & before) + min(place, want)] = lo + i;
      above += __popc(a);
      equal += __popc(e);
    }
  }
  for (int j = keep + rank * kSelectThreads + tid; j < L.budget; j += ctas * kSelectThreads) kept[j] = -1;
  if (L.weights_out)
    for (int j = keep + rank * kSelectThreads + tid; j < L.max_seqlen; j += ctas * kSelectThreads)
      L.weights_out[row * L.max_seqlen + j] = 0.f;
  if (tid == 0 && rank == 0 && h == 0) L.new_len[b] = keep;
  // a CTA's shared memory lives until its neighbours have read it
  if (keep == 0) cluster.barrier_arrive();
  cluster.barrier_wait();
}

// A destination tile of 16 slots per warp, all of whose pieces are in flight at once.
constexpr int kMoveWarps = 8;
template <int D>
__global__ void __launch_bounds__(32 * kMoveWarps) move_kernel(const EvictLaunch L) {
  using T = Tile<D>;
  constexpr int kChunks = T::kRow / 16;      // 16-byte pieces of a row of codes
  constexpr int kSteps = kChunks / 2;        // pieces of the tile's codes per lane, of K and of V
  const int lane = threadIdx.x % 32;
  const int b = blockIdx.z, h = blockIdx.y;
  const int slot0 = static_cast<int>(blockIdx.x * kMoveWarps + threadIdx.x / 32) * kTile;
  wait_for_stream();
  const int rows = min(kTile, L.new_len[b] - slot0);
  if (rows <= 0) return;
  const size_t row = static_cast<size_t>(b) * L.num_kv_heads + h;
  // lane t < 16 looks up the source of slot t
  size_t from = 0;                           // its tile
  int at = 0;                                // its row there
  if (lane < rows) {
    const int s = L.kept[row * L.budget + slot0 + lane];
    const int phys = L.page_table[static_cast<size_t>(b) * L.max_pages_per_req + (s >> L.page_shift)];
    from = tile_offset<D>(phys, h, s, L.num_kv_heads, L.page_shift);
    at = s % kTile;
    if (L.weights_out) L.weights_out[row * L.max_seqlen + slot0 + lane] = L.weights[row * L.max_seqlen + s];
  }
  const int dst_phys = page_of(L.dst_page_table, L.max_dst_pages, L, b, slot0);
  if (dst_phys < 0) return;
  uint8_t* dst = L.cache + tile_offset<D>(dst_phys, h, slot0, L.num_kv_heads, L.page_shift);
  uint4 k[kSteps], v[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int t = (i * 32 + lane) / kChunks, x = 16 * (lane % kChunks);
    const uint8_t* src = L.cache + __shfl_sync(0xffffffffu, from, t) + x;
    const int r = __shfl_sync(0xffffffffu, at, t);
    if (t < rows) {
      k[i] = *reinterpret_cast<const uint4*>(src + r * T::kRow);
      v[i] = *reinterpret_cast<const uint4*>(src + T::kVCodes + v_row(r) * T::kRow);
    }
  }
  // scales: lanes 0 to 15 of K, 16 to 31 of V
  const int t = lane % kTile, base = lane < kTile ? T::kKScales : T::kVScales;
  const uint8_t* src = L.cache + __shfl_sync(0xffffffffu, from, t) + base + __shfl_sync(0xffffffffu, at, t) * (2 * T::G);
  uint32_t sc[T::G / 2];
  if (t < rows)
#pragma unroll
    for (int g = 0; g < T::G / 2; ++g) sc[g] = reinterpret_cast<const uint32_t*>(src)[g];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int t = (i * 32 + lane) / kChunks, x = 16 * (lane % kChunks);
    if (t < rows) {
      *reinterpret_cast<uint4*>(dst + t * T::kRow + x) = k[i];
      *reinterpret_cast<uint4*>(dst + T::kVCodes + v_row(t) * T::kRow + x) = v[i];
    }
  }
  if (t < rows)
#pragma unroll
    for (int g = 0; g < T::G / 2; ++g) reinterpret_cast<uint32_t*>(dst + base + t * (2 * T::G))[g] = sc[g];
}

// Clusters of as many CTAs as fill the card (24 requests of 16K, 8 heads: 192 of one CTA 76 us, 384 of two 80, 768 of four 91),
// while each still has 2048 slots: with fewer, the pass over the keys costs less than the barriers that sharing it takes (8000
// slots of 8 heads with 512 / 2048 / 4096 slots a CTA: 18.5 / 14.3 / 16.4 us); and as many as it takes to hold the keys (131072
// slots: sixteen CTAs a head 53.8 us, eight 57.1).
cudaError_t launch_select(const EvictLaunch& L, cudaStream_t stream) {
  const int64_t items = static_cast<int64_t>(L.num_reqs) * L.num_kv_heads;
  int ctas = 1;
  while (ctas < kCluster && ((items * ctas < 152 && static_cast<int64_t>(ctas) * 2048 < L.max_seqlen) ||
                             static_cast<int64_t>(ctas) * kMaxKeys < L.max_seqlen))
    ctas *= 2;
  const int run = (L.max_seqlen - 1) / ctas + 1;
  const bool held = run <= kMaxKeys;
  auto* kernel = held ? select_kernel<true> : select_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && held) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxKeys * 4);
  if (e != cudaSuccess) return e;
  return launch_after(kernel, dim3(static_cast<unsigned>(items * ctas)), kSelectThreads, held ? whole_steps(run) * 4 : 0,
                      stream, ctas, L);
}

}  // namespace

cudaError_t launch_evict(const EvictLaunch& L, cudaStream_t stream) {
  const cudaError_t e = launch_select(L, stream);
  if (e != cudaSuccess) return e;
  const int64_t most = std::min(L.budget, L.max_seqlen);
  const dim3 grid(static_cast<unsigned>((most + kMoveWarps * kTile - 1) / (kMoveWarps * kTile)), static_cast<unsigned>(L.num_kv_heads),
                  static_cast<unsigned>(L.num_reqs));
  return launch_after(L.head_dim == 128 ? move_kernel<128> : move_kernel<64>, grid, 32 * kMoveWarps, 0, stream, 1, L);
}

}  // namespace cosa_kv
