// RMS norm of each query and key head, position rotation, and the bf16 cache write, in one pass.
//
// Per head x of d values:  y = x * rsqrt(mean(x^2) + eps) * w, then for each of the rotary_dim / 2 pairs (a, b):
// (y_a cos t - y_b sin t, y_b cos t + y_a sin t) with t = position * inv_freq[i].  A value is read once and written
// once (4 bytes), for about ten operations: bound by the memory where a token has many rows.
//
// A warp has a token, or a part of its heads where the tokens are few: four rows (d = 128; eight for d = 64) at a
// time, a row on d / 16 lanes.  The angles of a lane are the same in every row, so they are formed once and stay in
// registers; nothing is shared between warps, and each has three rows per lane in flight.  Where a token has few rows, a
// warp has two or four tokens, each on its share of the rows.
//
// Measured: 128K tokens of 32 + 8 + 8 heads of 128 into pages, 487 us, 3.22 GB at 6.6 TB/s (97 % of the measured copy rate);
// 64 tokens, 3.8 us, bound by the chain of loads (request, position, frequencies); 9.6K tokens of 12 + 4 + 4 heads of 64, 15.8 us,
// 49 MB at 3.1 TB/s: the same chain and the angles are paid per token for 2.5 KB of rows each way (issue slots 59 % busy, warps wait
// for loads more than for anything else).  Runs of tokens on a warp, with the
// frequencies kept, took 593 us and more for the 128K tokens (each warp then walks memory alone, in 12 KB pieces).
#include <cstdint>
#include <type_traits>

#include "cosa_kv.h"
#include "kv_internal.h"
#include "kv_layout.cuh"

namespace cosa_kv {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 3;      // rows per lane in flight

// The angle pos * freq less its whole turns, in half turns (-1 to 1), by the double multiplication.
__device__ __forceinline__ float half_turns(int64_t pos, double freq) {
  constexpr double kInvTwoPi = 0.15915494309189533577;
  const double turns = static_cast<double>(pos) * freq * kInvTwoPi;
  return 2.0f * static_cast<float>(turns - rint(turns));
}

// The same in integers, for the frequencies of ordinary rotations, since the SM has few units for doubles: 51K tokens of 3 + 1
// heads of 64 take 19.9 us instead of 25.6, 64 tokens of 32 + 8 heads 4.2 instead of 4.8.  freq = m 2^(e - 1075) has a
// significand m of 53 bits; m times round(2^66 / 2 pi), shifted, is the turns of one position in units of 2^-64, whole
// turns dropped; times the position it is good to 2^-31 of a turn (for frequencies up to 2^6 to 2^-33).
__device__ __forceinline__ bool ordinary(double freq) {       // 2^-36 <= |freq| < 2^10
  const int e = static_cast<int>(static_cast<uint64_t>(__double_as_longlong(freq)) >> 52) & 0x7FF;
  return e >= 1023 - 36 && e < 1023 + 10;
}
__device__ __forceinline__ uint64_t turn_of(double freq) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(freq));
  const int right = (1077 - (static_cast<int>(bits >> 52) & 0x7FF)) & 127;      // 45 to 90 where it is ordinary
  const uint64_t m = (bits & ((1ull << 52) - 1)) | (1ull << 52);
  constexpr uint64_t kTurn = 11743562013128004906ull;
  const uint64_t hi = __umul64hi(m, kTurn), lo = m * kTurn;
  const uint64_t turn = right < 64 ? (hi << (64 - right)) | (lo >> right) : hi >> (right - 64);
  return bits >> 63 ? 0 - turn : turn;
}
__device__ __forceinline__ float half_turns(int64_t pos, uint64_t turn) {
  const uint64_t angle = turn * static_cast<uint64_t>(pos);
  const bool neg = angle >> 63;
  const uint64_t size = neg ? 0 - angle : angle;
  const float hi = __uint2float_rn(static_cast<uint32_t>(size >> 32)), lo = __uint2float_rn(static_cast<uint32_t>(size));
  const float x = fmaf(hi, 0x1p-31f, lo * 0x1p-63f);
  return neg ? -x : x;
}

// Lane l of a row has two chunks of eight values, chosen so that both halves of every rotation pair are in one
// lane: chunks l and l + rotary_dim / 16 of the rotated part, then what is left of the head two by two.
// (Interleaved pairs are neighbours: any choice.)
template <int D, int TOKENS, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) rope_kernel(const RopeLaunch L, const int split_log2) {
  constexpr int kLanes = D / 16;
  constexpr int kRows = 32 / kLanes / TOKENS;       // rows of a token at a time
  constexpr unsigned kAll = 0xffffffffu;
  const int tid = threadIdx.x, lane = tid % 32, l = lane % kLanes, sub = lane / kLanes % kRows, own = lane / kLanes / kRows;
  wait_for_stream();
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kThreads + tid) / 32;
  const int last = L.cu_seqlens[L.num_reqs];
  if (blockIdx.x == 0 && tid == 0 && (L.cu_seqlens[0] != 0 || last > L.total_tokens))
    cosa::report_status(L.status, cosa::kStatusBadInput);
  const int split = 1 << split_log2;
  const int64_t t0 = (unit >> split_log2) * TOKENS;
  const int total = min(last, L.total_tokens);
  if (t0 >= total) return;
  const int64_t t = min(t0 + own, static_cast<int64_t>(total) - 1);      // this lane's token
  bool live = t0 + own < total;
  const int part = static_cast<int>(unit) & (split - 1);

  const int rot_chunks = L.rotary_dim / 8;        // chunks of eight rotated values
  const bool turned = l < rot_chunks / 2;         // this lane's chunks are rotated (both or neither)
  const int c0 = turned ? l : 2 * l, c1 = turned ? l + rot_chunks / 2 : 2 * l + 1;
  const int rows = L.num_q_heads + L.num_kv_heads + (L.k_cache ? L.num_kv_heads : 0);
  auto load = [&](int row, uint4& u0, uint4& u1) {
    u0 = u1 = make_uint4(0, 0, 0, 0);
    if (row >= rows) return;
    const uint16_t* src;
    if (row < L.num_q_heads)
      src = L.q + t * L.q_stride + row * D;
    else if (row < L.num_q_heads + L.num_kv_heads)
      src = L.k + t * L.k_stride + (row - L.num_q_heads) * D;
    else
      src = L.v + t * L.v_stride + (row - L.num_q_heads - L.num_kv_heads) * D;
    u0 = *reinterpret_cast<const uint4*>(src + 8 * c0);
    u1 = *reinterpret_cast<const uint4*>(src + 8 * c1);
  };
  uint4 u[kBatch][2];
#pragma unroll
  for (int k = 0; k < kBatch; ++k) load((part + k * split) * kRows + sub, u[k][0], u[k][1]);

  // the first token's request is the number of requests that end at or before it
  int b = 0;
  for (int i = lane; i < L.num_reqs; i += 32) b += L.cu_seqlens[i + 1] <= t0;
  b = __reduce_add_sync(kAll, b);
  if (TOKENS > 1)
    while (b < L.num_reqs && L.cu_seqlens[b + 1] <= t) ++b;
  const int off = b < L.num_reqs ? static_cast<int>(t) - L.cu_seqlens[b] : -1;
  const int64_t slot = off < 0 ? -1 : static_cast<int64_t>(off) + (L.start ? L.start[b] : 0);
  if (slot < 0 || (L.k_cache && slot >= L.max_seqlen)) {
    if (live) cosa::report_status(L.status, cosa::kStatusBadInput);
    live = false;
  }
  size_t page_row = 0;                            // (token, kv head 0) of the bf16 caches
  bool paged = false;
  if (L.k_cache && live) {
    const int phys = L.page_table[static_cast<size_t>(b) * L.max_pages_per_req + (slot >> L.page_shift)];
    paged = phys >= 0 && phys < L.num_pages;
    page_row = ((static_cast<size_t>(max(phys, 0)) << L.page_shift) + (slot & ((1 << L.page_shift) - 1))) * L.num_kv_heads;
  }

  // The lane's eight angles, formed in 64 bits: far positions have angles of 10^5 and more, which fp32 would lose.  The rows
  // of the warp share the work: sub-row s forms angles s, s + kRows, ...
  float cs[8], sn[8];
  const int64_t pos = L.positions ? L.positions[t] : slot;
  auto angles = [&](auto in_doubles) {            // whether all of them were formed
    bool all = true;
#pragma unroll
    for (int i0 = 0; i0 < 8; i0 += kRows) {
      const int i = i0 + sub;
      const double freq = turned ? L.inv_freq[L.interleaved ? 4 * (i < 4 ? c0 : c1) + i % 4 : 8 * c0 + i] : 1.0;
      float x, s, c;
      if constexpr (decltype(in_doubles)::value) {
        x = half_turns(pos, freq);
      } else {
        all &= ordinary(freq);
        x = half_turns(pos, turn_of(freq));
      }
      sincospif(turned ? x : 0.f, &s, &c);
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        cs[i0 + k] = __shfl_sync(kAll, c, (own * kRows + k) * kLanes + l);
        sn[i0 + k] = __shfl_sync(kAll, s, (own * kRows + k) * kLanes + l);
      }
    }
    return all;
  };
  if (!__all_sync(kAll, angles(std::false_type{}))) angles(std::true_type{});

  auto finish = [&](int row, const uint4& u0, const uint4& u1) {
    const bool query = row < L.num_q_heads, value = row >= L.num_q_heads + L.num_kv_heads;
    float a[8], z[8];
    unpack8(u0, a);
    unpack8(u1, z);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(z[i], z[i], ss));
#pragma unroll
    for (int m = 1; m < kLanes; m *= 2) ss += __shfl_xor_sync(kAll, ss, m);
    if (row >= rows || !live) return;
    uint4 y0 = u0, y1 = u1;
    if (!value) {
      const uint16_t* w = query ? L.q_weight : L.k_weight;
      if (w) {
        const float inv = rsqrtf(ss * (1.0f / D) + L.eps);
        float wa[8], wz[8];
        unpack8(*reinterpret_cast<const uint4*>(w + 8 * c0), wa);
        unpack8(*reinterpret_cast<const uint4*>(w + 8 * c1), wz);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[i] = a[i] * inv * wa[i];
          z[i] = z[i] * inv * wz[i];
        }
      }
      if (turned) {
        if (L.interleaved) {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float x = a[i], y = z[i];
            a[i] = x * cs[i / 2] - a[i + 1] * sn[i / 2];
            a[i + 1] = a[i + 1] * cs[i / 2] + x * sn[i / 2];
            z[i] = y * cs[4 + i / 2] - z[i + 1] * sn[4 + i / 2];
            z[i + 1] = z[i + 1] * cs[4 + i / 2] + y * sn[4 + i / 2];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x = a[i];
            a[i] = x * cs[i] - z[i] * sn[i];
            z[i] = z[i] * cs[i] + x * sn[i];
          }
        }
      }
      y0 = pack8(a);
      y1 = pack8(z);
    }
    auto put = [&](uint16_t* dst) {
      *reinterpret_cast<uint4*>(dst + 8 * c0) = y0;
      *reinterpret_cast<uint4*>(dst + 8 * c1) = y1;
    };
    if (query) {
      put(L.q_out + (t * L.num_q_heads + row) * D);
    } else if (!value) {
      const int h = row - L.num_q_heads;
      if (L.k_out) put(L.k_out + (t * L.num_kv_heads + h) * D);
      if (paged) put(L.k_cache + (page_row + h) * D);
    } else if (paged) {
      put(L.v_cache + (page_row + row - L.num_q_heads - L.num_kv_heads) * D);
    }
  };
  for (int r0 = part * kRows; r0 < rows; r0 += kBatch * split * kRows) {    // uniform over the warp
#pragma unroll
    for (int k = 0; k < kBatch; ++k) finish(r0 + k * split * kRows + sub, u[k][0], u[k][1]);
    if (r0 + kBatch * split * kRows >= rows) break;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) load(r0 + (kBatch + k) * split * kRows + sub, u[k][0], u[k][1]);
  }
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch& L, cudaStream_t stream) {
  constexpr int64_t kWarps = 152 * 32;
  const int rows = L.num_q_heads + L.num_kv_heads + (L.k_cache ? L.num_kv_heads : 0);
  const int at_once = L.head_dim == 128 ? 4 : 8;        // rows of a warp
  // A token's heads on several warps while the tokens alone leave an SM less than eight.  40 heads of 128: 64 tokens take 4.4 us
  // instead of 9.6, 600 5.9 instead of 9.6; more parts than that (up to 32 warps an SM) make it 7.0 for the 600, 11.1
  // instead of 7.9 for 1000.
  int split = 0;       // log2
  while ((2 << split) <= rows / at_once && (static_cast<int64_t>(L.total_tokens) << split) < 152 * 8) ++split;
  // several tokens on a warp, if they fill the card so and a batch still has all of a token's rows: 3 + 1 heads of 64 for 51K
  // tokens take 25.6 us instead of 44.7 (with the angles in doubles)
  int tokens = 1;
  while (split == 0 && tokens < at_once / 2 && L.total_tokens >= 2 * tokens * kWarps &&
         rows <= at_once / (2 * tokens) * kBatch)
    tokens *= 2;
  const int64_t warps = ((static_cast<int64_t>(L.total_tokens) + tokens - 1) / tokens) << split;
  const unsigned grid = static_cast<unsigned>((warps * 32 + kThreads - 1) / kThreads);
  // Three CTAs an SM have the registers that four have to save and load; with four more loads are in flight.  With three / four: 64
  // tokens of 40 heads of 128 take 3.8 / 4.3 us, 1000 6.3 / 6.9, 4000 17.8 / 18.7, but 9.6K of 16 heads of 64 (8 CTAs an SM) 17.2 / 15.8
  // and 128K of 48 into pages 499 / 487.
  const bool few = grid <= 6 * 152;
  auto* kernel = L.head_dim == 128 ? (tokens > 1 ? rope_kernel<128, 2, 4> : few ? rope_kernel<128, 1, 3> : rope_kernel<128, 1, 4>)
                 : tokens > 1      ? (tokens == 2 ? rope_kernel<64, 2, 4> : rope_kernel<64, 4, 4>)
                                   : (few ? rope_kernel<64, 1, 3> : rope_kernel<64, 1, 4>);
  return launch_after(kernel, dim3(grid), kThreads, 0, stream, 1, L, split);
}

}  // namespace cosa_kv
