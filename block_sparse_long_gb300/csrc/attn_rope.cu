// Norm and rotation of latent attention in one pass: the latent vector of a token normed, the 64 values of its shared key
// part and of every query head rotated, the key written to its page and to rows.
//
//     c <- c / sqrt(mean(c^2) + eps) * w,     (r_a, r_b) <- (r_a cos t - r_b sin t, r_b cos t + r_a sin t)
//
// A value is read once and written once or twice, for a few operations: bound by the memory, and with few tokens by the chain of
// loads.  A warp has a token, or a part of its query heads where the tokens are few.  Its 32 lanes hold the latent vector
// in 16-byte pieces; a query head (and the key part) is on four lanes, eight heads at a time, each lane with pieces l and l + 4
// of the eight, so that both halves of every pair are in one lane in either order.  There are 32 pairs: each lane
// forms one angle and the lanes take theirs by shuffles.
// 31.1K tokens of 32 heads and 512 + 64 values: 60 us, 6.0 TB/s.
#include <cstdint>

#include "attn_internal.h"
#include "kv_angles.cuh"
#include "kv_internal.h"
#include "kv_layout.cuh"

namespace cosa_attn {
namespace {

using cosa_kv::pack8;
using cosa_kv::unpack8;

constexpr int kThreads = 256;
constexpr int kRot = COSA_ATTN_ROPE_DIM;
constexpr int kBatch = 4;      // passes of eight heads in flight
constexpr unsigned kAll = 0xffffffffu;

template <int DL>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeLaunch L, const int split_log2) {
  constexpr int kPieces = DL / 256;      // of 16 bytes of the latent vector on a lane
  const int lane = threadIdx.x % 32, l = lane % 4, sub = lane / 4;
  cosa_kv::wait_for_stream();
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / 32;
  const int last = L.cu_seqlens[L.num_reqs];
  if (blockIdx.x == 0 && threadIdx.x == 0 && (L.cu_seqlens[0] != 0 || last > L.total_tokens))
    cosa::report_status(L.status, cosa::kStatusBadInput);
  const int64_t t = unit >> split_log2;
  if (t >= min(last, L.total_tokens)) return;
  const int split = 1 << split_log2, part = static_cast<int>(unit) & (split - 1);

  const bool key = part == split - 1;             // this warp has the token's key too
  uint4 c[kPieces], r0 = make_uint4(0, 0, 0, 0), r1 = r0;
  if (key) {
    const uint16_t* src = L.kv + t * L.kv_stride;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) c[i] = *reinterpret_cast<const uint4*>(src + 8 * (lane + 32 * i));
    if (sub == 0) {
      r0 = *reinterpret_cast<const uint4*>(src + DL + 8 * l);
      r1 = *reinterpret_cast<const uint4*>(src + DL + 8 * (l + 4));
    }
  }
  const int heads = L.q ? L.num_q_heads : 0;
  uint4 u[kBatch][2];
  auto load = [&](int row, uint4& u0, uint4& u1) {
    u0 = u1 = make_uint4(0, 0, 0, 0);
    if (row >= heads) return;
    const uint16_t* src = L.q + t * L.q_stride + row * L.q_head_stride;
    u0 = *reinterpret_cast<const uint4*>(src + 8 * l);
    u1 = *reinterpret_cast<const uint4*>(src + 8 * (l + 4));
  };
#pragma unroll
  for (int k = 0; k < kBatch; ++k) load((part + k * split) * 8 + sub, u[k][0], u[k][1]);

  // the token's request is the number of requests that end at or before it
  int b = 0;
  for (int i = lane; i < L.num_reqs; i += 32) b += L.cu_seqlens[i + 1] <= t;
  b = __reduce_add_sync(kAll, b);
  const int off = b < L.num_reqs ? static_cast<int>(t) - L.cu_seqlens[b] : -1;
  const int64_t slot = off < 0 ? -1 : static_cast<int64_t>(off) + (L.start ? L.start[b] : 0);
  if (slot < 0 || (L.cache && slot >= L.max_seqlen)) {
    if (lane == 0) cosa::report_status(L.status, cosa::kStatusBadInput);
    return;
  }
  uint16_t* page_row = nullptr;
  if (L.cache && key) {
    const int phys = L.page_table[static_cast<size_t>(b) * L.max_pages_per_req + (slot >> L.page_shift)];
    if (phys >= 0 && phys < L.num_pages)
      page_row = L.cache + ((static_cast<size_t>(phys) << L.page_shift) + (slot & ((1 << L.page_shift) - 1))) * (DL + kRot);
  }

  // the lane's angle, in 64 bits (far positions lose theirs in fp32), then those of its eight pairs
  float cs[8], sn[8];
  {
    const int64_t pos = L.positions ? L.positions[t] : slot;
    const double freq = L.inv_freq[lane];
    const float x = cosa_kv::ordinary(freq) ? cosa_kv::half_turns(pos, cosa_kv::turn_of(freq)) : cosa_kv::half_turns(pos, freq);
    float s, co;
    sincospif(x, &s, &co);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int from = L.interleaved ? 4 * l + (i < 4 ? i : 12 + i) : 8 * l + i;
      cs[i] = __shfl_sync(kAll, co, from);
      sn[i] = __shfl_sync(kAll, s, from);
    }
  }
  auto turn = [&](uint4& u0, uint4& u1) {
    float a[8], z[8];
    unpack8(u0, a);
    unpack8(u1, z);
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
    u0 = pack8(a);
    u1 = pack8(z);
  };

  if (key) {
    if (L.weight) {
      float x[kPieces][8], ss = 0.f;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        unpack8(c[i], x[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[i][e], x[i][e], ss);
      }
#pragma unroll
      for (int m = 1; m < 32; m *= 2) ss += __shfl_xor_sync(kAll, ss, m);
      const float inv = rsqrtf(ss * (1.0f / DL) + L.eps);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        float w[8];
        unpack8(*reinterpret_cast<const uint4*>(L.weight + 8 * (lane + 32 * i)), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = x[i][e] * inv * w[e];
        c[i] = pack8(x[i]);
      }
    }
    turn(r0, r1);
    auto put = [&](uint16_t* to_c, uint16_t* to_r) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) *reinterpret_cast<uint4*>(to_c + 8 * (lane + 32 * i)) = c[i];
      if (sub == 0) {
        *reinterpret_cast<uint4*>(to_r + 8 * l) = r0;
        *reinterpret_cast<uint4*>(to_r + 8 * (l + 4)) = r1;
      }
    };
    if (page_row) put(page_row, page_row + DL);
    if (L.c_out) put(L.c_out + t * DL, L.k_out + t * kRot);
  }
  for (int p0 = part; p0 * 8 < heads; p0 += kBatch * split) {     // uniform over the warp
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int row = (p0 + k * split) * 8 + sub;
      if (row >= heads) continue;
      turn(u[k][0], u[k][1]);
      uint16_t* dst = L.q_out + (t * heads + row) * kRot;
      *reinterpret_cast<uint4*>(dst + 8 * l) = u[k][0];
      *reinterpret_cast<uint4*>(dst + 8 * (l + 4)) = u[k][1];
    }
    if ((p0 + kBatch * split) * 8 >= heads) break;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) load((p0 + (kBatch + k) * split) * 8 + sub, u[k][0], u[k][1]);
  }
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch& L, cudaStream_t stream) {
  // a token's heads on several warps while the tokens alone leave an SM less than eight (64 tokens of 32 heads: 4.0 us with one, 3.5)
  const int passes = L.q ? (L.num_q_heads + 7) / 8 : 0;
  int split = 0;       // log2
  while ((2 << split) <= passes + 1 && (static_cast<int64_t>(L.total_tokens) << split) < 152 * 8) ++split;
  const int64_t warps = static_cast<int64_t>(L.total_tokens) << split;
  const unsigned grid = static_cast<unsigned>((warps * 32 + kThreads - 1) / kThreads);
  return cosa_kv::launch_after(L.latent_dim == 512 ? rope_kernel<512> : rope_kernel<256>, dim3(grid), kThreads, 0, stream, 1, L, split);
}

}  // namespace cosa_attn
