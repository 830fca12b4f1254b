// Causal attention of packed prompts in the expanded form of latent attention: per head keys of d + 64 values (the last 64 shared
// by the heads) and values of d.
//
//     S = Q K^T,  P = exp2(S * scale - m),  O = sum P V,  l = sum P,  out = O / l
//
// With hundreds of queries to a key the matrix products bound it: 2 (2 d + 64) operations per visible pair.  A CTA has 128
// queries of one head and walks their keys in blocks of 128.  S is double buffered in TMEM (P goes over its S), so that the
// softmax of one block runs under the products of its neighbours.
//
// Warp roles:
//   warp 0      copies Q once, then K and V block by block (TMA).
//   warp 1      issues the products: S(j + 2) behind O(j), whose P lies in the same buffer, in one thread's order.
//   warps 2, 3  make the values of the blocks on the diagonal, whose later keys some rows must not see, finite (0 times what is not
//               finite is not 0); a row that does see such a value gets it added at the end.  Warp 3 owns the TMEM.
//   warps 4-11  softmax, a thread has half a row.  The weights are taken against the row's reference of an earlier block; only if
//               one passes 2^8 the CTA stops for its maxima, scales O and takes them again.
// CTAs start with the longest rows of all requests and go through them four heads at a time, so that the last to start are short and
// those that run together read the same keys.  Head by head / 2 / 4 / 8 / 16 heads at a time, us: 4096 tokens of 8 heads of 128
// 66 / 62 / 46 / 45 / 45, 16K of 16 1032 / 1006 / 1009 / 1022 / 1050, 8 requests of 2048 of 16 198 / 191 / 193 / 198 / 209, five ragged
// prompts of 6 heads of 64 44.5 / 39.3 / 39.4 / 39.2 / 39.1.
//
// Measured on the way, 16K tokens of 16 heads of 128 + 64: two tiles of 128 queries to a CTA with an issuing warp each 1.43 ms (they
// fell into step: both softmaxes, then both products), with one issuing warp 1.37, both tiles' O before both tiles' S 1.14 (the keys'
// slots were free for longer than a copy takes; all of TMEM and the shared memory of two tiles left no second buffer of S); one tile
// and two buffers of S 1.25 with keys and values of a block behind one barrier, 1.02 with a barrier each.  A block then takes 2050
// cycles, the products 1340 of them as they issue (1280 at the rate of the pipe by itself) and the waits between them 700.  Not
// better: Q in TMEM and a third slot for keys (1.04); P in columns of its own and an issuing warp for each product (1.02 to 1.03;
// heads of 64, 8192 tokens of 16: 242 -> 231 us, 4096 of 8 heads of 128: 65 -> 67).
//
// What bounds it now: at 16K tokens of 16 heads of 128 + 64 1.01 ms, 1.36 PFLOP/s of the pairs that are seen; 5 prompts of 37 to 2011 tokens
// of 6 heads of 64 40 us: 390 CTAs of up to 19 blocks on 152 SMs, each of which waits 3700 to 7300 cycles for its first loads.
#include <cmath>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "attn_mma.cuh"
#include "attn_tma.h"
#include "kv_internal.h"
#include "kv_layout.cuh"

namespace cosa_attn {
namespace {

using cosa::mbar_arrive;
using cosa::mbar_arrive_expect_tx;
using cosa::mbar_init;
using cosa::smem_u32;
using cosa::tc_fence_after;
using cosa::tc_fence_before;
using cosa::umma_commit;
using cosa::wait_parity_bounded;

constexpr int kThreads = 384;
constexpr int kBlock = 128;                // keys
constexpr int kRows = 128;                 // queries of a CTA
constexpr int kColumn = kBlock * 128;      // bytes of a 64-value wide column of 128 rows
constexpr int kHeads = 4;                  // heads whose blocks are taken together
constexpr int kHalf = kBlock / 2;          // keys of a thread's half row
constexpr float kNone = -3e38f;            // reference of a row that has seen nothing
constexpr uint32_t kHigh = 0x4380;         // 2^8 in bf16
constexpr float kLn2 = 0.69314718055994531f;
constexpr uint32_t kTmemS = 0, kTmemO = 256;      // two buffers of 128 columns, and the output

template <int D_>
struct Shape {
  static constexpr int D = D_;
  static constexpr int kKeyColumns = D / 64 + 1, kValueColumns = D / 64;
  static constexpr int kSlots = D == 128 ? 2 : 3;      // blocks of keys, and of values
};

template <class S>
struct alignas(1024) Smem {
  uint8_t q[S::kKeyColumns][kColumn];
  uint8_t k[S::kSlots][S::kKeyColumns][kColumn];
  uint8_t v[S::kSlots][S::kValueColumns][kColumn];
  uint64_t q_full, k_full[S::kSlots], k_empty[S::kSlots], v_full[S::kSlots], v_empty[S::kSlots];
  uint64_t v_sent[2], v_clear[2];          // of the blocks on the diagonal: copy issued, values finite
  uint64_t s_full[2], p_full[2], pv_done[2], cleanup;      // by block, even and odd: a parity tells two phases apart
  float part[2][128];                      // of a row's halves: maxima, sums
  int32_t req, block;                      // this CTA's request (-1: none) and its block of queries
  int32_t odd_values;
  uint32_t tmem_base;
  int32_t abort_flag;
};

struct Args {
  const int32_t *cu_seqlens, *cu_kv;
  const uint16_t* v;
  uint16_t* out;
  float* lse;
  int32_t* status;
  int64_t v_stride, v_head_stride;
  int num_reqs, num_heads, total_tokens, total_kv_tokens, blocks;
  float scale_log2;
  int stall;
};

struct Request {
  int tok0, n;
  int64_t from, keys;      // key rows from .. from + keys - 1
  bool bad;                // rows are out of range (n = 0), or the keys are (keys = 0)
};

__device__ __forceinline__ Request request_of(const Args& a, int b) {
  Request r;
  r.tok0 = a.cu_seqlens[b];
  const int64_t n = static_cast<int64_t>(a.cu_seqlens[b + 1]) - r.tok0;
  r.from = a.cu_kv[b];
  r.keys = a.cu_kv[b + 1] - r.from;
  r.bad = r.tok0 < 0 || n < 0 || r.tok0 + n > a.total_tokens;
  r.n = r.bad ? 0 : static_cast<int>(n);
  if (r.n > 0 && (r.from < 0 || r.keys < n || r.from + r.keys > a.total_kv_tokens)) {
    r.bad = true;
    r.keys = 0;
  }
  return r;
}

template <class S>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap qrmap, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap krmap, const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Args a) {
  constexpr int D = S::D, KC = S::kKeyColumns, VC = S::kValueColumns;
  extern __shared__ uint8_t smem_raw[];
  Smem<S>& sm = *reinterpret_cast<Smem<S>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int* abort_flag = &sm.abort_flag;
  cosa_kv::wait_for_stream();

  const int heads = min(kHeads, a.num_heads), group = blockIdx.x / (a.blocks * heads), in_group = min(heads, a.num_heads - group * heads);
  const int in = blockIdx.x - group * a.blocks * heads, head = group * heads + in % in_group;
  if (warp == 0) {
    const bool over = gave_up(a.status);
    int at = in / in_group, req = -1, block = 0;      // which of all requests' blocks
    if (a.num_reqs <= 32) {
      // by what lies before them, the longest rows first: block i of a request has about before + i blocks of keys
      const Request r = request_of(a, min(lane, a.num_reqs - 1));
      if (blockIdx.x == 0 && r.bad) cosa::report_status(a.status, cosa::kStatusBadInput);
      const int all = lane < a.num_reqs ? (r.n + kRows - 1) / kRows : 0;
      const int before = static_cast<int>(max(r.keys - r.n + kBlock - 1, static_cast<int64_t>(0)) / kBlock);
      auto from = [&](int v) { return static_cast<int>(__reduce_add_sync(kAll, static_cast<unsigned>(max(min(before + all - v, all), 0)))); };
      if (from(0) > at) {
        int v = 0;                                    // the largest with more than `at` blocks from it on
        const unsigned most = __reduce_max_sync(kAll, static_cast<unsigned>(all ? before + all : 0));
        for (int step = 1 << (31 - __clz(most)); step > 0; step /= 2)
          if (from(v + step) > at) v += step;
        at -= from(v + 1);
        const unsigned have = __ballot_sync(kAll, v >= before && v < before + all);
        req = __ffs(__ballot_sync(kAll, (have >> lane & 1) && __popc(have & ((1u << lane) - 1)) == at)) - 1;
        block = v - __shfl_sync(kAll, before, max(req, 0));
      }
    } else {
      // request by request
      for (int b0 = 0; b0 < a.num_reqs && (req < 0 || blockIdx.x == 0); b0 += 32) {
        const Request r = request_of(a, min(b0 + lane, a.num_reqs - 1));
        if (blockIdx.x == 0 && r.bad) cosa::report_status(a.status, cosa::kStatusBadInput);
        const int64_t mine = b0 + lane < a.num_reqs ? (r.n + kRows - 1) / kRows : 0;
        int64_t upto = mine;
#pragma unroll
        for (int m = 1; m < 32; m *= 2) {
          const int64_t x = __shfl_up_sync(kAll, upto, m);
          if (lane >= m) upto += x;
        }
        const unsigned past = __ballot_sync(kAll, upto > at);
        if (past && req < 0) {
          const int l = __ffs(past) - 1;
          req = b0 + l;
          block = static_cast<int>(__shfl_sync(kAll, upto, l) - 1 - at);      // the longest rows first
        }
        at = static_cast<int>(max(at - __shfl_sync(kAll, upto, 31), int64_t{-1}));
      }
    }
    if (lane == 0) {
      sm.req = over ? -1 : req;
      sm.block = block;
      if (blockIdx.x == 0 && (a.cu_seqlens[0] != 0 || a.cu_seqlens[a.num_reqs] > a.total_tokens)) cosa::report_status(a.status, cosa::kStatusBadInput);
    }
  } else if (warp == 1 && lane == 0) {
    mbar_init(&sm.q_full, 1);
    for (int s = 0; s < S::kSlots; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.v_sent[s], 1);
      mbar_init(&sm.v_clear[s], 2);
      mbar_init(&sm.s_full[s], 1);
      mbar_init(&sm.p_full[s], 8);
      mbar_init(&sm.pv_done[s], 1);
    }
    mbar_init(&sm.cleanup, 1);
    sm.abort_flag = 0;
    sm.odd_values = 0;
    cosa::fence_mbarrier_init();
  } else if (warp == 3) {
    cosa::tmem_alloc(&sm.tmem_base, 512);
    cosa::tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  if (sm.req >= 0) {
    const Request r = request_of(a, sm.req);
    const int q0 = sm.block * kRows;
    const int64_t lim0 = r.keys - r.n + q0;       // last key that the first row sees
    // blocks of keys; the first with keys that some row does not see (two blocks at most are behind it)
    const int nb = r.keys == 0 ? 0 : static_cast<int>((r.keys - r.n + min(q0 + kRows, r.n) - 1) / kBlock) + 1;
    const int diagonal = nb == 0 ? 0 : static_cast<int>((lim0 + 1) / kBlock);

    if (warp == 0) {
      // =========================== copies ===========================
      const int tok = r.tok0 + q0, key = static_cast<int>(r.from);
      Ring<S::kSlots> kring, vring;
      int keys = 0, values = 0;               // slots taken, up to the rings' sizes
      bool ok = !a.stall && nb > 0;
      if (ok && lane == 0) {
        mbar_arrive_expect_tx(&sm.q_full, KC * kColumn);
        for (int c = 0; c < VC; ++c) cosa::tma_load_4d(sm.q[c], &qmap, &sm.q_full, 0, tok, c, head);
        cosa::tma_load_4d(sm.q[VC], &qrmap, &sm.q_full, 0, tok, 0, head);
      }
      for (int j = 0; j < nb && ok; ++j) {
        if (keys == S::kSlots) ok = warp_wait(&sm.k_empty[kring.at], kring.phase ^ 1, abort_flag, a.status);
        else ++keys;
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sm.k_full[kring.at], KC * kColumn);
          for (int c = 0; c < VC; ++c) cosa::tma_load_4d(sm.k[kring.at][c], &kmap, &sm.k_full[kring.at], 0, key + j * kBlock, c, head);
          cosa::tma_load_4d(sm.k[kring.at][VC], &krmap, &sm.k_full[kring.at], 0, key + j * kBlock, 0, 0);
        }
        kring.next();
        if (values == S::kSlots) ok = warp_wait(&sm.v_empty[vring.at], vring.phase ^ 1, abort_flag, a.status);
        else ++values;
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sm.v_full[vring.at], VC * kColumn);
          for (int c = 0; c < VC; ++c) cosa::tma_load_4d(sm.v[vring.at][c], &vmap, &sm.v_full[vring.at], 0, key + j * kBlock, c, head);
          if (j >= diagonal) mbar_arrive(&sm.v_sent[j - diagonal]);
        }
        vring.next();
      }
      // every copy lands before the CTA ends: the last use of each slot; all have one wait's time together
      if (lane == 0 && !a.stall && nb > 0) {
        const uint64_t since = cosa::global_timer_ns();
        cosa::wait_until(&sm.q_full, 0, since);
        for (; keys > 0; --keys) {
          kring.back();
          cosa::wait_until(&sm.k_full[kring.at], kring.phase, since);
        }
        for (; values > 0; --values) {
          vring.back();
          cosa::wait_until(&sm.v_full[vring.at], vring.phase, since);
        }
      }
      __syncwarp();
    } else if (warp == 2 || warp == 3) {
      // =========================== values on the diagonal ===========================
      // What no row may multiply by 0: keys behind the request's, and what is not finite among those that some row does not see.  A
      // slot's barrier is waited for once its copy has been issued, so that its phase is the one meant.
      const int tid = (warp - 2) * 32 + lane;
      for (int j = diagonal; j < nb; ++j) {
        const int s = j % S::kSlots;
        if (!warp_wait(&sm.v_sent[j - diagonal], 0, abort_flag, a.status) ||
            !warp_wait(&sm.v_full[s], (j / S::kSlots) & 1, abort_flag, a.status))
          break;
        const int64_t k0 = static_cast<int64_t>(j) * kBlock;
        const int first = static_cast<int>(max(lim0 + 1 - k0, static_cast<int64_t>(0)));      // rows of the block
        const int end = static_cast<int>(min(r.keys - k0, static_cast<int64_t>(kBlock)));
        uint32_t found = 0;
        constexpr int kBatch = 8, kPieces = VC * 8;      // 16-byte pieces of a row
        auto at = [&](int e) { return reinterpret_cast<uint4*>(&sm.v[s][e % kPieces / 8][e / kPieces * 128 + (e & 7) * 16]); };
        for (int e = max(first, end) * kPieces + tid; e < kBlock * kPieces; e += 64) *at(e) = make_uint4(0, 0, 0, 0);
#pragma unroll 1
        for (int e0 = first * kPieces + tid; e0 < end * kPieces; e0 += 64 * kBatch) {
          uint4 x[kBatch];
          uint32_t bad = 0;
#pragma unroll
          for (int k = 0; k < kBatch; ++k) x[k] = e0 + 64 * k < end * kPieces ? *at(e0 + 64 * k) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int k = 0; k < kBatch; ++k) bad |= odd(x[k]);
          found |= bad;
          if (bad) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
              if (e0 + 64 * k < end * kPieces) *at(e0 + 64 * k) = finite(x[k]);
          }
        }
        cosa::fence_proxy_async_smem();
        const bool any = __any_sync(kAll, found != 0);
        if (lane == 0) {
          if (any) sm.odd_values = 1;
          mbar_arrive(&sm.v_clear[j - diagonal]);
        }
        __syncwarp();
      }
    } else if (warp == 1) {
      // =========================== products ===========================
      constexpr uint32_t idesc_s = cosa::idesc_bf16_f32(128, kBlock, false, false), idesc_o = cosa::idesc_bf16_f32(128, D, false, true);
      constexpr uint32_t hi = desc_hi(1024, 2);
      const uint32_t qd = desc_lo(smem_u32(sm.q), 16), kd = desc_lo(smem_u32(sm.k), 16), vd = desc_lo(smem_u32(sm.v), kColumn);
      Ring<S::kSlots> kring, vring;
      bool ok = nb == 0 || warp_wait(&sm.q_full, 0, abort_flag, a.status);
      auto scores = [&](int j) {
        ok = ok && warp_wait(&sm.k_full[kring.at], kring.phase, abort_flag, a.status);
        if (!ok) return;
        tc_fence_after();
        const uint32_t to = tmem + kTmemS + (j & 1) * 128, k0 = kd + kring.at * (KC * kColumn >> 4);
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < KC * 4; ++s) {
            const int at = (s / 4) * (kColumn >> 4) + (s % 4) * 2;
            mma_ss(to, qd + at, hi, k0 + at, hi, idesc_s, s > 0);
          }
          umma_commit(&sm.k_empty[kring.at]);
          umma_commit(&sm.s_full[j & 1]);
        }
        __syncwarp();
        kring.next();
      };
      for (int j = 0; j < 2 && j < nb && ok; ++j) scores(j);
      for (int j = 0; j < nb && ok; ++j, vring.next()) {
        ok = warp_wait(&sm.v_full[vring.at], vring.phase, abort_flag, a.status);
        if (j >= diagonal) ok = ok && warp_wait(&sm.v_clear[j - diagonal], 0, abort_flag, a.status);
        ok = ok && warp_wait(&sm.p_full[j & 1], (j / 2) & 1, abort_flag, a.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t p = tmem + kTmemS + (j & 1) * 128, v0 = vd + vring.at * (VC * kColumn >> 4);
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < 8; ++s) mma_ts(tmem + kTmemO, p + s / 4 * 64 + s % 4 * 8, v0 + s * (2048 >> 4), hi, idesc_o, j > 0 || s > 0);
          umma_commit(&sm.v_empty[vring.at]);
          umma_commit(&sm.pv_done[j & 1]);
        }
        __syncwarp();
        if (j + 2 < nb) scores(j + 2);
      }
      if (elect_one()) {
        umma_commit(&sm.cleanup);
        wait_parity_bounded(&sm.cleanup, 0, nullptr, nullptr);
      }
      __syncwarp();
    } else if (warp >= 4) {
      // =========================== softmax ===========================
      const int half = (warp - 4) / 4, bar = 1;
      const int t = (warp % 4) * 32 + lane, pos = q0 + t;
      const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
      const uint32_t o_at = tmem + lanes + kTmemO + half * (D / 2);
      const int64_t lim = r.keys - r.n + pos;      // last key that the row sees
      const float scale = a.scale_log2;
      float ref = kNone, l = 0.f;                  // the row's reference; the sum of this half
      bool ok = true;
      for (int j = 0; j < nb; ++j) {
        const uint32_t s_at = tmem + lanes + kTmemS + (j & 1) * 128 + half * kHalf;
        bool fail = !warp_wait(&sm.s_full[j & 1], (j / 2) & 1, abort_flag, a.status);
        const int64_t left = lim - static_cast<int64_t>(j) * kBlock - half * kHalf;
        const int last = left >= kHalf - 1 ? kHalf : static_cast<int>(max(left, static_cast<int64_t>(-1)));      // last key seen of this half
        uint32_t w[32];
        float sum, top;
        // exp2(S * scale - ref) as bf16 pairs; whether one is high
        auto weights = [&](bool for_maximum) {
          uint32_t high = 0;
          float s4[4] = {};
          top = -INFINITY;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t x[32];
            cosa::tmem_ld32(s_at + c * 32, x);
            cosa::tmem_wait_ld();
            if (last < kHalf) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (c * 32 + e > last) x[e] = 0xFF800000u;
            }
            if (for_maximum) {
#pragma unroll
              for (int e = 0; e < 32; ++e) top = fmaxf(top, __uint_as_float(x[e]));
              continue;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float x0, x1;
              cosa::fma2_bc(x0, x1, __uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]), scale, -ref);
              const float p0 = cosa::ex2_approx(x0), p1 = cosa::ex2_approx(x1);
              cosa::add2_acc(s4[(e & 1) * 2], s4[(e & 1) * 2 + 1], p0, p1);
              w[c * 16 + e] = cosa::pack_bf16x2(p0, p1);
              high = __vmaxu2(high, w[c * 16 + e]);
            }
          }
          sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
          __syncwarp();
          return (high & 0xFFFFu) > kHigh || high >> 16 > kHigh;
        };
        tc_fence_after();
        bool redo = j == 0;      // no row has a reference yet
        if (!redo) {
          const bool high = !fail && weights(false);
          redo = cosa::named_bar_red_or(bar, 256, high || fail);
        }
        if (redo) {
          if (cosa::named_bar_red_or(bar, 256, fail)) { ok = false; break; }
          // some weight is far above its row's reference (or NaN): the rows' maxima over the block, and the weights again
          weights(true);
          sm.part[half][t] = top;
          cosa::named_bar_sync(bar, 256);
          top = fmaxf(top, sm.part[half ^ 1][t]);
          const float now = top == -INFINITY ? ref : fmaxf(ref, top * scale), alpha = now == ref ? 1.f : cosa::ex2_approx(ref - now);
          ref = now;
          l *= alpha;
          weights(false);
          if (j > 0) {
            fail = !warp_wait(&sm.pv_done[(j - 1) & 1], ((j - 1) / 2) & 1, abort_flag, a.status);
            if (!fail) {
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D / 2; c += 16) {
                uint32_t o[16];
                cosa::tmem_ld16(o_at + c, o);
                cosa::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                cosa::tmem_st16(o_at + c, o);
              }
            }
          }
          cosa::named_bar_sync(bar, 256);      // the maxima have been read
        }
        if (fail) continue;      // the abort flag is set: the next wait ends too, and its vote stops the tile
        l += sum;
        cosa::tmem_st32(s_at, w);
        cosa::tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[j & 1]);
      }
      if (ok) {
        bool fail = false;
        if (nb > 0) fail = !warp_wait(&sm.pv_done[(nb - 1) & 1], ((nb - 1) / 2) & 1, abort_flag, a.status);
        sm.part[half][t] = l;
        ok = !cosa::named_bar_red_or(bar, 256, fail);
      }
      if (ok) {
        tc_fence_after();
        l += sm.part[half ^ 1][t];
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t row = static_cast<int64_t>(r.tok0 + pos) * a.num_heads + head;
        const bool live = pos < r.n;
        if (live && a.lse && half == 0) a.lse[row] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
        const bool odd_values = nb > 0 && *reinterpret_cast<volatile int*>(&sm.odd_values);
#pragma unroll
        for (int c = 0; c < D / 2; c += 16) {
          uint32_t o[16];
          __syncwarp();
          if (nb > 0) {
            cosa::tmem_ld16(o_at + c, o);
            cosa::tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = 0;
          }
          if (!live) continue;
          float f[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) f[e] = __uint_as_float(o[e]);
          if (odd_values) {
            // what was not finite among the values on the diagonal, for the rows that see it
            for (int64_t s = lim0 + 1; s <= lim; ++s) {
              const uint16_t* v = a.v + (r.from + s) * a.v_stride + head * a.v_head_stride + half * (D / 2) + c;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if ((v[e] & 0x7F80) == 0x7F80) f[e] += __uint_as_float(static_cast<uint32_t>(v[e]) << 16);
            }
          }
          uint32_t b[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) b[e] = cosa::pack_bf16x2(f[2 * e] * inv, f[2 * e + 1] * inv);
          uint4* to = reinterpret_cast<uint4*>(a.out + row * D + half * (D / 2) + c);
          to[0] = make_uint4(b[0], b[1], b[2], b[3]);
          to[1] = make_uint4(b[4], b[5], b[6], b[7]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    cosa::tmem_dealloc(tmem, 512);
  }
}

// At most so many blocks of queries: what the tokens fill and a part of one for every request.
int64_t most_blocks(int64_t total_tokens, int64_t num_reqs) { return total_tokens / kRows + num_reqs; }

template <int D>
cudaError_t launch_shape(const PrefillLaunch& L, cudaStream_t stream) {
  using S = Shape<D>;
  Args a{};
  a.cu_seqlens = L.cu_seqlens;
  a.cu_kv = L.cu_kv ? L.cu_kv : L.cu_seqlens;
  a.v = L.v;
  a.out = L.out;
  a.lse = L.lse;
  a.status = L.status;
  a.v_stride = L.v_stride;
  a.v_head_stride = L.v_head_stride;
  a.num_reqs = L.num_reqs;
  a.num_heads = L.num_heads;
  a.total_tokens = L.total_tokens;
  a.total_kv_tokens = L.total_kv_tokens;
  a.scale_log2 = L.scale_log2;
  a.stall = L.stall;
  const int64_t blocks = most_blocks(L.total_tokens, L.num_reqs);
  a.blocks = static_cast<int>(blocks);
  // rows as (64 values, token, 64-value column, head)
  CUtensorMap maps[5];
  const struct {
    const void* base;
    int64_t tokens, width, heads, stride, head_stride;
  } t[5] = {{L.q, L.total_tokens, D, L.num_heads, L.q_stride, L.q_head_stride},
            {L.q_rope, L.total_tokens, 64, L.num_heads, L.q_rope_stride, L.q_rope_head_stride},
            {L.k, L.total_kv_tokens, D, L.num_heads, L.k_stride, L.k_head_stride},
            {L.k_rope, L.total_kv_tokens, 64, 1, L.k_rope_stride, 64},
            {L.v, L.total_kv_tokens, D, L.num_heads, L.v_stride, L.v_head_stride}};
  const uint32_t box[4] = {64, 128, 1, 1};
  for (int i = 0; i < 5; ++i) {
    const uint64_t dims[4] = {64, static_cast<uint64_t>(t[i].tokens), static_cast<uint64_t>(t[i].width / 64), static_cast<uint64_t>(t[i].heads)};
    const uint64_t strides[3] = {static_cast<uint64_t>(t[i].stride) * 2, 128, static_cast<uint64_t>(t[i].head_stride) * 2};
    if (!encode_bf16(&maps[i], t[i].base, dims, strides, box)) return cudaErrorInvalidValue;
  }
  const size_t smem = sizeof(Smem<S>) + 1024;
  static_assert(sizeof(Smem<S>) + 1024 <= 227 * 1024, "shared memory");
  auto* kernel = prefill_kernel<S>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return cosa_kv::launch_after(kernel, dim3(static_cast<unsigned>(blocks * L.num_heads)), kThreads, smem, stream, 1, maps[0], maps[1], maps[2],
                               maps[3], maps[4], a);
}

}  // namespace

bool prefill_fits(int total_tokens, int num_reqs, int num_heads) { return most_blocks(total_tokens, num_reqs) * num_heads <= INT32_MAX; }

cudaError_t launch_prefill(const PrefillLaunch& L, cudaStream_t stream) {
  return L.head_dim == 128 ? launch_shape<128>(L, stream) : launch_shape<64>(L, stream);
}

}  // namespace cosa_attn
