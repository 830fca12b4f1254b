// Attention of the newest tokens of each request over the paged 4-bit cache.
//
// Per (request, kv head) the rows are the request's query tokens times the Hq / Hkv query heads of the
// kv head, eight or sixteen of them at a time:  o = softmax(scale q K^T) V with K = c_k s_k, V = c_v s_v.
// Both products run on mma.sync m16n8k16 with bf16 operands and fp32 sums:
//   q K^T   A = q (exact), B = the codes of 8 tokens; the codes of one scale group (32 values = two
//           products) are summed apart and then multiplied by the token's scale in fp32;
//   p V     A = V^T codes (16 values of the head by 16 tokens), B = p * s per scale group in bf16.
// A code of magnitude m becomes the subnormal bf16 number +-m 2^-129 (three bits of significand and the sign
// bit where the layout has them), two codes by a shift and an AND; matrix instructions take subnormal
// operands exactly.  The other operands carry 2^96 to keep the products normal: q is multiplied by it, and
// the exponent of p is raised by 96.  What is left, 2^-33, goes into the softmax scale and the last division.
//
// What bounds it: 9 d / 8 bytes of cache per token and kv head (144 at d = 128, K and V) against HBM; close
// behind, the issue slots that unpack the codes.  So a warp works alone on tiles of 16 tokens out of its own
// ring in shared memory, and nothing is shared between warps until the end of the CTA's part of a request.
//
// The work is the list of all (request, kv head, row tile, 16-token tile); every CTA takes an equal
// run of it, whatever the lengths are.  A CTA that has all of a (request, kv head, row tile) writes its
// output; otherwise it leaves its maximum, sum and unnormalised output in the workspace (a CTA has at
// most two unfinished ones, the first and the last of its run) and kv4_combine_kernel joins them in order.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "cosa_kv.h"
#include "kv_internal.h"
#include "kv_layout.cuh"

namespace cosa_kv {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 4;        // tiles in flight per warp
constexpr int kMaxCtas = 304;     // two per SM; one with sixteen rows to a tile, which take twice the registers
constexpr int kMinTiles = 8;      // tiles per CTA at least: one per warp

// What a CTA leaves about the unfinished (request, kv head, row tile) that begins in its run.
struct Owner {
  int b, h, rt;     // b < 0: none
  int last;         // last CTA that has a part of it
};

struct Args {
  AttnLaunch L;
  Owner* owner;       // [kMaxCtas]
  float* part_ml;     // [kMaxCtas][2][16][2]
  float* part_o;      // [kMaxCtas][2][16][d]
  float* stats;       // [Hkv][T * g][2]: maximum (scaled) and sum of a row, with weights only
  float* logits;      // [Hkv][T * g][pitch]: logits as the first product leaves them, with weights only
  int64_t pitch;
  int group;          // Hq / Hkv
  int page_shift;     // log2(P)
};

struct Request {
  int tok0, n, len;   // first row of q, query tokens, cache length
  int64_t tiles, rts; // 16-token tiles (one at least, to write an empty request's zeros), row tiles
};

__device__ __forceinline__ Request request_of(const Args& a, int b, int rows, bool tell) {
  Request r;
  r.tok0 = a.L.cu_seqlens[b];
  r.n = a.L.cu_seqlens[b + 1] - r.tok0;
  r.len = a.L.kv_len[b];
  if (r.tok0 < 0 || r.n < 0 || static_cast<int64_t>(r.tok0) + r.n > a.L.total_tokens || r.len < 0 || r.len > a.L.max_seqlen) {
    if (tell) cosa::report_status(a.L.status, cosa::kStatusBadInput);
    r.n = r.len = 0;
  }
  r.tiles = max(1, (r.len + kTile - 1) / kTile);
  r.rts = (static_cast<int64_t>(r.n) * a.group + rows - 1) / rows;
  return r;
}

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int m = 16; m > 0; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// All units of the batch (whole warp).
__device__ __forceinline__ int64_t total_units(const Args& a, int rows, bool tell) {
  int64_t u = 0;
  for (int b = threadIdx.x % 32; b < a.L.num_reqs; b += 32) {
    const Request r = request_of(a, b, rows, tell);
    u += r.tiles * r.rts * a.L.num_kv_heads;
  }
  return warp_sum(u);
}

// Request that holds unit `at`, and the unit at which it begins (whole warp).
__device__ __forceinline__ int find_request(const Args& a, int rows, int64_t at, int64_t& begin) {
  const int lane = threadIdx.x % 32;
  int64_t base = 0;
  for (int b0 = 0; b0 < a.L.num_reqs; b0 += 32) {
    int64_t u = 0;
    if (b0 + lane < a.L.num_reqs) {
      const Request r = request_of(a, b0 + lane, rows, false);
      u = r.tiles * r.rts * a.L.num_kv_heads;
    }
    int64_t end = u;
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
      const int64_t v = __shfl_up_sync(0xffffffffu, end, m);
      if (lane >= m) end += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, base + end > at);
    if (past) {
      const int first = __ffs(past) - 1;
      begin = base + __shfl_sync(0xffffffffu, end - u, first);
      return b0 + first;
    }
    base += __shfl_sync(0xffffffffu, end, 31);
  }
  begin = base;
  return a.L.num_reqs;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Nibbles P of both halves of a word as bf16 pairs; `swapped` is the word with the bytes of each half exchanged,
// which brings nibbles 2 and 3, and the signs of theirs, to where nibbles 0 and 1 and theirs were.
__device__ __forceinline__ uint32_t swap_bytes(uint32_t w) { return __byte_perm(w, 0, 0x2301); }
template <int P>
__device__ __forceinline__ uint32_t codes(uint32_t w, uint32_t swapped) {
  const uint32_t x = P < 2 ? w : swapped;
  return (P % 2 ? x : x << 4) & 0x80708070u;
}

constexpr float kUp = 79228162514264337593543950336.0f;      // 2^96
constexpr float kDown = 8589934592.0f;                       // 2^33

template <int D, int NT>
struct AttnSmem {
  static constexpr int kRows = 8 * NT;
  alignas(16) uint8_t ring[kWarps][kStages][Tile<D>::kBytes];
  alignas(16) float o[kWarps][kRows][D];
  float ml[kWarps][kRows][2];
};

// Rows of a warp's accumulators: lane = 4 i + c.  In q K^T a lane holds rows i (and i + 8) and tokens
// 2c, 2c + 1 of each 8-token half; in p V it holds rows 2c, 2c + 1 (of each 8-row half) and of every scale
// group g the values 32 g + 4 i .. + 3.
template <int D, int NT, bool WEIGHTS>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) attention_kernel(const Args a) {
  using T = Tile<D>;
  constexpr int G = T::G;
  constexpr int kRows = 8 * NT;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  AttnSmem<D, NT>& sm = *reinterpret_cast<AttnSmem<D, NT>*>(smem_raw);
  const AttnLaunch& L = a.L;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, i = lane / 4, c = lane % 4;

  const int64_t units = total_units(a, kRows, blockIdx.x == 0 && warp == 0);
  const int64_t ctas = min(static_cast<int64_t>(gridDim.x), max(static_cast<int64_t>(1), units / kMinTiles));
  const int64_t me = blockIdx.x;
  Owner own{-1, 0, 0, 0};
  if (me >= ctas || units == 0) {
    if (tid == 0) a.owner[me] = own;
    return;
  }
  const int64_t lo = units * me / ctas, hi = units * (me + 1) / ctas;
  int64_t at = lo, req_begin;
  int b = find_request(a, kRows, at, req_begin);

  while (at < hi) {
    const Request r = request_of(a, b, kRows, false);
    const int64_t req_units = r.tiles * r.rts * L.num_kv_heads;
    if (at >= req_begin + req_units) {     // the next request that has units
      req_begin += req_units;
      ++b;
      continue;
    }
    const int64_t item = (at - req_begin) / r.tiles;          // (kv head, row tile)
    const int h = static_cast<int>(item / r.rts), rt = static_cast<int>(item % r.rts);
    const int64_t item_begin = req_begin + item * r.tiles, item_end = item_begin + r.tiles;
    const int t_begin = static_cast<int>(at - item_begin);
    const int t_end = static_cast<int>(min(hi, item_end) - item_begin);
    const int nrows = static_cast<int>(min(static_cast<int64_t>(kRows), static_cast<int64_t>(r.n) * a.group - static_cast<int64_t>(rt) * kRows));

    // ---- this lane's rows of q: A operands ----
    uint32_t qa[NT][2 * G][2];        // [row half][product][k half]
    int limit[NT];                    // slots that the row sees
    int all_see = r.len;              // slots that every row sees
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      const int row = rt * kRows + 8 * x + i;
      const bool in = 8 * x + i < nrows;
      const int tok = in ? row / a.group : 0, head = in ? row - tok * a.group : 0;
      limit[x] = in ? max(0, r.len - r.n + tok + 1) : 0;
      if (in) all_see = min(all_see, limit[x]);
      const uint16_t* src = L.q + ((static_cast<int64_t>(r.tok0) + tok) * L.num_q_heads + h * a.group + head) * D + 8 * c;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (in) u = *reinterpret_cast<const uint4*>(src + 32 * g);
        float v[8];
        unpack8(u, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= kUp;
        // values e and e + 4 meet in a pair of codes
        qa[x][2 * g][0] = cosa::pack_bf16x2(v[0], v[4]);
        qa[x][2 * g][1] = cosa::pack_bf16x2(v[1], v[5]);
        qa[x][2 * g + 1][0] = cosa::pack_bf16x2(v[2], v[6]);
        qa[x][2 * g + 1][1] = cosa::pack_bf16x2(v[3], v[7]);
      }
    }
#pragma unroll
    for (int m = 4; m < 32; m *= 2) all_see = min(all_see, __shfl_xor_sync(0xffffffffu, all_see, m));

    float o[NT][2 * G][4];            // [row half][m tile]
    float m2[NT], l[NT];              // running maximum (scaled, base 2) and this lane's part of the sum
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      m2[x] = -INFINITY;
      l[x] = 0.f;
#pragma unroll
      for (int mt = 0; mt < 2 * G; ++mt)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[x][mt][k] = 0.f;
    }

    // ---- the warp's tiles: t_begin + warp, + 8, ... ----
    const int32_t* table = L.page_table + static_cast<size_t>(b) * L.max_pages_per_req;
    uint32_t there = 0;               // per stage: the tile's page exists
    auto page_at = [&](int t) -> int {
      if (t >= t_end || t * kTile >= r.len) return -1;
      const int phys = table[(t * kTile) >> a.page_shift];
      return phys < L.num_kv4_pages ? phys : -1;
    };
    const uint8_t* head = L.cache + (static_cast<size_t>(h) << (a.page_shift - 4)) * T::kBytes + lane * 16;
    const size_t page_bytes = (static_cast<size_t>(L.num_kv_heads) << (a.page_shift - 4)) * T::kBytes;
    const int tile_mask = (1 << (a.page_shift - 4)) - 1;
    auto issue = [&](int t, int stage, int phys) {
      if (phys >= 0) {
        const uint8_t* src = head + phys * page_bytes + (t & tile_mask) * T::kBytes;
        const uint32_t dst = cosa::smem_u32(sm.ring[warp][stage]) + lane * 16;
#pragma unroll
        for (int k = 0; k < (T::kBytes + 511) / 512; ++k)
          if (k < T::kBytes / 512 || lane * 16 < T::kBytes % 512) copy16(dst + k * 512, src + k * 512);
        there |= 1u << stage;
      } else {
        there &= ~(1u << stage);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int s = 0; s < kStages; ++s) {
      const int t = t_begin + warp + s * kWarps;
      issue(t, s, page_at(t));
    }
    int stage = 0;
    int next_phys = page_at(t_begin + warp + kStages * kWarps);
    for (int t = t_begin + warp; t < t_end; t += kWarps) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();
      const uint8_t* tile = sm.ring[warp][stage];
      const bool exists = (there >> stage) & 1u;
      const int slot0 = t * kTile;
      const bool clear = exists && slot0 + kTile <= all_see;   // every row sees every token of the tile

      // q K^T: logits of 16 tokens
      float s[2][4];                  // [8-token half][row i: 2c, 2c + 1; row i + 8: 2c, 2c + 1]
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t kw[G], sc[G];        // sc: scales of tokens 2c and 2c + 1, two groups to a word
        if constexpr (G == 4) {
          const uint4 u = *reinterpret_cast<const uint4*>(tile + (8 * j + i) * T::kRow + 16 * c);
          kw[0] = u.x; kw[1] = u.y; kw[2] = u.z; kw[3] = u.w;
          const uint4 v = *reinterpret_cast<const uint4*>(tile + T::kKScales + (8 * j + 2 * c) * G * 2);
          sc[0] = v.x; sc[1] = v.y; sc[2] = v.z; sc[3] = v.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(tile + (8 * j + i) * T::kRow + 8 * c);
          kw[0] = u.x; kw[1] = u.y;
          const uint2 v = *reinterpret_cast<const uint2*>(tile + T::kKScales + (8 * j + 2 * c) * G * 2);
          sc[0] = v.x; sc[1] = v.y;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) s[j][k] = 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const uint32_t w = kw[g], z = swap_bytes(w);
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
          mma_bf16(acc, qa[0][2 * g][0], NT == 2 ? qa[NT - 1][2 * g][0] : 0u, qa[0][2 * g][1],
                   NT == 2 ? qa[NT - 1][2 * g][1] : 0u, codes<0>(w, z), codes<1>(w, z));
          mma_bf16(acc, qa[0][2 * g + 1][0], NT == 2 ? qa[NT - 1][2 * g + 1][0] : 0u, qa[0][2 * g + 1][1],
                   NT == 2 ? qa[NT - 1][2 * g + 1][1] : 0u, codes<2>(w, z), codes<3>(w, z));
          const float s0 = g % 2 ? bf16_hi(sc[g / 2]) : bf16_lo(sc[g / 2]);
          const float s1 = g % 2 ? bf16_hi(sc[G / 2 + g / 2]) : bf16_lo(sc[G / 2 + g / 2]);
          s[j][0] = fmaf(acc[0], s0, s[j][0]);
          s[j][1] = fmaf(acc[1], s1, s[j][1]);
          if (NT == 2) {
            s[j][2] = fmaf(acc[2], s0, s[j][2]);
            s[j][3] = fmaf(acc[3], s1, s[j][3]);
          }
        }
      }
      uint32_t seen = 0xFFu;          // bit 4 x + 2 j + e: row half x sees token 8 j + 2 c + e
      if (!clear) {
        seen = 0;
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (exists && slot0 + 8 * j + 2 * c + e < limit[x])
                seen |= 1u << (4 * x + 2 * j + e);
              else
                s[j][2 * x + e] = -INFINITY;
            }
      }
      if (WEIGHTS) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
          if (8 * x + i < nrows) {
            const int64_t row = (static_cast<int64_t>(h) * L.total_tokens + r.tok0) * a.group + rt * kRows + 8 * x + i;
#pragma unroll
            for (int j = 0; j < 2; ++j)
              *reinterpret_cast<float2*>(a.logits + row * a.pitch + slot0 + 8 * j + 2 * c) = make_float2(s[j][2 * x], s[j][2 * x + 1]);
          }
      }

      // running maximum; the sums so far are rescaled where it grows
      float p[NT][4];                 // [row half][2 j + e]
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        float mx = fmaxf(fmaxf(s[0][2 * x], s[0][2 * x + 1]), fmaxf(s[1][2 * x], s[1][2 * x + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * L.scale_log2;
        if (__any_sync(0xffffffffu, mx > m2[x])) {
          const float m_new = fmaxf(m2[x], mx);
          const float f = m2[x] == -INFINITY ? 0.f : cosa::ex2_approx(m2[x] - m_new);
          m2[x] = m_new;
          l[x] *= f;
          // rows 2c and 2c + 1 of the output accumulators live in the lanes whose i is that row
          const float f0 = __shfl_sync(0xffffffffu, f, 8 * c), f1 = __shfl_sync(0xffffffffu, f, 8 * c + 4);
#pragma unroll
          for (int mt = 0; mt < 2 * G; ++mt) {
            o[x][mt][0] *= f0; o[x][mt][1] *= f1; o[x][mt][2] *= f0; o[x][mt][3] *= f1;
          }
        }
        const float up = 96.f - (m2[x] == -INFINITY ? 0.f : m2[x]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          p[x][k] = cosa::ex2_approx(fmaf(s[k / 2][2 * x + k % 2], L.scale_log2, up));
          l[x] += p[x][k];
        }
      }

      // p V
      uint32_t vs[2][G];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if constexpr (G == 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(tile + T::kVScales + (8 * j + 2 * c) * G * 2);
          vs[j][0] = v.x; vs[j][1] = v.y; vs[j][2] = v.z; vs[j][3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(tile + T::kVScales + (8 * j + 2 * c) * G * 2);
          vs[j][0] = v.x; vs[j][1] = v.y;
        }
      }
      uint32_t vw[4][G / 2];          // tokens 2c, 2c + 1, 8 + 2c, 9 + 2c: rows c, 8 + c, 4 + c, 12 + c
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint8_t* src = tile + T::kVCodes + (c + 8 * (k % 2) + 4 * (k / 2)) * T::kRow + i * (2 * G);
        if constexpr (G == 4) {
          const uint2 u = *reinterpret_cast<const uint2*>(src);
          vw[k][0] = u.x; vw[k][1] = u.y;
        } else {
          vw[k][0] = *reinterpret_cast<const uint32_t*>(src);
        }
      }
      auto product = [&](auto all) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          uint32_t pb[NT][2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float s0 = g % 2 ? bf16_hi(vs[j][g / 2]) : bf16_lo(vs[j][g / 2]);
            const float s1 = g % 2 ? bf16_hi(vs[j][G / 2 + g / 2]) : bf16_lo(vs[j][G / 2 + g / 2]);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
              float y0 = p[x][2 * j] * s0, y1 = p[x][2 * j + 1] * s1;
              if constexpr (!decltype(all)::value) {      // an unseen token adds nothing, whatever its scale is
                if (!((seen >> (4 * x + 2 * j)) & 1u)) y0 = 0.f;
                if (!((seen >> (4 * x + 2 * j + 1)) & 1u)) y1 = 0.f;
              }
              pb[x][j] = cosa::pack_bf16x2(y0, y1);
            }
          }
          // the group's codes of both tokens of a pair, and the same with the bytes exchanged
          const uint32_t sel = g % 2 ? 0x7632 : 0x5410, swp = g % 2 ? 0x6723 : 0x4501;
          const uint32_t w0 = __byte_perm(vw[0][g / 2], vw[1][g / 2], sel), z0 = __byte_perm(vw[0][g / 2], vw[1][g / 2], swp);
          const uint32_t w1 = __byte_perm(vw[2][g / 2], vw[3][g / 2], sel), z1 = __byte_perm(vw[2][g / 2], vw[3][g / 2], swp);
#pragma unroll
          for (int x = 0; x < NT; ++x) {
            mma_bf16(o[x][2 * g], codes<0>(w0, z0), codes<1>(w0, z0), codes<0>(w1, z1), codes<1>(w1, z1), pb[x][0], pb[x][1]);
            mma_bf16(o[x][2 * g + 1], codes<2>(w0, z0), codes<3>(w0, z0), codes<2>(w1, z1), codes<3>(w1, z1), pb[x][0], pb[x][1]);
          }
        }
      };
      if (clear)
        product(std::true_type{});
      else
        product(std::false_type{});

      __syncwarp();                   // every lane has read the stage
      issue(t + kStages * kWarps, stage, next_phys);
      next_phys = page_at(t + (kStages + 1) * kWarps);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // ---- join the warps ----
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      if (c == 0) {
        sm.ml[warp][8 * x + i][0] = m2[x];
        sm.ml[warp][8 * x + i][1] = l[x];
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        // m tile 2g: values +0 (first half) and +1, m tile 2g + 1: +2 and +3
        *reinterpret_cast<float4*>(&sm.o[warp][8 * x + 2 * c][32 * g + 4 * i]) =
            make_float4(o[x][2 * g][0], o[x][2 * g][2], o[x][2 * g + 1][0], o[x][2 * g + 1][2]);
        *reinterpret_cast<float4*>(&sm.o[warp][8 * x + 2 * c + 1][32 * g + 4 * i]) =
            make_float4(o[x][2 * g][1], o[x][2 * g][3], o[x][2 * g + 1][1], o[x][2 * g + 1][3]);
      }
    }
    __syncthreads();
    const bool whole = t_begin == 0 && t_end == r.tiles;
    const int slot_of_part = t_begin == 0 ? 1 : 0;
    for (int k = tid; k < nrows * (D / 4); k += kThreads) {
      const int row = k / (D / 4), d0 = 4 * (k % (D / 4));
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.ml[w][row][0]);
      float sum = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = sm.ml[w][row][0];
        // a warp that saw nothing has sums of zero, or of NaN where a logit was NaN: then so is its factor's product
        const float f = mw == -INFINITY ? 1.f : cosa::ex2_approx(mw - M);
        sum = fmaf(f, sm.ml[w][row][1], sum);
        const float4 u = *reinterpret_cast<const float4*>(&sm.o[w][row][d0]);
        v.x = fmaf(f, u.x, v.x); v.y = fmaf(f, u.y, v.y); v.z = fmaf(f, u.z, v.z); v.w = fmaf(f, u.w, v.w);
      }
      if (whole) {
        const int rr = rt * kRows + row;
        const int tok = rr / a.group, head = rr - tok * a.group;
        const float inv = sum == 0.f ? 0.f : kDown / (sum * (1.0f / kUp));
        uint16_t* dst = L.out + ((static_cast<int64_t>(r.tok0) + tok) * L.num_q_heads + h * a.group + head) * D + d0;
        *reinterpret_cast<uint2*>(dst) = make_uint2(cosa::pack_bf16x2(v.x * inv, v.y * inv), cosa::pack_bf16x2(v.z * inv, v.w * inv));
        if (WEIGHTS && d0 == 0) {
          float* st = a.stats + ((static_cast<int64_t>(h) * L.total_tokens + r.tok0) * a.group + rr) * 2;
          st[0] = M;
          st[1] = sum * (1.0f / kUp);
        }
      } else {
        const size_t at_part = (static_cast<size_t>(me) * 2 + slot_of_part) * 16 + row;
        *reinterpret_cast<float4*>(a.part_o + at_part * D + d0) = v;
        if (d0 == 0) {
          a.part_ml[at_part * 2] = M;
          a.part_ml[at_part * 2 + 1] = sum;
        }
      }
    }
    if (!whole && t_begin == 0) {
      // the CTA that has the item's last unit
      int64_t j = (item_end - 1) * ctas / units;
      while (units * (j + 1) / ctas <= item_end - 1) ++j;
      while (units * j / ctas > item_end - 1) --j;
      own = Owner{b, h, rt, static_cast<int>(j)};
    }
    __syncthreads();
    at = item_begin + t_end;
  }
  if (tid == 0) a.owner[me] = own;
}

// Joins the parts of the items that no CTA had whole: block (x, row) goes through the owner CTAs x, x + gridDim.x, ...
// The parts' maxima and sums are read at once, then their outputs, eight in flight per thread.
template <int D, int NT, bool WEIGHTS>
__global__ void __launch_bounds__(D) combine_kernel(const Args a, const int ctas) {
  constexpr int kRows = 8 * NT;
  __shared__ float s_factor[kMaxCtas];
  __shared__ float s_red[2][D / 32];
  const int d = threadIdx.x, warp = d / 32, lane = d % 32;
  for (int first = blockIdx.x; first < ctas; first += gridDim.x) {
    const Owner own = a.owner[first];
    if (own.b < 0) continue;
    const Request r = request_of(a, own.b, kRows, false);
    const int row = own.rt * kRows + static_cast<int>(blockIdx.y);
    if (row >= static_cast<int64_t>(r.n) * a.group) continue;
    // part j: the second place of the owner, the first of every later CTA
    auto place = [&](int j) { return (static_cast<size_t>(first + j) * 2 + (j == 0 ? 1 : 0)) * 16 + blockIdx.y; };
    const int parts = own.last - first + 1;
    float M = -INFINITY;
    for (int j = d; j < parts; j += D) M = fmaxf(M, a.part_ml[place(j) * 2]);
#pragma unroll
    for (int m = 16; m > 0; m /= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
    if (lane == 0) s_red[0][warp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < D / 32; ++w) M = fmaxf(M, s_red[0][w]);
    float sum = 0.f;
    for (int j = d; j < parts; j += D) {
      const float m = a.part_ml[place(j) * 2];
      const float f = m == -INFINITY ? 1.f : cosa::ex2_approx(m - M);     // nothing seen: sums of zero, or NaN
      s_factor[j] = f;
      sum = fmaf(f, a.part_ml[place(j) * 2 + 1], sum);
    }
#pragma unroll
    for (int m = 16; m > 0; m /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (lane == 0) s_red[1][warp] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < D / 32; ++w) sum += s_red[1][w];
    float v = 0.f;
#pragma unroll 8
    for (int j = 0; j < parts; ++j) v = fmaf(s_factor[j], a.part_o[place(j) * D + d], v);
    const int tok = row / a.group, head = row - tok * a.group;
    const float y = sum == 0.f ? 0.f : v * (kDown / (sum * (1.0f / kUp)));
    a.L.out[((static_cast<int64_t>(r.tok0) + tok) * a.L.num_q_heads + own.h * a.group + head) * D + d] =
        static_cast<uint16_t>(cosa::pack_bf16x2(y, y));
    if (WEIGHTS && d == 0) {
      float* st = a.stats + ((static_cast<int64_t>(own.h) * a.L.total_tokens + r.tok0) * a.group + row) * 2;
      st[0] = M;
      st[1] = sum * (1.0f / kUp);
    }
    __syncthreads();
  }
}

// weights[b, h, s] += sum over the rows of exp2(scale * logit - M) / sum, rows in order; four slots per thread.
constexpr int kWeightRows = 32;       // rows whose maxima and sums a CTA holds at a time
__global__ void __launch_bounds__(256) weights_kernel(const Args a, const int rows_per_tile) {
  __shared__ float2 s_stat[kWeightRows];
  const int b = blockIdx.z, h = blockIdx.y;
  const Request r = request_of(a, b, rows_per_tile, false);
  const int slot = (static_cast<int>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (static_cast<int>(blockIdx.x) * 1024 >= r.len || r.n == 0) return;
  const bool in = slot < r.len;
  const int64_t row0 = (static_cast<int64_t>(h) * a.L.total_tokens + r.tok0) * a.group;
  const int64_t rows = static_cast<int64_t>(r.n) * a.group;
  float w[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t i0 = 0; i0 < rows; i0 += kWeightRows) {
    const int n = static_cast<int>(min(static_cast<int64_t>(kWeightRows), rows - i0));    // unseen slots have -inf
    __syncthreads();
    if (threadIdx.x < n) {
      const float2 st = *reinterpret_cast<const float2*>(a.stats + (row0 + i0 + threadIdx.x) * 2);
      s_stat[threadIdx.x] = make_float2(-st.x, 1.0f / st.y);
    }
    __syncthreads();
    if (!in) continue;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float2 st = s_stat[i];
      const float4 s = *reinterpret_cast<const float4*>(a.logits + (row0 + i0 + i) * a.pitch + slot);
      w[0] += s.x == -INFINITY ? 0.f : cosa::ex2_approx(fmaf(s.x, a.L.scale_log2, st.x)) * st.y;
      w[1] += s.y == -INFINITY ? 0.f : cosa::ex2_approx(fmaf(s.y, a.L.scale_log2, st.x)) * st.y;
      w[2] += s.z == -INFINITY ? 0.f : cosa::ex2_approx(fmaf(s.z, a.L.scale_log2, st.x)) * st.y;
      w[3] += s.w == -INFINITY ? 0.f : cosa::ex2_approx(fmaf(s.w, a.L.scale_log2, st.x)) * st.y;
    }
  }
  if (!in) return;
  float* dst = a.L.weights + (static_cast<int64_t>(b) * a.L.num_kv_heads + h) * a.L.max_seqlen + slot;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (slot + k < r.len) dst[k] += w[k];
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

template <int D, int NT, bool WEIGHTS>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  constexpr size_t smem = sizeof(AttnSmem<D, NT>);
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  auto* kernel = attention_kernel<D, NT, WEIGHTS>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  constexpr int kCtas = kMaxCtas / NT;
  kernel<<<kCtas, kThreads, smem, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  combine_kernel<D, NT, WEIGHTS><<<dim3(std::min(kCtas, 64), 8 * NT), D, 0, stream>>>(a, kCtas);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (WEIGHTS) {
    const dim3 grid(static_cast<unsigned>((a.L.max_seqlen + 1023LL) / 1024), static_cast<unsigned>(a.L.num_kv_heads),
                    static_cast<unsigned>(a.L.num_reqs));
    weights_kernel<<<grid, 256, 0, stream>>>(a, 8 * NT);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace

size_t attn_workspace_bytes(int num_q_heads, int head_dim, int total_tokens, int max_seqlen, bool with_weights) {
  size_t n = align256(kMaxCtas * sizeof(Owner)) + align256(size_t(kMaxCtas) * 2 * 16 * 2 * 4) +
             align256(size_t(kMaxCtas) * 2 * 16 * head_dim * 4);
  if (with_weights) {
    const size_t rows = static_cast<size_t>(total_tokens) * num_q_heads;
    const size_t pitch = (static_cast<size_t>(max_seqlen) + kTile - 1) / kTile * kTile;
    n += align256(rows * 8) + align256(rows * pitch * 4);
  }
  return n;
}

cudaError_t launch_attention(const AttnLaunch& L, cudaStream_t stream) {
  Args a{};
  a.L = L;
  a.L.scale_log2 = L.scale_log2 * kDown;      // of the logits as the first product leaves them
  a.group = L.num_q_heads / L.num_kv_heads;
  for (a.page_shift = 4; (1 << a.page_shift) < L.page_size;) ++a.page_shift;
  a.pitch = (static_cast<int64_t>(L.max_seqlen) + kTile - 1) / kTile * kTile;
  uint8_t* w = static_cast<uint8_t*>(L.workspace);
  a.owner = reinterpret_cast<Owner*>(w);
  w += align256(kMaxCtas * sizeof(Owner));
  a.part_ml = reinterpret_cast<float*>(w);
  w += align256(size_t(kMaxCtas) * 2 * 16 * 2 * 4);
  a.part_o = reinterpret_cast<float*>(w);
  w += align256(size_t(kMaxCtas) * 2 * 16 * L.head_dim * 4);
  if (L.weights) {
    a.stats = reinterpret_cast<float*>(w);
    w += align256(static_cast<size_t>(L.total_tokens) * L.num_q_heads * 8);
    a.logits = reinterpret_cast<float*>(w);
  }
  const bool wide = static_cast<int64_t>(L.max_new_tokens) * a.group > 8;
  const bool d128 = L.head_dim == 128;
  if (L.weights) {
    if (d128) return wide ? launch<128, 2, true>(a, stream) : launch<128, 1, true>(a, stream);
    return wide ? launch<64, 2, true>(a, stream) : launch<64, 1, true>(a, stream);
  }
  if (d128) return wide ? launch<128, 2, false>(a, stream) : launch<128, 1, false>(a, stream);
  return wide ? launch<64, 2, false>(a, stream) : launch<64, 1, false>(a, stream);
}

}  // namespace cosa_kv
