// Attention of the newest tokens of each request over the paged 4-bit cache.
//
// Per (request, kv head) the rows are the request's query tokens times the Hq / Hkv query heads of the
// kv head, eight, sixteen or twenty-four of them at a time:  o = softmax(scale q K^T) V with K = c_k s_k, V = c_v s_v.
// Both products run on mma.sync m16n8k16 with bf16 operands and fp32 sums, the tokens or the head's values as the
// sixteen rows and the query rows as the eight columns, so that no part of an instruction is empty for eight rows:
//   K q^T   A = the codes of 16 tokens, B = q (exact); the codes of one scale group (32 values = two products) are
//           summed apart and then multiplied by the token's scale in fp32;
//   V^T p   A = the codes of 16 values of the head by 16 tokens, B = p * s per scale group in bf16, turned from the
//           first product's layout (tokens down) to the second's (tokens across) by movmatrix.
// A code of magnitude m becomes the subnormal bf16 number +-m 2^-129 (three bits of significand and the sign
// bit where the layout has them), two codes by a shift and an AND; matrix instructions take subnormal
// operands exactly.  The other operands, q and p * s, carry 2^96 to keep the products normal; what is
// left, 2^-33, goes into the softmax scale and the last division.
//
// The one rounding to fewer bits than fp32: p * s becomes a bf16 operand.  It is off by 2^-8 of a term at most and by much less
// in their sum: outputs are 1.7e-3 to 1.8e-3 from a 64-bit form, where their own rounding to bf16 alone makes 1.6e-3 to 1.7e-3.
// A second operand with what is cut off would double the second product and the turns of its layout, eight more of each, and
// takes about 40 other instructions beside the 320 per 16 tokens, for an error that the output's rounding hides.  The accumulated weights are
// formed from fp32 logits and take no part in it.
//
// Work: 9/8 d bytes of cache per token and kv head (144 at d = 128) and 4 d operations per row.  A warp works alone on
// units of 16 or 32 tokens, one bulk copy each, out of its own ring in shared memory, and nothing is shared between
// warps until the end of the CTA's part of a request.  No unit of the card is full: over a context of 131072 tokens the issue slots
// are 55 % busy (320 instructions of a warp per 16 tokens at d = 128, most of them unpacking), the ALU pipe 48 %, the memory 54 %,
// the matrix pipe 22 %.  It streams at 5.6 TB/s; what is lost are the first loads, the CTAs' uneven ends and the join.
//
// Two ways to share the work.  As one list of all (request, kv head, row tile, unit), of which every CTA takes an equal run
// whatever the lengths are (with an allowance for the ends of its pieces): a CTA that has all of a (request, kv head, row
// tile) writes its output, otherwise it leaves its maximum, sum and unnormalised output in the workspace (a CTA has at most
// two unfinished ones, the first and the last of its run) and a second kernel joins them in order.  Or, where warps have
// few tokens, a cluster to each (request, kv head, row tile), whose CTAs join their parts through distributed shared memory.
//
// Measured (32 query and 8 kv heads of 128, one new token): one context of 131072 tokens, 37 us, 151 MB at 4.0 TB/s (59 % of the
// measured copy rate, 27 us of it streaming);
// one of 777 tokens, 5.8 us; 48 ragged contexts (417K tokens), two new tokens and weights, 125 us, of which the weights'
// logits (107 MB written and read) take about 35.  Heads of 64: 27 us and 5.3 us.  A row tile streams and unpacks the cache for
// itself: 8 contexts of 16K (151 MB) take 58, 60, 93 and 170 us with 12, 16, 32 and 64 rows.

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include <cooperative_groups.h>

#include "cosa_kv.h"
#include "kv_internal.h"
#include "kv_layout.cuh"

namespace cosa_kv {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kSms = 152;
constexpr int kMaxCtas = 3 * kSms;
constexpr int kMaxRows = 24;     // query rows of a row tile: 8, 16 or 24
// Units per CTA at least (with kPiece), where an item is shared between CTAs.  A context of 1500 tokens and 8 kv heads, one of
// 6000, three of 3000 with 2 kv heads: with 2 units 10.9, 12.4 and 10.1 us, with 4 10.2, 10.9 and 10.6, with 8 11.3, 12.1
// and 11.8.
constexpr int kMinUnits = 4;
// Units of an average item up to which one CTA takes it alone: 16 contexts of 200 tokens in tables for 32K, 7.7 us instead of
// 11.4 (with none); with 32 units nothing changes for those, and 8 contexts of 250 tokens take 10.8 us instead of 10.7.
constexpr int kWholeUnits = 8;
// What the beginning and the end of a CTA's part of an item cost, in units: a CTA whose run crosses into a next item has so many
// fewer.  With none, 4 and 12: a context of 128K 38.5, 37.5 and 37.1 us, 48 ragged ones with weights 127.9, 126.8 and 123.1 us,
// one of 1500 tokens 12.3, 11.3 and 10.2 us.
constexpr int kPiece = 12;
constexpr int kMaxCluster = 16;  // CTAs of a cluster
// Tokens per warp up to which items go to clusters.  No list of the batch to make before the first load and no second kernel
// after the last: a context of 777 tokens takes 5.8 us instead of 11.4, 7 x 14K with 2 kv heads 17.5 instead of 18.7, 15 x 6K
// 14.3 instead of 21.6; but shares are even only within an item and the clusters may fill the card badly: one of 32K takes
// 23.8 us instead of 19.0.
constexpr int kClusterTokens = 256;
// Items up to which the join has a block per row: a context of 128K takes 45.1 us so, 55.4 with a warp per row, 48 ragged ones
// 153.3 and 135.5.
constexpr int kFewItems = 64;

// What a CTA leaves about the unfinished (request, kv head, row tile) that begins in its run.
struct Owner {
  int rows;         // query rows of the tile; 0: none
  int last;         // last CTA that has a part of it
  int tok0, h, rt;  // first row of q of the request, kv head, row tile
};

struct Args {
  AttnLaunch L;
  Owner* owner;       // [kMaxCtas]
  float* part_ml;     // [kMaxCtas][2][kMaxRows][2]
  float* part_o;      // [kMaxCtas][2][kMaxRows][d]
  float* stats;       // [Hkv][T * g][2]: maximum (scaled) and sum of a row, with weights only
  float* logits;      // [Hkv][T * g][pitch]: logits as the first product leaves them, with weights only
  int64_t pitch;
  int group;          // Hq / Hkv
  int page_shift;     // log2(P)
  bool stall;         // test hook: no copy is issued
  int row_tiles;      // row tiles of a request, as far as max_new_tokens tells
};

struct Request {
  int tok0, n, len;   // first row of q, query tokens, cache length
  int64_t units, rts; // units of tokens (one at least, to write an empty request's zeros), row tiles
};

// `rows`: query rows of a row tile, `tokens`: of a unit.
__device__ __forceinline__ Request request_of(const Args& a, int b, int rows, int tokens, bool tell) {
  Request r;
  r.tok0 = a.L.cu_seqlens[b];
  r.n = a.L.cu_seqlens[b + 1] - r.tok0;
  r.len = a.L.kv_len[b];
  if (r.tok0 < 0 || r.n < 0 || static_cast<int64_t>(r.tok0) + r.n > a.L.total_tokens || r.len < 0 || r.len > a.L.max_seqlen) {
    if (tell) cosa::report_status(a.L.status, cosa::kStatusBadInput);
    r.n = r.len = 0;
  }
  r.units = max(1, (r.len + tokens - 1) / tokens);
  r.rts = (static_cast<int64_t>(r.n) * a.group + rows - 1) / rows;
  return r;
}

// A quotient of numbers that are not negative, with the 32-bit division where it is enough (a fifth of the 64-bit one's
// time, and there are several in a row before a CTA's first load).
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}

// The units of the batch, kPiece added to every item's, in even shares: the first `more` CTAs have one more than `each`.
struct Shares {
  int64_t units, items, each, more;
  int ctas;
  __device__ __forceinline__ int64_t begin(int64_t cta) const { return cta * each + min(cta, more); }
  __device__ __forceinline__ int owner(int64_t unit) const {
    const int64_t big = more * (each + 1);
    return static_cast<int>(unit < big ? quotient(unit, each + 1) : more + quotient(unit - big, each));
  }
};

// This lane's request of the 32 from b0, its units, and their sum up to and with it (whole warp).
struct LaneUnits {
  int64_t own, end, items;
};
__device__ __forceinline__ LaneUnits lane_units(const Args& a, int rows, int tokens, int b0, bool tell) {
  const int lane = threadIdx.x % 32;
  LaneUnits u{0, 0, 0};
  if (b0 + lane < a.L.num_reqs) {
    const Request r = request_of(a, b0 + lane, rows, tokens, tell);
    u.items = r.rts * a.L.num_kv_heads;
    u.own = (r.units + kPiece) * u.items;
  }
  u.end = u.own;
#pragma unroll
  for (int m = 1; m < 32; m *= 2) {
    const int64_t v = __shfl_up_sync(0xffffffffu, u.end, m);
    if (lane >= m) u.end += v;
  }
  return u;
}

// The batch's shares (whole warp).  `first`: what the lanes have of the first 32 requests, for find_request.
__device__ __forceinline__ Shares shares_of(const Args& a, int rows, int tokens, int grid, bool tell, LaneUnits& first) {
  Shares s{0, 0, 0, 0, 0};
  for (int b0 = 0; b0 < a.L.num_reqs; b0 += 32) {
    const LaneUnits u = lane_units(a, rows, tokens, b0, tell);
    if (b0 == 0) first = u;
    s.units += __shfl_sync(0xffffffffu, u.end, 31);
    int64_t n = u.items;
#pragma unroll
    for (int m = 16; m > 0; m /= 2) n += __shfl_xor_sync(0xffffffffu, n, m);
    s.items += n;
  }
  // Short contexts stay whole: with up to kWholeUnits units in the average item, a CTA takes at least one item, and few
  // parts are left to join.
  const int64_t fit = s.units <= (kWholeUnits + kPiece) * s.items ? s.items : max(s.items, quotient(s.units, kMinUnits));
  s.ctas = static_cast<int>(max(static_cast<int64_t>(1), min(static_cast<int64_t>(grid), fit)));
  s.each = quotient(s.units, s.ctas);
  s.more = s.units - s.each * s.ctas;
  return s;
}

// Request that holds unit `at`, and the unit at which it begins (whole warp; `at` is below the batch's units).
__device__ __forceinline__ int find_request(const Args& a, int rows, int tokens, int64_t at, const LaneUnits& first, int64_t& begin) {
  int64_t base = 0;
  for (int b0 = 0; b0 < a.L.num_reqs; b0 += 32) {
    const LaneUnits u = b0 == 0 ? first : lane_units(a, rows, tokens, b0, false);
    const unsigned past = __ballot_sync(0xffffffffu, base + u.end > at);
    if (past) {
      const int lane = __ffs(past) - 1;
      begin = base + __shfl_sync(0xffffffffu, u.end - u.own, lane);
      return b0 + lane;
    }
    base += __shfl_sync(0xffffffffu, u.end, 31);
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

// The same with a sum that begins at zero.
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// `bytes` neighbouring bytes into shared memory (both ends 16-byte aligned), counted by a barrier of this CTA.
__device__ __forceinline__ void copy_bulk(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
                   cosa::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(cosa::smem_u32(bar)), "l"(policy)
               : "memory");
}

// Cache policy for bytes that a call reads once: they make room in L2 first (the logits, which are read again, stay).
__device__ __forceinline__ uint64_t read_once() {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}

// Nibbles P of both halves of a word as bf16 pairs; `swapped` is the word with the bytes of each half exchanged,
// which brings nibbles 2 and 3, and the signs of theirs, to where nibbles 0 and 1 and theirs were.
__device__ __forceinline__ uint32_t swap_bytes(uint32_t w) { return __byte_perm(w, 0, 0x2301); }
template <int P>
__device__ __forceinline__ uint32_t codes(uint32_t w, uint32_t swapped) {
  const uint32_t x = P < 2 ? w : swapped;
  return (P % 2 ? x : x << 4) & 0x80708070u;
}

// An 8 x 8 matrix of 16-bit values, a row in four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

constexpr float kUp = 79228162514264337593543950336.0f;      // 2^96
constexpr float kDown = 8589934592.0f;                       // 2^33

// A unit is TP tiles that a warp takes at a time: with eight and sixteen rows two, whose chains of dependent instructions fill
// each other's gaps; with more rows one, for the registers.  (Eight rows, one 128K context with TP = 1, 2, 4: 49, 39 and 38 us;
// 48 ragged ones with weights: 149, 130 and 134 us; a context of 777 tokens: 12, 11.5 and 14.5 us.  Sixteen rows, 8 contexts
// of 16K: with TP = 1 on two and on three CTAs an SM 70 and 77 us, with TP = 2 on two 59.)
template <int NT>
struct Steps {
  static constexpr int TP = NT <= 2 ? 2 : 1;
  static constexpr int kStages = NT <= 2 ? 2 : 4;        // units in flight per warp
  static constexpr int kCtas = NT == 1 ? 3 : 2;          // CTAs of an SM: 168 or 255 registers a thread
  static constexpr int kResident = kCtas * kSms;
};

// A warp's part of the output before the join lies where its units were.
template <int D, int NT>
struct AttnSmem {
  static constexpr int kRows = 8 * NT, TP = Steps<NT>::TP;
  union Ring {
    uint8_t unit[Steps<NT>::kStages][TP * Tile<D>::kBytes];
    float o[kRows][D];
  };
  alignas(16) Ring ring[kWarps];
  float ml[kWarps][kRows][2];
  alignas(8) float joined[kRows][2];
  alignas(8) uint64_t full[kWarps][Steps<NT>::kStages];
};

// A warp's accumulators: lane = 4 i + c has query rows 2c and 2c + 1 of each eight; of the logits the tokens i and i + 8,
// of the output the values 32 g + 4 i .. + 3 of every scale group g.
//
// CLUSTERED: a cluster has one (request, kv head, row tile) at a time, its CTAs even shares of the units, and joins its parts
// through distributed shared memory.  Else every CTA has a run of the whole list, and a second kernel joins the parts.
template <int D, int NT, bool WEIGHTS, bool CLUSTERED>
__global__ void __launch_bounds__(kThreads, Steps<NT>::kCtas) attention_kernel(const Args a) {
  using T = Tile<D>;
  constexpr int G = T::G;
  constexpr int kRows = 8 * NT;
  constexpr int TP = Steps<NT>::TP, kStages = Steps<NT>::kStages, kUnit = TP * kTile;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  auto& sm = *reinterpret_cast<AttnSmem<D, NT>*>(smem_raw);
  const AttnLaunch& L = a.L;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, i = lane / 4, c = lane % 4;

  wait_for_stream();
  let_next_start();
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < kStages; ++k) cosa::mbar_init(&sm.full[warp][k], 1);
    cosa::fence_mbarrier_init();
    cosa::fence_proxy_async_smem();
  }
  __syncwarp();
  uint32_t phase = 0;               // bit k: parity of the next completion of stage k's barrier
  bool alive = true;                // no wait of this warp has run out
  const uint64_t once = read_once();

  const int me = static_cast<int>(blockIdx.x);
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = CLUSTERED ? static_cast<int>(cluster.num_blocks()) : 1;
  const int rank = CLUSTERED ? static_cast<int>(cluster.block_rank()) : 0;
  Request r;                        // the request at hand
  int b, h, rt;                     // and the kv head and row tile
  int t_begin, t_end;               // this CTA's units of it
  Shares sh;
  int64_t hi = 0, at = 0, req_begin = 0, item_end = 0;
  Owner own{0, 0, 0, 0, 0};
  if (CLUSTERED) {
    const int item = me / ctas;
    rt = item % a.row_tiles;
    h = item / a.row_tiles % L.num_kv_heads;
    b = item / a.row_tiles / L.num_kv_heads;
    r = request_of(a, b, kRows, kUnit, rank == 0 && h == 0 && rt == 0 && tid == 0);
    if (me == 0 && tid == 0 && r.tok0 != 0) cosa::report_status(L.status, cosa::kStatusBadInput);
    t_begin = static_cast<int>(r.units * rank / ctas);
    t_end = static_cast<int>(r.units * (rank + 1) / ctas);
  } else {
    LaneUnits first;
    if (me == 0 && tid == 0 && L.cu_seqlens[0] != 0) cosa::report_status(L.status, cosa::kStatusBadInput);
    sh = shares_of(a, kRows, kUnit, static_cast<int>(gridDim.x), blockIdx.x == 0 && warp == 0, first);
    if (me >= sh.ctas || sh.units == 0) {
      if (tid == 0) a.owner[me] = own;
      return;
    }
    hi = sh.begin(me + 1);
    at = sh.begin(me);
    b = find_request(a, kRows, kUnit, at, first, req_begin);
  }

  for (;;) {
    if (CLUSTERED) {
      if (rt >= r.rts) break;        // the same in the whole cluster
    } else {
      if (at >= hi) break;
      r = request_of(a, b, kRows, kUnit, false);
      const int64_t item_units = r.units + kPiece, req_units = item_units * r.rts * L.num_kv_heads;
      if (at >= req_begin + req_units) {     // the next request that has units
        req_begin += req_units;
        ++b;
        continue;
      }
      const int64_t item = quotient(at - req_begin, item_units);   // (kv head, row tile)
      h = static_cast<int>(quotient(item, r.rts));
      rt = static_cast<int>(item - h * r.rts);
      const int64_t item_begin = req_begin + item * item_units;
      item_end = item_begin + r.units;
      t_begin = static_cast<int>(at - item_begin);
      t_end = static_cast<int>(min(hi, item_end) - item_begin);
      at = item_end + kPiece;
      if (t_begin >= r.units) continue;
    }
    const int nrows = static_cast<int>(
        min(static_cast<int64_t>(kRows), static_cast<int64_t>(r.n) * a.group - static_cast<int64_t>(rt) * kRows));

    // ---- the warp's units: t_begin + warp, + kWarps, ... ----
    const int32_t* table = L.page_table + static_cast<size_t>(b) * L.max_pages_per_req;
    uint32_t there = 0;               // bit stage * TP + u: the page of the stage's tile u exists
    const bool copies = lane == 0 && !a.stall;
    int phys[TP];                     // pages of the tiles of the unit that is asked for next
    const bool one_page = kUnit <= (1 << a.page_shift);
    const int page_tiles = 1 << (a.page_shift - 4);
    auto look_up = [&](int t) {
#pragma unroll
      for (int u = 0; u < TP; ++u) {
        if (u > 0 && (one_page || (u & (page_tiles - 1)))) {
          phys[u] = phys[u - 1];
          continue;
        }
        const int slot = t * kUnit + u * kTile;
        phys[u] = -1;
        if (t < t_end && slot < r.len) {
          const int page = table[slot >> a.page_shift];
          if (page < L.num_kv4_pages) phys[u] = page;
        }
      }
    };
    const uint8_t* head = L.cache + (static_cast<size_t>(h) << (a.page_shift - 4)) * T::kBytes;
    const uint32_t page_bytes = (static_cast<uint32_t>(L.num_kv_heads) << (a.page_shift - 4)) * T::kBytes;   // below 2^31
    // one copy per page that the unit lies on, all counted by the stage's barrier
    auto issue = [&](int t, int stage) {
      if (t >= t_end || !alive) return;
#pragma unroll
      for (int u = 0; u < TP; ++u) {
        const uint32_t bit = 1u << (stage * TP + u);
        there = phys[u] >= 0 ? there | bit : there & ~bit;
      }
      if (copies) {
        uint64_t* bar = &sm.full[warp][stage];
        uint8_t* dst = sm.ring[warp].unit[stage];
        auto page = [&](int u) { return head + static_cast<uint64_t>(static_cast<uint32_t>(phys[u])) * page_bytes; };
        if (one_page) {
          cosa::mbar_arrive_expect_tx(bar, phys[0] >= 0 ? TP * T::kBytes : 0);
          if (phys[0] >= 0) copy_bulk(dst, page(0) + (t * TP & (page_tiles - 1)) * T::kBytes, TP * T::kBytes, bar, once);
        } else {
          int tiles = 0;
#pragma unroll
          for (int u = 0; u < TP; ++u) tiles += phys[u] >= 0;
          cosa::mbar_arrive_expect_tx(bar, tiles * T::kBytes);
#pragma unroll
          for (int u = 0; u < TP; ++u)
            if (phys[u] >= 0 && (u & (page_tiles - 1)) == 0)
              copy_bulk(dst + u * T::kBytes, page(u), page_tiles * T::kBytes, bar, once);
        }
      }
    };
    const int t_first = t_begin + warp;
#pragma unroll
    for (int s = 0; s < kStages; ++s) {
      look_up(t_first + s * kWarps);
      issue(t_first + s * kWarps, s);
    }
    look_up(t_first + kStages * kWarps);

    // ---- this lane's row of q: B operands ----
    uint32_t qb[NT][2 * G][2];        // row 8 x + i: [eight rows][product][k half]
    int limit[NT][2];                 // slots that rows 8 x + 2c and + 1 see
    int all_see = r.len;              // slots that every row sees
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      const int row = rt * kRows + 8 * x + i;
      const bool in = 8 * x + i < nrows;
      const int tok = in ? row / a.group : 0, head = in ? row - tok * a.group : 0;
      const int sees = in ? max(0, r.len - r.n + tok + 1) : 0;
      if (in) all_see = min(all_see, sees);
      limit[x][0] = __shfl_sync(0xffffffffu, sees, 8 * c);
      limit[x][1] = __shfl_sync(0xffffffffu, sees, 8 * c + 4);
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
        qb[x][2 * g][0] = cosa::pack_bf16x2(v[0], v[4]);
        qb[x][2 * g][1] = cosa::pack_bf16x2(v[1], v[5]);
        qb[x][2 * g + 1][0] = cosa::pack_bf16x2(v[2], v[6]);
        qb[x][2 * g + 1][1] = cosa::pack_bf16x2(v[3], v[7]);
      }
    }
#pragma unroll
    for (int m = 4; m < 32; m *= 2) all_see = min(all_see, __shfl_xor_sync(0xffffffffu, all_see, m));

    const int clear_units = all_see / kUnit;
    float o[NT][2 * G][4];            // [eight rows][m tile]
    // rows 8 x + 2c and + 1: running maximum (unscaled), minus the scaled one (0 for none), this lane's part of the sum
    float top[NT][2], off[NT][2], l[NT][2];
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      top[x][0] = top[x][1] = -INFINITY;
      off[x][0] = off[x][1] = 0.f;
      l[x][0] = l[x][1] = 0.f;
#pragma unroll
      for (int mt = 0; mt < 2 * G; ++mt)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[x][mt][k] = 0.f;
    }

    int stage = 0;
    for (int t = t_first; alive && t < t_end; t += kWarps) {
      if (!cosa::wait_parity_bounded(&sm.full[warp][stage], (phase >> stage) & 1u, nullptr, L.status)) {
        // The copies in flight have one more budget together to land before the CTA's memory is anyone else's; what follows is
        // undefined.  The stage j places ahead has unit t + j kWarps; no copy was made for it if none of its pages exists.
        const uint64_t since = cosa::global_timer_ns();
        for (int j = 0; j < kStages; ++j) {
          const int k = (stage + j) % kStages;
          if (!a.stall && t + j * kWarps < t_end && ((there >> (k * TP)) & ((1u << TP) - 1u)))
            cosa::wait_until(&sm.full[warp][k], (phase >> k) & 1u, since);
        }
        alive = false;
      }
      alive = __all_sync(0xffffffffu, alive);
      if (!alive) break;
      phase ^= 1u << stage;
      const uint8_t* tiles = sm.ring[warp].unit[stage];
      const uint32_t exists = there >> (stage * TP);           // bit u
      // every row sees every token of the unit
      const bool clear = (exists & ((1u << TP) - 1u)) == (1u << TP) - 1u && t < clear_units;

      // K q^T: logits of 16 TP tokens
      float s[TP][NT][4];             // [tile][eight rows][token i: rows 2c, 2c + 1; token i + 8: rows 2c, 2c + 1]
#pragma unroll
      for (int u = 0; u < TP; ++u) {
        const uint8_t* tile = tiles + u * T::kBytes;
        uint32_t kw[2][G], sc[2][G / 2];      // tokens i and i + 8: codes, and scales two groups to a word
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if constexpr (G == 4) {
            const uint4 w = *reinterpret_cast<const uint4*>(tile + (8 * j + i) * T::kRow + 16 * c);
            kw[j][0] = w.x; kw[j][1] = w.y; kw[j][2] = w.z; kw[j][3] = w.w;
            const uint2 v = *reinterpret_cast<const uint2*>(tile + T::kKScales + (8 * j + i) * G * 2);
            sc[j][0] = v.x; sc[j][1] = v.y;
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(tile + (8 * j + i) * T::kRow + 8 * c);
            kw[j][0] = w.x; kw[j][1] = w.y;
            sc[j][0] = *reinterpret_cast<const uint32_t*>(tile + T::kKScales + (8 * j + i) * G * 2);
          }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const uint32_t w0 = kw[0][g], z0 = swap_bytes(w0), w1 = kw[1][g], z1 = swap_bytes(w1);
          const uint32_t a0 = codes<0>(w0, z0), a1 = codes<0>(w1, z1), a2 = codes<1>(w0, z0), a3 = codes<1>(w1, z1);
          const uint32_t e0 = codes<2>(w0, z0), e1 = codes<2>(w1, z1), e2 = codes<3>(w0, z0), e3 = codes<3>(w1, z1);
          const float s0 = g % 2 ? bf16_hi(sc[0][g / 2]) : bf16_lo(sc[0][g / 2]);
          const float s1 = g % 2 ? bf16_hi(sc[1][g / 2]) : bf16_lo(sc[1][g / 2]);
#pragma unroll
          for (int x = 0; x < NT; ++x) {
            float acc[4];
            mma_bf16_first(acc, a0, a1, a2, a3, qb[x][2 * g][0], qb[x][2 * g][1]);
            mma_bf16(acc, e0, e1, e2, e3, qb[x][2 * g + 1][0], qb[x][2 * g + 1][1]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float sk = k < 2 ? s0 : s1;
              s[u][x][k] = g == 0 ? acc[k] * sk : fmaf(acc[k], sk, s[u][x][k]);
            }
          }
        }
      }
      // bit 4 (NT u + x) + k: the row of s[u][x][k] sees its token
      uint32_t seen = ~0u;
      if (!clear) {
        seen = 0;
#pragma unroll
        for (int u = 0; u < TP; ++u)
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (((exists >> u) & 1u) && t * kUnit + u * kTile + i + 8 * (k / 2) < limit[x][k % 2])
                seen |= 1u << (4 * (NT * u + x) + k);
              else
                s[u][x][k] = -INFINITY;
            }
      }
      if (WEIGHTS) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (8 * x + 2 * c + e < nrows) {
              const int64_t row = (static_cast<int64_t>(h) * L.total_tokens + r.tok0) * a.group + rt * kRows + 8 * x + 2 * c + e;
              float* dst = a.logits + row * a.pitch + t * kUnit + i;
#pragma unroll
              for (int u = 0; u < TP; ++u) {
                dst[16 * u] = s[u][x][e];
                dst[16 * u + 8] = s[u][x][2 + e];
              }
            }
      }

      // Running maximum.  The lanes of a row agree on it, so whether any of them has a larger logit is one vote; only
      // then is the maximum found and are the sums so far rescaled.
      float mx[NT][2];
      bool grows = false;
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[x][e] = fmaxf(s[0][x][e], s[0][x][2 + e]);
#pragma unroll
          for (int u = 1; u < TP; ++u) mx[x][e] = fmaxf(mx[x][e], fmaxf(s[u][x][e], s[u][x][2 + e]));
          grows |= mx[x][e] > top[x][e];
        }
      if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = mx[x][e];
#pragma unroll
            for (int k = 4; k < 32; k *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
            m = fmaxf(top[x][e], m);
            const float now = m == -INFINITY ? 0.f : -m * L.scale_log2;
            f[e] = top[x][e] == -INFINITY ? 0.f : cosa::ex2_approx(now - off[x][e]);
            top[x][e] = m;
            off[x][e] = now;
            l[x][e] *= f[e];
          }
#pragma unroll
          for (int mt = 0; mt < 2 * G; ++mt) {
            o[x][mt][0] *= f[0]; o[x][mt][1] *= f[1]; o[x][mt][2] *= f[0]; o[x][mt][3] *= f[1];
          }
        }
      }
      float p[TP][NT][4];
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int u = 0; u < TP; ++u)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float e = cosa::ex2_approx(fmaf(s[u][x][k], L.scale_log2, off[x][k % 2]));
            l[x][k % 2] += e;
            p[u][x][k] = e * kUp;
          }

      // V^T p
      auto product = [&](auto all) {
#pragma unroll
        for (int u = 0; u < TP; ++u) {
          const uint8_t* tile = tiles + u * T::kBytes;
          uint32_t sc[2][G / 2];      // tokens i and i + 8
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if constexpr (G == 4) {
              const uint2 v = *reinterpret_cast<const uint2*>(tile + T::kVScales + (8 * j + i) * G * 2);
              sc[j][0] = v.x; sc[j][1] = v.y;
            } else {
              sc[j][0] = *reinterpret_cast<const uint32_t*>(tile + T::kVScales + (8 * j + i) * G * 2);
            }
          }
          uint32_t vw[4][G / 2];      // tokens 2c, 2c + 1, 8 + 2c, 9 + 2c: rows c, 8 + c, 4 + c, 12 + c
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint8_t* src = tile + T::kVCodes + (c + 8 * (k % 2) + 4 * (k / 2)) * T::kRow + i * (2 * G);
            if constexpr (G == 4) {
              const uint2 w = *reinterpret_cast<const uint2*>(src);
              vw[k][0] = w.x; vw[k][1] = w.y;
            } else {
              vw[k][0] = *reinterpret_cast<const uint32_t*>(src);
            }
          }
#pragma unroll
          for (int g = 0; g < G; ++g) {
            uint32_t pb[NT][2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float sj = g % 2 ? bf16_hi(sc[j][g / 2]) : bf16_lo(sc[j][g / 2]);
#pragma unroll
              for (int x = 0; x < NT; ++x) {
                float y0 = p[u][x][2 * j] * sj, y1 = p[u][x][2 * j + 1] * sj;
                if constexpr (!decltype(all)::value) {      // an unseen token adds nothing, whatever its scale is
                  if (!((seen >> (4 * (NT * u + x) + 2 * j)) & 1u)) y0 = 0.f;
                  if (!((seen >> (4 * (NT * u + x) + 2 * j + 1)) & 1u)) y1 = 0.f;
                }
                pb[x][j] = transpose8(cosa::pack_bf16x2(y0, y1));
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
        }
      };
      if (clear)
        product(std::true_type{});
      else
        product(std::false_type{});

      __syncwarp();                   // every lane has read the stage
      issue(t + kStages * kWarps, stage);
      look_up(t + (kStages + 1) * kWarps);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }

    // ---- join the warps ----
#pragma unroll
    for (int x = 0; x < NT; ++x) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int m = 4; m < 32; m *= 2) l[x][e] += __shfl_xor_sync(0xffffffffu, l[x][e], m);
        if (i == 0) {
          sm.ml[warp][8 * x + 2 * c + e][0] = top[x][e] == -INFINITY ? -INFINITY : -off[x][e];
          sm.ml[warp][8 * x + 2 * c + e][1] = l[x][e];
        }
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        // m tile 2g: values +0 (first half) and +1, m tile 2g + 1: +2 and +3
        *reinterpret_cast<float4*>(&sm.ring[warp].o[8 * x + 2 * c][32 * g + 4 * i]) =
            make_float4(o[x][2 * g][0], o[x][2 * g][2], o[x][2 * g + 1][0], o[x][2 * g + 1][2]);
        *reinterpret_cast<float4*>(&sm.ring[warp].o[8 * x + 2 * c + 1][32 * g + 4 * i]) =
            make_float4(o[x][2 * g][1], o[x][2 * g][3], o[x][2 * g + 1][1], o[x][2 * g + 1][3]);
      }
    }
    // a warp whose wait ran out ends the others' work too: their next waits would come one after the other
    alive = __syncthreads_and(alive);
    // four values of a row whose maximum is M: the output, and what the weights need
    auto finish = [&](int row, int d0, float M, float sum, const float4& v) {
      const int rr = rt * kRows + row;
      const int tok = rr / a.group, head = rr - tok * a.group;
      const float inv = sum == 0.f ? 0.f : kDown / sum;
      uint16_t* dst = L.out + ((static_cast<int64_t>(r.tok0) + tok) * L.num_q_heads + h * a.group + head) * D + d0;
      *reinterpret_cast<uint2*>(dst) = make_uint2(cosa::pack_bf16x2(v.x * inv, v.y * inv), cosa::pack_bf16x2(v.z * inv, v.w * inv));
      if (WEIGHTS && d0 == 0) {
        float* st = a.stats + ((static_cast<int64_t>(h) * L.total_tokens + r.tok0) * a.group + rr) * 2;
        st[0] = M;
        st[1] = sum;
      }
    };
    const bool whole = CLUSTERED ? ctas == 1 : t_begin == 0 && t_end == r.units;
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
        const float4 u = *reinterpret_cast<const float4*>(&sm.ring[w].o[row][d0]);
        v.x = fmaf(f, u.x, v.x); v.y = fmaf(f, u.y, v.y); v.z = fmaf(f, u.z, v.z); v.w = fmaf(f, u.w, v.w);
      }
      if (whole) {
        finish(row, d0, M, sum, v);
      } else if (CLUSTERED) {
        *reinterpret_cast<float4*>(&sm.ring[0].o[row][d0]) = v;      // which only this thread has read
        if (d0 == 0) {
          sm.joined[row][0] = M;
          sm.joined[row][1] = sum;
        }
      } else {
        const size_t at_part = (static_cast<size_t>(me) * 2 + (t_begin == 0 ? 1 : 0)) * kMaxRows + row;
        *reinterpret_cast<float4*>(a.part_o + at_part * D + d0) = v;
        if (d0 == 0) {
          a.part_ml[at_part * 2] = M;
          a.part_ml[at_part * 2 + 1] = sum;
        }
      }
    }
    if (CLUSTERED && !whole) {
      cluster.sync();
      for (int k = rank * kThreads + tid; k < nrows * (D / 4); k += ctas * kThreads) {
        const int row = k / (D / 4), d0 = 4 * (k % (D / 4));
        float M = -INFINITY, sum = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int j = 0; j < ctas; ++j) M = fmaxf(M, *cluster.map_shared_rank(&sm.joined[row][0], j));
#pragma unroll 4
        for (int j = 0; j < ctas; ++j) {
          const float2 ml = *reinterpret_cast<const float2*>(cluster.map_shared_rank(&sm.joined[row][0], j));
          const float4 u = *reinterpret_cast<const float4*>(cluster.map_shared_rank(&sm.ring[0].o[row][d0], j));
          const float f = ml.x == -INFINITY ? 1.f : cosa::ex2_approx(ml.x - M);
          sum = fmaf(f, ml.y, sum);
          v.x = fmaf(f, u.x, v.x); v.y = fmaf(f, u.y, v.y); v.z = fmaf(f, u.z, v.z); v.w = fmaf(f, u.w, v.w);
        }
        finish(row, d0, M, sum, v);
      }
      cosa::fence_proxy_async_smem();
      cluster.sync();                  // the cluster's memory has been read
    } else {
      if (!CLUSTERED && !whole && t_begin == 0) own = Owner{nrows, sh.owner(item_end - 1), r.tok0, h, rt};
      cosa::fence_proxy_async_smem();  // the rings are free for copies again
      __syncthreads();
    }
    if (CLUSTERED) rt += a.row_tiles;
  }
  if (!CLUSTERED && tid == 0) a.owner[me] = own;
}

// Joins the parts of the items that no CTA had whole, for few items of many parts.  Block (x, y) goes through the owner
// CTAs x, x + gridDim.x, ..., and through rows y, y + gridDim.y, ... of theirs.  A thread has four values of the row and
// every kJoin-th part, all of which are asked for before the first is needed.
constexpr int kJoinThreads = 256;
template <int D, bool WEIGHTS>
__global__ void __launch_bounds__(kJoinThreads) combine_wide_kernel(const Args a, const int ctas, const int tile_rows) {
  constexpr int kLanes = D / 4, kJoin = kJoinThreads / kLanes, kDeep = 8;
  constexpr int kWarpsHere = kJoinThreads / 32;
  __shared__ float s_factor[kMaxCtas];
  __shared__ float s_red[2][kWarpsHere];
  __shared__ float4 s_o[kJoin][kLanes];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, d4 = tid % kLanes, part0 = tid / kLanes;
  wait_for_stream();
  let_next_start();
  for (int first = blockIdx.x; first < ctas; first += gridDim.x) {
    const Owner own = a.owner[first];
    for (int row = blockIdx.y; row < own.rows; row += gridDim.y) {
      // part j: the second place of the owner, the first of every later CTA
      auto place = [&](int j) { return (static_cast<size_t>(first + j) * 2 + (j == 0 ? 1 : 0)) * kMaxRows + row; };
      const int parts = own.last - first + 1;
      float4 o[kDeep];
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        const int j = part0 + k * kJoin;
        o[k] = j < parts ? *reinterpret_cast<const float4*>(a.part_o + place(j) * D + 4 * d4) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float M = -INFINITY;
      for (int j = tid; j < parts; j += kJoinThreads) M = fmaxf(M, a.part_ml[place(j) * 2]);
#pragma unroll
      for (int m = 16; m > 0; m /= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
      if (lane == 0) s_red[0][warp] = M;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarpsHere; ++w) M = fmaxf(M, s_red[0][w]);
      float sum = 0.f;
      for (int j = tid; j < parts; j += kJoinThreads) {
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
      for (int w = 0; w < kWarpsHere; ++w) sum += s_red[1][w];
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      auto add = [&](int j, const float4& x) {
        const float f = s_factor[j];
        v.x = fmaf(f, x.x, v.x); v.y = fmaf(f, x.y, v.y); v.z = fmaf(f, x.z, v.z); v.w = fmaf(f, x.w, v.w);
      };
#pragma unroll
      for (int k = 0; k < kDeep; ++k)
        if (part0 + k * kJoin < parts) add(part0 + k * kJoin, o[k]);
      for (int j = part0 + kDeep * kJoin; j < parts; j += kJoin)
        add(j, *reinterpret_cast<const float4*>(a.part_o + place(j) * D + 4 * d4));
      s_o[part0][d4] = v;
      __syncthreads();
      if (part0 == 0) {
#pragma unroll
        for (int k = 1; k < kJoin; ++k) {
          const float4 x = s_o[k][d4];
          v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
        }
        const int rr = own.rt * tile_rows + row;
        const int tok = rr / a.group, head = rr - tok * a.group;
        const float inv = sum == 0.f ? 0.f : kDown / sum;
        uint16_t* dst = a.L.out + ((static_cast<int64_t>(own.tok0) + tok) * a.L.num_q_heads + own.h * a.group + head) * D + 4 * d4;
        *reinterpret_cast<uint2*>(dst) = make_uint2(cosa::pack_bf16x2(v.x * inv, v.y * inv), cosa::pack_bf16x2(v.z * inv, v.w * inv));
        if (WEIGHTS && d4 == 0) {
          float* st = a.stats + ((static_cast<int64_t>(own.h) * a.L.total_tokens + own.tok0) * a.group + rr) * 2;
          st[0] = M;
          st[1] = sum;
        }
      }
      __syncthreads();
    }
  }
}

// The same for many items of few parts: a block per owner CTA, a warp per row.
template <int D, bool WEIGHTS>
__global__ void __launch_bounds__(kJoinThreads) combine_kernel(const Args a, const int tile_rows) {
  constexpr int V = D / 32;          // values of a lane
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int first = blockIdx.x;
  wait_for_stream();
  let_next_start();
  const Owner own = a.owner[first];
  for (int row = warp; row < own.rows; row += kJoinThreads / 32) {
    auto place = [&](int j) { return (static_cast<size_t>(first + j) * 2 + (j == 0 ? 1 : 0)) * kMaxRows + row; };
    const int parts = own.last - first + 1;
    float M = -INFINITY;
    for (int j = lane; j < parts; j += 32) M = fmaxf(M, a.part_ml[place(j) * 2]);
#pragma unroll
    for (int m = 16; m > 0; m /= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
    float sum = 0.f, v[V];
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = 0.f;
#pragma unroll 4
    for (int j = 0; j < parts; ++j) {
      const float m = a.part_ml[place(j) * 2];
      const float f = m == -INFINITY ? 1.f : cosa::ex2_approx(m - M);       // nothing seen: sums of zero, or NaN
      sum = fmaf(f, a.part_ml[place(j) * 2 + 1], sum);
#pragma unroll
      for (int k = 0; k < V; k += 2) {
        const float2 x = *reinterpret_cast<const float2*>(a.part_o + place(j) * D + V * lane + k);
        v[k] = fmaf(f, x.x, v[k]);
        v[k + 1] = fmaf(f, x.y, v[k + 1]);
      }
    }
    const int rr = own.rt * tile_rows + row;
    const int tok = rr / a.group, head = rr - tok * a.group;
    const float inv = sum == 0.f ? 0.f : kDown / sum;
    uint16_t* dst = a.L.out + ((static_cast<int64_t>(own.tok0) + tok) * a.L.num_q_heads + own.h * a.group + head) * D + V * lane;
#pragma unroll
    for (int k = 0; k < V; k += 2) *reinterpret_cast<uint32_t*>(dst + k) = cosa::pack_bf16x2(v[k] * inv, v[k + 1] * inv);
    if (WEIGHTS && lane == 0) {
      float* st = a.stats + ((static_cast<int64_t>(own.h) * a.L.total_tokens + own.tok0) * a.group + rr) * 2;
      st[0] = M;
      st[1] = sum;
    }
  }
}

// weights[b, h, s] += sum over the rows of exp2(scale * logit - M) / sum, rows in order; four slots per thread.
constexpr int kWeightRows = 32;       // rows whose maxima and sums a CTA holds at a time
__global__ void __launch_bounds__(256) weights_kernel(const Args a) {
  __shared__ float2 s_stat[kWeightRows];
  wait_for_stream();
  const int b = blockIdx.z, h = blockIdx.y;
  const Request r = request_of(a, b, 8, kTile, false);
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

// Row pitch of the logits: whole units, of which the last is written to its end.
int64_t logits_pitch(int max_seqlen) { return (static_cast<int64_t>(max_seqlen) + 31) / 32 * 32; }

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

template <int D, int NT, bool WEIGHTS>
cudaError_t launch(Args a, cudaStream_t stream) {
  using S = Steps<NT>;
  constexpr size_t smem = sizeof(AttnSmem<D, NT>);
  static_assert(S::kCtas * (smem + 1024) <= 228 * 1024, "shared memory of an SM");
  const int64_t rows = static_cast<int64_t>(a.L.max_new_tokens) * a.group;
  const int64_t row_tiles = std::min<int64_t>((rows + 8 * NT - 1) / (8 * NT), INT32_MAX);
  // how many (request, kv head, row tile) there are and how many units they have, as far as the parameters tell (either way
  // of sharing them is right for any number)
  const int64_t items = static_cast<int64_t>(a.L.num_reqs) * a.L.num_kv_heads * row_tiles;
  const int64_t units = (static_cast<int64_t>(a.L.max_seqlen) + S::TP * kTile - 1) / (S::TP * kTile);
  int ctas = 1;
  while (ctas < kMaxCluster && 2 * ctas * items <= S::kResident && ctas * kWarps < units) ctas *= 2;
  cudaError_t e;
  // Clusters where a warp has few tokens: up to 512 of them where the clusters fill half of the card, else up to 256.
  const int64_t tokens = (units + ctas * kWarps - 1) / (ctas * kWarps) * (S::TP * kTile);
  if (ctas * items <= S::kResident && tokens <= (2 * ctas * items >= S::kResident ? 2 * kClusterTokens : kClusterTokens)) {
    auto* kernel = attention_kernel<D, NT, WEIGHTS, true>;
    a.row_tiles = static_cast<int>(row_tiles);
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = launch_after(kernel, dim3(static_cast<unsigned>(items * ctas)), kThreads, smem, stream, ctas, a);
  } else {
    auto* kernel = attention_kernel<D, NT, WEIGHTS, false>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e == cudaSuccess) e = launch_after(kernel, dim3(S::kResident), kThreads, smem, stream, 1, a);
    if (e != cudaSuccess) return e;
    if (items <= kFewItems)
      e = launch_after(combine_wide_kernel<D, WEIGHTS>, dim3(64, static_cast<unsigned>(std::min<int64_t>(8 * NT, rows))),
                       kJoinThreads, 0, stream, 1, a, S::kResident, 8 * NT);
    else
      e = launch_after(combine_kernel<D, WEIGHTS>, dim3(S::kResident), kJoinThreads, 0, stream, 1, a, 8 * NT);
  }
  if (e != cudaSuccess || !WEIGHTS) return e;
  const dim3 grid(static_cast<unsigned>((a.L.max_seqlen + 1023LL) / 1024), static_cast<unsigned>(a.L.num_kv_heads),
                  static_cast<unsigned>(a.L.num_reqs));
  return launch_after(weights_kernel, grid, 256, 0, stream, 1, a);
}

// Row tiles of 8, 16 or 24 rows: the smallest that has all of a request's rows, else of 16, the least time per row.  Tiles of
// 8 / 16 / 24 rows, 8 contexts of 16K with 8 kv heads: 12 rows 62 / 57 / - us, 16 rows 63 / 59 / - us, 32 rows 113 / 91 / -
// us, 64 rows 213 / 166 / 203 us; 17 contexts of 4K with 20 rows 53 / 55 / 46 us.
template <int D, bool WEIGHTS>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(a.L.max_new_tokens) * a.group;
  if (rows <= 8) return launch<D, 1, WEIGHTS>(a, stream);
  return rows > 16 && rows <= 24 ? launch<D, 3, WEIGHTS>(a, stream) : launch<D, 2, WEIGHTS>(a, stream);
}

}  // namespace

// 0 if it passes 2^61 bytes (the logits of rows and slots that no memory holds).
size_t attn_workspace_bytes(int num_q_heads, int head_dim, int total_tokens, int max_seqlen, bool with_weights) {
  size_t n = align256(kMaxCtas * sizeof(Owner)) + align256(size_t(kMaxCtas) * 2 * kMaxRows * 2 * 4) +
             align256(size_t(kMaxCtas) * 2 * kMaxRows * head_dim * 4);
  if (with_weights) {
    const size_t rows = static_cast<size_t>(total_tokens) * num_q_heads;
    if (rows > (size_t(1) << 61) / (logits_pitch(max_seqlen) * 4)) return 0;
    n += align256(rows * 8) + align256(rows * logits_pitch(max_seqlen) * 4);
  }
  return n;
}

cudaError_t launch_attention(const AttnLaunch& L, cudaStream_t stream) {
  Args a{};
  a.L = L;
  a.L.max_new_tokens = std::min(L.max_new_tokens, L.total_tokens);
  a.L.scale_log2 = L.scale_log2 * kDown;      // of the logits as the first product leaves them
  a.group = L.num_q_heads / L.num_kv_heads;
  for (a.page_shift = 4; (1 << a.page_shift) < L.page_size;) ++a.page_shift;
  a.pitch = logits_pitch(L.max_seqlen);
  a.stall = L.stall;
  uint8_t* w = static_cast<uint8_t*>(L.workspace);
  a.owner = reinterpret_cast<Owner*>(w);
  w += align256(kMaxCtas * sizeof(Owner));
  a.part_ml = reinterpret_cast<float*>(w);
  w += align256(size_t(kMaxCtas) * 2 * kMaxRows * 2 * 4);
  a.part_o = reinterpret_cast<float*>(w);
  w += align256(size_t(kMaxCtas) * 2 * kMaxRows * L.head_dim * 4);
  if (L.weights) {
    a.stats = reinterpret_cast<float*>(w);
    w += align256(static_cast<size_t>(L.total_tokens) * L.num_q_heads * 8);
    a.logits = reinterpret_cast<float*>(w);
  }
  if (L.head_dim == 128) return L.weights ? launch<128, true>(a, stream) : launch<128, false>(a, stream);
  return L.weights ? launch<64, true>(a, stream) : launch<64, false>(a, stream);
}

}  // namespace cosa_kv
