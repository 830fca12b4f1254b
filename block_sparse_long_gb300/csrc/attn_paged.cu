// Attention of each request's newest tokens over pages: the tree attention's keys and values, or latent vectors (one key
// head whose first values are the value).
//
//     s = k . q (slot by row),  p = exp2(s * scale - m_row),  o = sum p v,  l = sum p
//
// A row is a (new token, query head of the kv head): R = n * Hq / Hkv of them share every key, one to some hundreds.  With so few
// the cache is read once and the memory bounds the call, so the matrix instructions are set up for what there is plenty of.
//   Up to 32 rows (of latent vectors 64 at a time): the 128 slots of a tile, or 128 values of the output, are the 128 rows of a
//   tcgen05.mma, and the 16, 32 or 64 query rows its columns.  S^T = K Q^T has a slot per TMEM lane, O^T = V^T P^T a value per
//   lane; K comes as it lies in its page, and as V read the other way (values contiguous), so latent vectors are loaded once for
//   both products.  P^T goes through shared memory.
//   More rows (kRowLanes): the 128 rows of the product are query rows, S = Q K^T, O = P V with P in TMEM, so that a softmax thread has a
//   row (half of its slots), needs no other thread's maximum and keeps the reference in a register.  64 new tokens of 4 heads to a
//   kv head after 128K slots: 231 us with the rows as 128 columns, 177 with a quarter of the slots to a thread, with half of them (fewer
//   warps, of whose 168 registers 4 to 8 bytes spill) and pages looked up a tile ahead 11 % less.
//
// A CTA per SM.  The tiles of all (request, kv head, row tile) items stand in one list, which the CTAs share evenly, one unit per
// tile and one per item; a CTA's piece of an item that others have too leaves m, l and o (32 bits) in the workspace and
// join_kernel puts them together.  Short contexts go whole to a CTA or to a cluster that joins them through distributed shared
// memory (900 slots: list and join 10.3 us, cluster 8.9).  With several row tiles of 128 rows to the same keys as many CTAs walk the
// list together, a CTA to a row tile, so that HBM is read once (the same 128K: 177 us apart, 140 together; then 125 as above).
//
// What bounds it (32 query over 8 kv heads of 128, 64-slot pages): 13-token trees of 24 ragged contexts 158 us, 5.7 TB/s; 64 tokens
// after 128K 125 us, 4.3 TB/s and 1.1 PFLOP/s, a tile's chain of product, softmax, product (2000 cycles, of which the products run
// 1024); one token after 900 slots 8.9 us, the chain of first loads, products and join.  Latent vectors of 512 + 64, 32 heads: one token after
// 128K 43 us, 3.5 TB/s; 7 tokens of 24 ragged contexts 144 us: a tile (147 KB) fills shared memory, so a block of the next can only be copied
// once the second product is done with it (6000 cycles a tile, of which the products run 3300).
//
// Warp roles:
//   warp 0     producer: looks up the pages of a tile and copies them by TMA into a ring of 32 KB slots (two 128-byte wide
//              columns of 128 slots), four to six of them.
//   warp 1     issues the first product of every tile into one of two TMEM buffers.
//   warp 2     issues the second; clears rows of V that no slot has, and in the tile of the new tokens what is not finite (0 times
//              that is not 0; the rows that see it get it added at the end).
//   warp 3     owns the TMEM; writes down what is to be joined.
//   warps 4-   softmax.  The reference m of a row is that of an earlier tile until some weight exceeds 2^8, so that most tiles need
//              no maximum over the slots: one vote, the exponentials, and P as bf16 (2^-9 of each term; l sums the unrounded ones).
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "attn_mma.cuh"
#include "attn_tma.h"
#include "kv_internal.h"
#include "kv_layout.cuh"

namespace cosa_attn {
namespace {

using cosa::fence_proxy_async_smem;
using cosa::mbar_arrive;
using cosa::mbar_arrive_expect_tx;
using cosa::mbar_init;
using cosa::named_bar_red_or;
using cosa::named_bar_sync;
using cosa::smem_u32;
using cosa::tc_fence_after;
using cosa::tc_fence_before;
using cosa::umma_commit;
using cosa::wait_parity_bounded;

constexpr int kTile = 128;                 // slots
constexpr int kCtas = 152;
constexpr int kMaxCluster = 8;
constexpr int kColumn = kTile * 128;       // bytes of a 64-value wide column of a tile
constexpr int kPair = 2 * kColumn;
constexpr float kNone = -3e38f;            // reference of a row that has seen nothing
constexpr float kHigh = 8.0f;              // log2 of the weight from which on a row's reference moves
constexpr uint32_t kHighBits = 0x4380;     // the weight, 2^8, in bf16
constexpr float kLn2 = 0.69314718055994531f;

// DK, DV: values of a key and a value.  kLatent: the value is the key's first DV values.  N: query rows of a row tile.
template <int DK_, int DV_, bool LATENT, int N_>
struct Shape {
  static constexpr int DK = DK_, DV = DV_, N = N_;
  static constexpr bool kLatent = LATENT;
  static constexpr bool kRowLanes = N == 128;                    // a query row per TMEM lane: S = Q K^T, O = P V, P in TMEM
  static constexpr int kGroups = N == 16 ? 1 : N == 64 ? 4 : 2;  // warpgroups of the softmax
  static constexpr int NC = kRowLanes ? 1 : 16;                  // query rows of a softmax thread
  // Row tiles of 64 have 640 threads and so 96 registers each, of which 20 bytes (latent vectors of 512) or 116 (of 256) spill.
  static constexpr int kThreads = 128 + 128 * kGroups;
  static constexpr int kBlocks = DV > 128 ? DV / 128 : 1;        // of 128 output values
  static constexpr int kPairs = LATENT ? DV / 128 : DK == 128 ? 2 : 1;      // ring slots of a tile; 64 + 64: K and V in one
  static constexpr int kQBytes = N * DK * 2;
  static constexpr int kPBytes = N * kTile * 2;
  // The widest latent rows leave no room for P: it goes over the rotated part of the keys, which S^T has used by then.
  static constexpr bool kAlias = LATENT && DV == 512 && N == 64;
  static constexpr int kPBufs = kAlias || (LATENT && DV == 512 && N == 32) ? 1 : 2;
  static constexpr int kPSmem = kAlias || kRowLanes ? 0 : kPBufs;    // of them in shared memory, in their own place
  static constexpr int kRopes = LATENT && DV + N <= 528 ? 2 : 1;      // (1, unused, without latent vectors)
  static constexpr int kSmall = 2048 + N * (56 + 8 * kMaxCluster);
  static constexpr int kRoom = 227 * 1024 - 1024 - kSmall - kQBytes - kPSmem * kPBytes - (LATENT ? kRopes * kColumn : 1024);
  // Keys and values in slots of their own are waited for by different warps, and a parity wait tells only two phases apart: an even
  // number of slots has either keys or values in a slot, so that each barrier's phases are waited for by one warp, in order.
  static constexpr int kFit = kRoom / kPair < 6 ? kRoom / kPair : 6;
  static constexpr bool kSplit = kPairs == 2 && !LATENT;
  static constexpr int kSlots = kSplit ? kFit / 2 * 2 : kFit;
  // A tile's place: one slot (of a pair, for kSplit: an even one for keys and the odd one behind it for values), kLatent: several.
  static constexpr int kRing = kSplit ? kSlots / 2 : kSlots, kStep = kSplit ? 2 : 1;
  static_assert(kSlots >= kPairs, "a tile fits the ring");
  static constexpr uint32_t kTmemO = 0, kTmemS = kRowLanes ? DV : kBlocks * N, kTmemP = kTmemS + 2 * N;
  static_assert(kTmemP + (kRowLanes ? kPBufs * kTile / 2 : 0) <= 512, "TMEM columns");
  // P^T: rows of 32, 64 or 128 bytes per slot, swizzled at that width
  static constexpr int kPRow = N >= 64 ? 128 : 2 * N;
};

// What join_kernel has to put together: `parts` parts of an item, the first in slot `first`, the others in next, next + step, ...
struct Join {
  int32_t parts, first, next, step, tok0, rows, head, row_tile;
};

struct Args {
  const uint16_t *q, *q_rope, *k_cache, *v_cache;
  const int32_t *cu_seqlens, *page_table, *kv_len;
  const int64_t* tree_mask;
  uint16_t* out;
  float *lse, *part_o, *part_ml;
  Join* joins;
  int32_t* status;
  int64_t q_stride, q_head_stride, q_rope_stride, q_rope_head_stride;
  int num_reqs, num_q_heads, num_kv_heads, group, page_shift, total_tokens, max_seqlen, num_pages, max_pages_per_req;
  int join_items;      // entries of `joins` if they are by item, 0 if by CTA
  int whole;           // items are not cut: a unit is an item
  int cluster;         // CTAs that share an item by its tiles and join it themselves (whole), or 1
  int together;        // CTAs that walk the list as one, for as many row tiles of the same keys, or 1
  int walkers;         // CTAs, or as many times so many
  float scale_log2;
  int stall;
};

// A request: its tokens, rows, tiles.  Without keys (lengths that contradict each other) it has no tiles, but its rows are written.
struct Request {
  int tok0, n, len, tiles, row_tiles;
  bool bad;
};

template <int N>
__device__ __forceinline__ Request request_of(const Args& a, int b) {
  Request r;
  r.tok0 = __ldg(a.cu_seqlens + b);
  const int64_t n = static_cast<int64_t>(__ldg(a.cu_seqlens + b + 1)) - r.tok0;
  r.len = __ldg(a.kv_len + b);
  r.bad = r.tok0 < 0 || n < 0 || r.tok0 + n > a.total_tokens;
  r.n = r.bad ? 0 : static_cast<int>(n);
  if (r.n > 0 && (r.len < r.n || r.len > a.max_seqlen || (a.tree_mask && r.n > COSA_ATTN_MAX_TREE))) r.bad = true;
  if (r.bad || r.n == 0) r.len = 0;
  r.tiles = (r.len + kTile - 1) / kTile;
  r.row_tiles = static_cast<int>((static_cast<uint32_t>(r.n) * static_cast<uint32_t>(a.group) + N - 1) / N);     // total_tokens * Hq fits 31 bits
  return r;
}

// An item of the list is a (request, kv head, up to `together` row tiles).
template <int N>
__device__ __forceinline__ int together_of(const Args& a) {
  return N == 128 ? a.together : 1;
}
template <int N>
__device__ __forceinline__ int rounds_of(const Args& a, const Request& r) {
  return (r.row_tiles + together_of<N>(a) - 1) / together_of<N>(a);
}
template <int N>
__device__ __forceinline__ int units_of(const Args& a, const Request& r) {
  return a.num_kv_heads * rounds_of<N>(a, r) * (a.whole ? 1 : r.tiles + 1);
}

// How `total` units are shared by the walkers (CTAs, clusters, or CTAs together): the first `more` have one unit more than `each`.
struct Shares {
  uint32_t each, more;
  __device__ __forceinline__ Shares(int total, int walkers) : each(0), more(total) {
    if (total < walkers) return;
    each = static_cast<uint32_t>(total) / walkers;
    more = total - each * walkers;
  }
  __device__ __forceinline__ int first(uint32_t walker) const { return static_cast<int>(each * walker + min(walker, more)); }
  __device__ __forceinline__ int owner(uint32_t unit) const {
    const uint32_t all = more * (each + 1);
    return static_cast<int>(unit < all ? unit / (each + 1) : more + (unit - all) / each);
  }
};

// What a CTA does of one item: tiles t0 .. t1 - 1 of its row tile (none if the request has fewer row tiles).
struct Piece {
  Request r;
  int b, head, row_tile, t0, t1;
  int slot;          // of the workspace, or -1: all of the item
  bool begins;       // it has the item's first unit
  int item;          // number of the item in the batch
  int item_end;      // behind its last unit
};

// The pieces of a walker in order; every role walks them by itself.
template <int N>
struct Pieces {
  int pos, first, end, before, units, items, b;      // units and items before and of request b
  Request r;

  __device__ __forceinline__ bool next(const Args& a, Piece& p) {
    if (pos >= end) return false;
    while (pos >= before + units) {
      before += units;
      items += a.num_kv_heads * rounds_of<N>(a, r);
      r = request_of<N>(a, ++b);
      units = units_of<N>(a, r);
    }
    const uint32_t per = a.whole ? 1 : r.tiles + 1, item = a.whole ? pos - before : static_cast<uint32_t>(pos - before) / per;
    const int u = static_cast<int>(pos - before - item * per), take = min(static_cast<int>(per) - u, end - pos);
    p.r = r;
    p.b = b;
    const uint32_t rounds = rounds_of<N>(a, r);
    p.head = rounds == 1 ? item : item / rounds;
    p.row_tile = (static_cast<int>(item) - p.head * static_cast<int>(rounds)) * together_of<N>(a) + blockIdx.x % together_of<N>(a);
    p.t0 = a.whole ? 0 : max(u - 1, 0);
    p.t1 = a.whole ? r.tiles : u + take - 1;
    if (together_of<N>(a) > 1 && p.row_tile >= r.row_tiles) p.t0 = p.t1 = 0;
    if (a.cluster > 1) {
      const int rank = blockIdx.x % a.cluster;
      p.t1 = r.tiles * (rank + 1) / a.cluster;
      p.t0 = r.tiles * rank / a.cluster;
    }
    p.slot = take == static_cast<int>(per) ? -1 : 2 * static_cast<int>(blockIdx.x) + (pos != first);
    p.begins = u == 0;
    p.item = items + static_cast<int>(item);
    p.item_end = pos + static_cast<int>(per) - u;
    pos += take;
    return true;
  }
};

// The list's units and items, and a CTA's walk of it after its first piece.  (A call is refused where they could pass 31 bits.)
template <int N>
struct Start {
  int32_t total, items;
  Pieces<N> rest;
  Piece first;
  bool any;
};

// By one warp, a request to a lane at a time.
template <int N>
__device__ __forceinline__ Start<N> find_start(const Args& a, bool report) {
  const int per = a.cluster * together_of<N>(a), walker = per == 1 ? blockIdx.x : blockIdx.x / static_cast<unsigned>(per);
  const int lane = threadIdx.x % 32;
  Start<N> st;
  Request r{};
  int units = 0, items = 0;       // of this lane's last request
  auto look = [&](int b) {
    units = items = 0;
    if (b >= a.num_reqs) return;
    r = request_of<N>(a, b);
    units = units_of<N>(a, r);
    items = a.num_kv_heads * rounds_of<N>(a, r);
  };
  st.items = 0;
  uint64_t total = 0;
  for (int b0 = 0; b0 < a.num_reqs; b0 += 32) {
    look(b0 + lane);
    if (b0 + lane < a.num_reqs && r.bad && report) cosa::report_status(a.status, cosa::kStatusBadInput);
    const uint32_t u = units;
    total += (static_cast<uint64_t>(__reduce_add_sync(kAll, u >> 16)) << 16) + __reduce_add_sync(kAll, u & 0xFFFFu);
    st.items += __reduce_add_sync(kAll, items);
  }
  // Requests that share tokens (cu_seqlens that falls and rises) can have more units than the call was checked for: then nothing is done.
  if (total > INT32_MAX) {
    total = st.items = 0;
    if (report && lane == 0) cosa::report_status(a.status, cosa::kStatusBadInput);
  }
  st.total = static_cast<int>(total);
  Pieces<N>& w = st.rest;
  const Shares shares(st.total, a.walkers);
  w.first = w.pos = shares.first(walker);
  w.end = walker < a.walkers ? shares.first(walker + 1) : w.pos;
  if (a.cluster > 1) w.end = min(w.end, w.pos + 1);
  w.before = w.items = w.units = 0;
  st.any = w.pos < w.end;
  if (!st.any) return st;
  for (int b0 = 0;; b0 += 32) {
    if (a.num_reqs > 32) look(b0 + lane);
    int upto = units, upto_items = items;
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
      const int x = __shfl_up_sync(kAll, upto, m), y = __shfl_up_sync(kAll, upto_items, m);
      if (lane >= m) upto += x, upto_items += y;
    }
    const unsigned past = __ballot_sync(kAll, w.before + upto > w.pos);
    const int l = past ? __ffs(past) - 1 : 31;
    w.before += __shfl_sync(kAll, past ? upto - units : upto, l);
    w.items += __shfl_sync(kAll, past ? upto_items - items : upto_items, l);
    if (!past) continue;
    w.b = b0 + l;
    w.units = __shfl_sync(kAll, units, l);
    w.r.tok0 = __shfl_sync(kAll, r.tok0, l);
    w.r.n = __shfl_sync(kAll, r.n, l);
    w.r.len = __shfl_sync(kAll, r.len, l);
    w.r.tiles = __shfl_sync(kAll, r.tiles, l);
    w.r.row_tiles = __shfl_sync(kAll, r.row_tiles, l);
    w.r.bad = false;
    w.next(a, st.first);
    return st;
  }
}

template <class S>
struct alignas(1024) Smem {
  uint8_t ring[S::kSlots][kPair];
  uint8_t rope[S::kRopes][S::kLatent ? kColumn : 1024];
  uint8_t q[S::kQBytes];
  uint8_t p[S::kPSmem ? S::kPSmem : 1][S::kPSmem ? S::kPBytes : 16];
  uint64_t full[S::kSlots], empty[S::kSlots];
  uint64_t rope_full[2], rope_empty[2];
  uint64_t q_ready, s_full[2], s_empty[2], p_full[2], pv_done[2], groups, cleanup;
  uint64_t mask[S::N];               // tree mask of a row's token
  alignas(16) float base[S::N];      // a row's reference (log2 units), negated; read four at a time
  float alpha[S::N];                 // a reference's last change
  float part[4][S::N];               // maxima and sums of the four warps that have a row's slots
  int32_t row[S::N];                 // output row, or -1
  int32_t node[S::N];                // token of the request
  int64_t q_at[S::N], r_at[S::N];    // its values in q and q_rope
  float2 ml[kMaxCluster][S::N];      // references and sums of the cluster's CTAs
  Start<S::N> start;
  int32_t odd_values;                // something among the new tokens' values is not finite
  int32_t over;                      // a wait of the call had run out before this CTA started
  uint32_t tmem_base;
  int32_t abort_flag;
};

// (d0, d1) = (a0, a1) * b + (c0, c1)
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b, float c0, float c1) {
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%5, %6};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}

__device__ __forceinline__ void copy16(void* dst, const void* src, bool there) {      // asynchronous; zeros if there is nothing
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// Shared memory of another CTA of the cluster.
__device__ __forceinline__ uint32_t remote(const void* p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void store_remote(uint32_t to, float x) { asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(x) : "memory"); }
__device__ __forceinline__ void store_remote(uint32_t to, float x, float y, float z, float w) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}
__device__ __forceinline__ void store_remote(const void* to, int rank, float2 x) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(remote(to, rank)), "f"(x.x), "f"(x.y) : "memory");
}
// Every thread of every CTA of the cluster arrives, whatever became of its waits before.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The first of them in halves: it orders no memory (900 slots of one token: 0.15 us less than with a release).
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// Where 16-byte piece c of row t of P^T goes (the swizzle of rows of kRow bytes).
template <int kRow>
__device__ __forceinline__ int p_offset(int t, int c) {
  const int x = kRow == 128 ? t & 7 : kRow == 64 ? t >> 1 & 3 : t >> 2 & 1;
  return t * kRow + ((c ^ x) << 4);
}

template <int NC>
__device__ __forceinline__ void load_columns(uint32_t taddr, float (&x)[NC]) {
  uint32_t r[NC];
  if constexpr (NC == 16) {
    cosa::tmem_ld16(taddr, r);
  } else {
#pragma unroll
    for (int i = 0; i < NC; i += 32) cosa::tmem_ld32(taddr + i, *reinterpret_cast<uint32_t(*)[32]>(&r[i]));
  }
  cosa::tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < NC; ++i) x[i] = __uint_as_float(r[i]);
}

// The first n bits.
__device__ __forceinline__ uint64_t ones(int n) { return n <= 0 ? 0 : n >= 64 ? ~uint64_t{0} : (uint64_t{1} << n) - 1; }

// The largest value of a warp; NaN counts as nothing.
__device__ __forceinline__ float warp_max(float x) {
  if (x != x) x = -INFINITY;
  int i = __float_as_int(x);
  i ^= (i >> 31) & 0x7fffffff;
  i = __reduce_max_sync(kAll, i);
  i ^= (i >> 31) & 0x7fffffff;
  return __int_as_float(i);
}

template <class S>
__global__ void __launch_bounds__(S::kThreads, 1)
    paged_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Args a) {
  constexpr int N = S::N, NC = S::NC, DV = S::DV;
  extern __shared__ uint8_t smem_raw[];
  Smem<S>& sm = *reinterpret_cast<Smem<S>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, cta = blockIdx.x;
  volatile int* abort_flag = &sm.abort_flag;
  cosa_kv::wait_for_stream();
  cosa_kv::let_next_start();
  if (a.cluster > 1) cluster_arrive();      // (waited for before the first store to another CTA)

  if (warp == 0) {
    const bool over = gave_up(a.status);
    const Start<N> st = find_start<N>(a, cta == 0);
    if (lane == 0) {
      sm.start = st;
      sm.over = over;
      if (cta == 0 && (a.cu_seqlens[0] != 0 || a.cu_seqlens[a.num_reqs] > a.total_tokens)) cosa::report_status(a.status, cosa::kStatusBadInput);
    }
  } else if (warp == 1 && lane == 0) {
    for (int s = 0; s < S::kSlots; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.rope_full[s], 1);
      mbar_init(&sm.rope_empty[s], 1);
      mbar_init(&sm.s_full[s], 1);
      mbar_init(&sm.s_empty[s], 4 * S::kGroups);
      mbar_init(&sm.p_full[s], 4 * S::kGroups);
      mbar_init(&sm.pv_done[s], 2);       // the products, and the issuing warp's own arrival
    }
    mbar_init(&sm.q_ready, 1);
    mbar_init(&sm.groups, 4 * S::kGroups);
    mbar_init(&sm.cleanup, 2);
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
  // for (more = ...) below: the pieces of this CTA
  Pieces<N> pieces = sm.start.rest;
  Piece pc = sm.start.first;
  const bool works = sm.start.any && !sm.over;
  bool more = works;
  const int pages_per_tile = kTile >> a.page_shift;

  if (warp == 0) {
    // =========================== producer ===========================
    if (lane == 0) {
      cosa::tma_prefetch_desc(&kmap);
      cosa::tma_prefetch_desc(&vmap);
    }
    Ring<S::kRing> ring, vring;      // (vring: kSplit's values)
    Ring<S::kRopes> rope;
    int pairs = 0, vpairs = 0, ropes = 0;      // slots taken, up to the rings' sizes
    bool ok = !a.stall;
    const int page = lane & (pages_per_tile - 1), column = lane / pages_per_tile, to = (page << a.page_shift) * 128;
    // The pages of a tile, a page and column to a lane.
    struct Tile {
      uint32_t bytes;      // of a 64-value column
      int place, head;     // row of the lane's page in the cache, kv head
      bool copies;
    };
    auto take = [&](Ring<S::kRing>& r, int& taken, int odd) {
      if (taken == S::kRing) ok = warp_wait(&sm.empty[r.at * S::kStep + odd], r.phase ^ 1, abort_flag, a.status);
      else ++taken;
      return r.at * S::kStep + odd;
    };
    // A pair of columns from c0 on, of one cache or of both.
    auto copy = [&](const Tile& x, int s, const CUtensorMap* first, const CUtensorMap* second, int c0, int c1) {
      if (lane == 0) mbar_arrive_expect_tx(&sm.full[s], 2 * x.bytes);
      __syncwarp();
      if (column < 2 && x.copies)
        cosa::tma_load_4d(&sm.ring[s][column * kColumn + to], column ? second : first, &sm.full[s], 0, x.place, column ? c1 : c0, x.head);
    };
    Tile last{};
    bool waiting = false;      // kSplit: the last tile's values, which come behind the next tile's keys (keys are free sooner)
    auto values = [&] {
      const int s = take(vring, vpairs, 1);
      if (!ok) return;
      copy(last, s, &vmap, &vmap, 0, 1);
      vring.next();
      waiting = false;
    };
    for (; ok && more; more = pieces.next(a, pc)) {
      const int32_t* table = a.page_table + static_cast<size_t>(pc.b) * a.max_pages_per_req;
      auto look_up = [&](int t) {
        const int p = t * pages_per_tile + lane;
        return t < pc.t1 && lane < pages_per_tile && p << a.page_shift < pc.r.len ? __ldg(table + p) : -1;
      };
      int phys_next = look_up(pc.t0);
      for (int t = pc.t0; t < pc.t1 && ok; ++t) {
        const int phys = phys_next;
        phys_next = look_up(t + 1);
        const unsigned there = __ballot_sync(kAll, phys >= 0 && phys < a.num_pages);
        Tile x;
        x.bytes = static_cast<uint32_t>(__popc(there)) << a.page_shift << 7;
        x.place = __shfl_sync(kAll, phys, page) << a.page_shift;
        x.head = S::kLatent ? 0 : pc.head;
        x.copies = there >> page & 1;
        auto rotated = [&] {
          if (ropes == S::kRopes) ok = warp_wait(&sm.rope_empty[rope.at], rope.phase ^ 1, abort_flag, a.status);
          else ++ropes;
          if (!ok) return;
          if (lane == 0) mbar_arrive_expect_tx(&sm.rope_full[rope.at], x.bytes);
          __syncwarp();
          if (column == 0 && x.copies) cosa::tma_load_4d(&sm.rope[rope.at][to], &kmap, &sm.rope_full[rope.at], 0, x.place, DV / 64, 0);
          rope.next();
        };
        if constexpr (S::kLatent && !S::kAlias) rotated();
        for (int i = 0; i < (S::kSplit ? 1 : S::kPairs) && ok; ++i) {
          const int s = take(ring, pairs, 0);
          if (!ok) break;
          if (S::kLatent) copy(x, s, &kmap, &kmap, 2 * i, 2 * i + 1);
          else if (S::kSplit) copy(x, s, &kmap, &kmap, 0, 1);
          else copy(x, s, &kmap, &vmap, 0, 0);
          ring.next();
        }
        if constexpr (S::kAlias) {
          if (ok) rotated();
        }
        if constexpr (S::kSplit) {
          if (ok && waiting) values();
          last = x;
          waiting = true;
        }
      }
    }
    if (ok && waiting) values();
    // every copy lands before the CTA ends: the last use of each slot (those before it have landed, or it had not been taken); all of
    // them have one wait's time together
    if (lane == 0) {
      const uint64_t since = cosa::global_timer_ns();
      for (; pairs > 0; --pairs) {
        ring.back();
        cosa::wait_until(&sm.full[ring.at * S::kStep], ring.phase, since);
      }
      for (; vpairs > 0; --vpairs) {
        vring.back();
        cosa::wait_until(&sm.full[vring.at * S::kStep + 1], vring.phase, since);
      }
      for (; ropes > 0; --ropes) {
        rope.back();
        cosa::wait_until(&sm.rope_full[rope.at], rope.phase, since);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // =========================== S^T = K Q^T ===========================
    constexpr uint32_t idesc = cosa::idesc_bf16_f32(128, N, false, false), hi = desc_hi(1024, 2);
    const uint32_t qd = desc_lo(smem_u32(sm.q), 16), kd = desc_lo(smem_u32(sm.ring), 16), rd = desc_lo(smem_u32(sm.rope), 16);
    Ring<S::kRing> ring;
    Ring<S::kRopes> rope;
    Ring<2> sbuf;
    int tile = 0, turn = 0;
    bool ok = true;
    for (; ok && more; more = pieces.next(a, pc)) {
      if (pc.t0 == pc.t1) continue;
      ok = warp_wait(&sm.q_ready, turn++ & 1, abort_flag, a.status);
      for (int t = pc.t0; t < pc.t1 && ok; ++t) {
        if (tile == 2) ok = warp_wait(&sm.s_empty[sbuf.at], sbuf.phase ^ 1, abort_flag, a.status);
        else ++tile;
        const uint32_t d = tmem + S::kTmemS + sbuf.at * N;
        // the rotated part comes last where P^T goes over it, else first
        auto rotated = [&] {
          ok = ok && warp_wait(&sm.rope_full[rope.at], rope.phase, abort_flag, a.status);
          if (!ok) return;
          tc_fence_after();
          const uint32_t k0 = rd + rope.at * (kColumn >> 4);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_ss(d, k0 + 2 * k, hi, qd + ((DV / 64 * N * 128) >> 4) + 2 * k, hi, idesc, S::kAlias || k > 0);
            if (!S::kAlias) umma_commit(&sm.rope_empty[rope.at]);
          }
          __syncwarp();
          rope.next();
        };
        if constexpr (S::kLatent && !S::kAlias) rotated();
        constexpr int kKeys = S::kLatent ? S::kPairs : 1;      // ring slots with keys
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
          const int s = ring.at * S::kStep;
          ok = ok && warp_wait(&sm.full[s], ring.phase, abort_flag, a.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t k0 = kd + s * (kPair >> 4);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < (S::DK == 64 ? 4 : 8); ++k) {
              const uint32_t key = k0 + (k / 4) * (kColumn >> 4) + (k % 4) * 2, query = qd + (2 * i + k / 4) * (N * 128 >> 4) + (k % 4) * 2;
              mma_ss(d, S::kRowLanes ? query : key, hi, S::kRowLanes ? key : query, hi, idesc, (S::kLatent && !S::kAlias) || i > 0 || k > 0);
            }
            if (S::kSplit) umma_commit(&sm.empty[s]);
          }
          __syncwarp();
          ring.next();
        }
        if constexpr (S::kAlias) rotated();
        if (ok && elect_one()) umma_commit(&sm.s_full[sbuf.at]);
        __syncwarp();
        sbuf.next();
      }
    }
    if (elect_one()) {
      umma_commit(&sm.cleanup);
      wait_parity_bounded(&sm.cleanup, 0, nullptr, nullptr);
    }
    __syncwarp();
  } else if (warp == 2) {
    // =========================== O^T += V^T P^T ===========================
    constexpr uint32_t idesc = S::kRowLanes ? cosa::idesc_bf16_f32(128, DV, false, true) : cosa::idesc_bf16_f32(128, N, true, true);
    constexpr uint32_t v_hi = desc_hi(1024, 2), p_hi = desc_hi(8 * S::kPRow, S::kPRow == 128 ? 2 : S::kPRow == 64 ? 4 : 6);
    constexpr int kFirst = S::DK == 64 ? 1 : 0;      // columns of a slot from here on are values
    const uint32_t vd = desc_lo(smem_u32(sm.ring), kColumn), pd = desc_lo(S::kAlias ? smem_u32(sm.rope) : smem_u32(sm.p), kColumn);
    Ring<S::kRing> ring;
    Ring<S::kPBufs> pbuf;
    int tile = 0;
    bool ok = true;
    for (; ok && more; more = pieces.next(a, pc)) {
      const int32_t* table = a.page_table + static_cast<size_t>(pc.b) * a.max_pages_per_req;
      const int ctx = pc.r.len - pc.r.n;
      const bool differ = pc.r.n > 1 || a.tree_mask;      // the rows may differ in what they see
      bool begun = false;
      for (int t = pc.t0; t < pc.t1 && ok; ++t, ++tile) {
        // The product runs over the groups of 16 slots that have any (pages are whole groups); in the last of them the values
        // behind the sequence must be 0, since 0 times what is not finite is not.
        const int group0 = t * kTile + 16 * lane;
        bool has = lane < 8 && group0 < pc.r.len;
        if (has) {
          const int phys = __ldg(table + (group0 >> a.page_shift));
          has = phys >= 0 && phys < a.num_pages;
        }
        unsigned groups = __ballot_sync(kAll, has);
        int zero0 = min(pc.r.len - t * kTile, kTile), zero1 = (zero0 + 15) & ~15;      // rows to clear
        if (!(groups >> (zero1 / 16 - 1) & 1)) zero0 = zero1;
        if (groups == 0 && !begun) groups = 1, zero0 = 0, zero1 = 16;      // the output starts from something
        const int tail0 = differ ? max(ctx - t * kTile, 0) : kTile, tail1 = min(pc.r.len - t * kTile, kTile);
        const bool unclean = zero0 < zero1 || tail0 < tail1;
        bool found = false;
        // The values of a slot of the ring, as zeros where there are none or they are not finite (in the new tokens').
        auto clean = [&](uint8_t* values) {
          for (int e = zero0 * 16 + lane; e < zero1 * 16; e += 32)
            if ((e & 15) >= 8 * kFirst) *reinterpret_cast<uint4*>(values + (e & 15) / 8 * kColumn + (e >> 4) * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
          __syncwarp();
          for (int e = tail0 * 16 + lane; e < tail1 * 16; e += 32) {      // 16-byte pieces of the new tokens' values
            if ((e & 15) < 8 * kFirst) continue;
            uint4* at = reinterpret_cast<uint4*>(values + (e & 15) / 8 * kColumn + (e >> 4) * 128 + (e & 7) * 16);
            const uint4 x = *at;
            if (odd(x)) {
              found = true;
              *at = finite(x);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
        };
        // keys and values in one slot have been waited for by the first product already
        if (unclean || S::kSplit) {
          Ring<S::kRing> at = ring;
#pragma unroll
          for (int m = 0; m < S::kBlocks; ++m, at.next()) ok = ok && warp_wait(&sm.full[at.at * S::kStep + S::kStep - 1], at.phase, abort_flag, a.status);
        }
        ok = ok && warp_wait(&sm.p_full[pbuf.at], pbuf.phase, abort_flag, a.status);
        if (!ok) break;
        if (unclean) {
          Ring<S::kRing> at = ring;
#pragma unroll 1
          for (int m = 0; m < S::kBlocks; ++m, at.next()) clean(sm.ring[at.at * S::kStep + S::kStep - 1]);
        }
        tc_fence_after();
        const bool issue = elect_one();
        const uint32_t p0 = pd + pbuf.at * (S::kPBytes >> 4);
#pragma unroll
        for (int m = 0; m < S::kBlocks; ++m, ring.next()) {
          const int s = ring.at * S::kStep + S::kStep - 1;
          const uint32_t v0 = vd + s * (kPair >> 4);
          if (issue) {
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
              if (groups >> k & 1) {
                const bool add = begun || groups & ((1u << k) - 1);
                if constexpr (S::kRowLanes)
                  mma_ts(tmem + S::kTmemO, tmem + S::kTmemP + pbuf.at * (kTile / 2) + k * 8, v0 + kFirst * (kColumn >> 4) + k * (2048 >> 4), v_hi, idesc, add);
                else
                  mma_ss(tmem + S::kTmemO + m * N, v0 + k * (2048 >> 4), v_hi, p0 + k * S::kPRow, p_hi, idesc, add);
              }
            umma_commit(&sm.empty[s]);
          }
        }
        begun |= groups != 0;
        if (unclean) found = __any_sync(kAll, found);
        if (issue) {
          if (found) sm.odd_values = 1;
          if (S::kAlias) umma_commit(&sm.rope_empty[0]);
          umma_commit(&sm.pv_done[tile & 1]);
          mbar_arrive(&sm.pv_done[tile & 1]);
        }
        __syncwarp();
        pbuf.next();
      }
    }
    if (elect_one()) {
      umma_commit(&sm.cleanup);
      wait_parity_bounded(&sm.cleanup, 0, nullptr, nullptr);
    }
    __syncwarp();
  } else if (warp == 3) {
    // =========================== what is to be joined ===========================
    if (lane == 0 && !a.whole) {
      more = sm.start.any;      // whatever became of the call: join_kernel goes by what stands there
      Join none{}, mine{};
      const Shares shares(sm.start.total, a.walkers);
      for (; more; more = pieces.next(a, pc)) {
        if (!pc.begins) continue;
        Join j{};
        j.parts = 1;
        if (pc.slot >= 0 && pc.row_tile < pc.r.row_tiles) {
          j.parts = shares.owner(pc.item_end - 1) - cta / together_of<N>(a) + 1;
          j.first = pc.slot;
          j.next = 2 * (cta + together_of<N>(a));
          j.step = 2 * together_of<N>(a);
          j.tok0 = pc.r.tok0;
          j.rows = pc.r.n * a.group;
          j.head = pc.head;
          j.row_tile = pc.row_tile;
          mine = j;
        }
        const int entry = pc.item * together_of<N>(a) + cta % together_of<N>(a);
        if (entry < a.join_items) a.joins[entry] = j;
      }
      if (!a.join_items) a.joins[cta] = mine;
      else if (cta == 0)
        for (int i = sm.start.items * together_of<N>(a); i < a.join_items; ++i) a.joins[i] = none;
    }
    __syncwarp();
  } else {
    // =========================== softmax ===========================
    const int g = warp / 4 - 1, quarter = warp % 4, tid = threadIdx.x - 128;
    const int at = quarter * 32 + lane;                // TMEM lane: slot of the tile, value of an output block
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    constexpr int kSoftmax = 128 * S::kGroups;
    // Threads that share rows: a group has 16 rows (a thread a slot of the tile), or, kRowLanes, the warps of a quarter of the lanes,
    // one of each group, have 32 (a thread half of the slots).
    constexpr int kSharers = S::kRowLanes ? 32 * S::kGroups : 128, kParts = kSharers / 32;
    constexpr int kSlotsOf = kTile / S::kGroups, kWidth = DV / S::kGroups;      // kRowLanes: slots and values of a thread
    const int my_bar = 1 + (S::kRowLanes ? quarter : g);
    const int c0 = S::kRowLanes ? at : g * 16;         // first row
    const bool owns = S::kRowLanes ? g == 0 : at < 16;      // of those threads, the one that a row's reference, sum and result belong to,
    const int own = S::kRowLanes ? at : c0 + at;            // and the row
    const float scale = a.scale_log2;
    int tile = 0, meetings = 0;
    bool ok = true;
    // All groups meet; one that gave up does not come, so the wait is bounded.
    auto meet = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.groups);
      return warp_wait(&sm.groups, meetings++ & 1, abort_flag, a.status);
    };
    // What the products have left: `to(o, c, d)` for value d of each 16 rows from c on (kRowLanes: values d to d + 7 of row c).
    auto outputs = [&](bool odd_values, auto to) {
      const int32_t* table = a.page_table + static_cast<size_t>(pc.b) * a.max_pages_per_req;
      const int ctx = pc.r.len - pc.r.n;
      // what was not finite among the new tokens' values, for the rows that see it: `add(v, j)` for values d on of new token j
      auto odd_ones = [&](int d, auto add) {
        for (int s = max(ctx, pc.t0 * kTile); s < min(pc.r.len, pc.t1 * kTile); ++s) {
          const int phys = table[s >> a.page_shift];
          if (phys < 0 || phys >= a.num_pages) continue;
          const int64_t place = (static_cast<int64_t>(phys) << a.page_shift) + (s & ((1 << a.page_shift) - 1));
          add(S::kLatent ? a.k_cache + place * S::DK + d : a.v_cache + (place * a.num_kv_heads + pc.head) * DV + d, s - ctx);
        }
      };
      auto sees = [&](int c, int j) -> bool { return a.tree_mask ? sm.mask[c] >> j & 1 : j <= sm.node[c]; };
      auto plus = [](float& o, uint16_t v) {
        if ((v & 0x7F80) == 0x7F80) o += __uint_as_float(static_cast<uint32_t>(v) << 16);
      };
      tc_fence_after();
      if constexpr (S::kRowLanes) {
#pragma unroll 1
        for (int d = g * kWidth; d < (g + 1) * kWidth; d += 16) {
          float o[16] = {};
          __syncwarp();
          if (pc.t0 < pc.t1) load_columns<16>(tmem + lanes + S::kTmemO + d, o);
          if (odd_values)
            odd_ones(d, [&](const uint16_t* v, int j) {
              if (sees(at, j))
#pragma unroll
                for (int e = 0; e < 16; ++e) plus(o[e], v[e]);
            });
#pragma unroll
          for (int e = 0; e < 16; e += 8) to(*reinterpret_cast<const float(*)[8]>(&o[e]), at, d + e);
        }
      } else {
        constexpr int kSkip = DV == 64 ? 64 : 0;       // lanes of a block that are keys
#pragma unroll 1
        for (int m = 0; m < S::kBlocks; ++m) {
          const int d = m * 128 + at - kSkip;
          float o[16] = {};
          __syncwarp();
          if (pc.t0 < pc.t1) load_columns<16>(tmem + lanes + S::kTmemO + m * N + c0, o);
          if (d < 0) continue;
          if (odd_values)
            odd_ones(d, [&](const uint16_t* v, int j) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (sees(c0 + e, j)) plus(o[e], *v);
            });
          to(o, c0, d);
        }
      }
    };
    for (; ok && more; more = pieces.next(a, pc)) {
      const Request& r = pc.r;
      const int rows = r.n * a.group;      // fits 32 bits: total_tokens * Hq does
      if (together_of<N>(a) > 1 && pc.row_tile >= r.row_tiles) continue;
      const int row0 = pc.row_tile * N;
      if (!meet()) { ok = false; break; }      // the last piece is done with what follows
      if (tid < N) {
        const int row = row0 + tid, node = static_cast<uint32_t>(min(row, rows - 1)) / static_cast<uint32_t>(a.group);
        const int head = pc.head * a.group + row - node * a.group;
        sm.row[tid] = row < rows ? (r.tok0 + node) * a.num_q_heads + head : -1;
        sm.node[tid] = node;
        sm.q_at[tid] = row < rows ? (r.tok0 + node) * a.q_stride + head * a.q_head_stride : -1;
        if (S::kLatent) sm.r_at[tid] = (r.tok0 + node) * a.q_rope_stride + head * a.q_rope_head_stride;
        sm.mask[tid] = a.tree_mask ? static_cast<uint64_t>(__ldg(a.tree_mask + r.tok0 + node)) : 0;
        sm.base[tid] = -kNone;
      }
      if (pc.t0 < pc.t1) {
        // queries into rows of 128 bytes per 64 values, swizzled; rows behind the last are 0
        if (!meet()) { ok = false; break; }
        constexpr int kPieces16 = S::DK / 8;
#pragma unroll 3
        for (int e = tid; e < N * kPieces16; e += kSoftmax) {
          const int row = e / kPieces16, c = e % kPieces16;
          const int64_t at = sm.q_at[row];
          const uint16_t* src = S::kLatent && c >= DV / 8 ? a.q_rope + sm.r_at[row] + c * 8 - DV : a.q + at + c * 8;
          copy16(&sm.q[c / 8 * N * 128 + row * 128 + ((c ^ row) & 7) * 16], at < 0 ? a.q : src, at >= 0);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
      }
      if (!meet()) { ok = false; break; }
      if (tid == 0 && pc.t0 < pc.t1) mbar_arrive(&sm.q_ready);

      const int32_t* table = a.page_table + static_cast<size_t>(pc.b) * a.max_pages_per_req;
      const int ctx = r.len - r.n;
      float l[NC];                         // sums of this thread's slots
#pragma unroll
      for (int i = 0; i < NC; ++i) l[i] = 0.f;
      float ref = kNone;                   // kRowLanes: the row's reference (log2 units)
      // kRowLanes: pages of the thread's groups of 16 slots, one to a lane, a tile ahead
      auto look_up = [&](int t) {
        const int s = t * kTile + g * kSlotsOf + lane * 16;
        return S::kRowLanes && t < pc.t1 && lane < kSlotsOf / 16 && s < r.len ? __ldg(table + (s >> a.page_shift)) : -1;
      };
      int phys_next = look_up(pc.t0);
      for (int t = pc.t0; t < pc.t1; ++t, ++tile) {
        const int sb = tile & 1;
        // what the thread's slots are: one, or kSlotsOf with a bit each for those that the row sees
        const int slot = t * kTile + (S::kRowLanes ? g * kSlotsOf : at);
        bool there = false;
        uint64_t seen = 0;
        if constexpr (S::kRowLanes) {
          const bool page = phys_next >= 0 && phys_next < a.num_pages;
          phys_next = look_up(t + 1);
          const unsigned pages = __ballot_sync(kAll, page);      // of groups of 16 slots (pages are whole ones)
          seen = ones(r.len - slot);
#pragma unroll
          for (int k = 0; k < kSlotsOf / 16; ++k)
            if (!(pages >> k & 1)) seen &= ~(uint64_t{0xFFFF} << 16 * k);
          const int j = slot - ctx;               // the first slot as a new token, or before them
          if (j + kSlotsOf > 0) {
            uint64_t those;
            if (a.tree_mask) those = j >= 64 ? 0 : j >= 0 ? sm.mask[at] >> j : sm.mask[at] << -j;
            else those = ones(sm.node[at] + 1 - j);
            seen &= those | ones(-j);
          }
        } else {
          there = slot < r.len;
          if (there) {
            const int phys = __ldg(table + (slot >> a.page_shift));
            there = phys >= 0 && phys < a.num_pages;
          }
        }
        bool fail = !warp_wait(&sm.s_full[sb], (tile / 2) & 1, abort_flag, a.status);
        constexpr int kHave = S::kRowLanes ? kSlotsOf : 16;
        float x[kHave];                      // logits: the thread's row's slots, or its slot's 16 rows
        uint32_t w[kHave / 2];               // kRowLanes: weights as bf16
        float sum = 0.f;                     // and their sum
        // -infinity where the row does not see the slot
        auto logits = [&] {
          load_columns(tmem + lanes + S::kTmemS + sb * N + (S::kRowLanes ? g * kSlotsOf : c0), x);
          if constexpr (S::kRowLanes) {
            if (seen != ~uint64_t{0}) {
#pragma unroll
              for (int e = 0; e < kHave; ++e)
                if (!(seen >> e & 1)) x[e] = -INFINITY;
            }
          } else if (!there) {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = -INFINITY;
          } else if (slot >= ctx) {
            const int j = slot - ctx;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (a.tree_mask ? !(sm.mask[c0 + e] >> j & 1) : j > sm.node[c0 + e]) x[e] = -INFINITY;
          }
          __syncwarp();
        };
        // kRowLanes: exp2(x * scale - ref); whether one is high or NaN
        auto weights = [&] {
          uint32_t high = 0;
          float s4[4] = {};
#pragma unroll
          for (int e = 0; e < kHave / 2; ++e) {
            float x0, x1;
            cosa::fma2_bc(x0, x1, x[2 * e], x[2 * e + 1], scale, -ref);
            const float p0 = cosa::ex2_approx(x0), p1 = cosa::ex2_approx(x1);
            cosa::add2_acc(s4[(e & 1) * 2], s4[(e & 1) * 2 + 1], p0, p1);
            w[e] = cosa::pack_bf16x2(p0, p1);
            high = __vmaxu2(high, w[e]);
          }
          sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
          return (high & 0xFFFFu) > kHighBits || high >> 16 > kHighBits;
        };
        bool redo = t == pc.t0;      // no row has a reference yet
        if (!fail) {
          tc_fence_after();
          logits();
        }
        if (!redo) {
          // is some logit far above its row's reference (NaN is not: it stays what it is)
          bool high = false;
          if (fail) {
          } else if constexpr (S::kRowLanes) {
            high = weights();
          } else {
            float top = -INFINITY;
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 b = *reinterpret_cast<const float4*>(&sm.base[c0 + e]);
              float d[4];
              fma2(d[0], d[1], x[e], x[e + 1], scale, b.x, b.y);
              fma2(d[2], d[3], x[e + 2], x[e + 3], scale, b.z, b.w);
              top = fmaxf(top, fmaxf(fmaxf(d[0], d[1]), fmaxf(d[2], d[3])));
            }
            high = top > kHigh;
          }
          redo = named_bar_red_or(my_bar, kSharers, high || fail);
        }
        if (redo) {
          if (named_bar_red_or(my_bar, kSharers, fail)) { ok = false; break; }
          // the rows' maxima over the tile become references
          float mine = S::kRowLanes ? -INFINITY : 0.f;
          if constexpr (S::kRowLanes) {
            if (t > pc.t0) logits();       // (registers that live until here would be spilled)
#pragma unroll
            for (int e = 0; e < kHave; ++e) mine = fmaxf(mine, x[e]);
            sm.part[g][at] = mine;
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float top = warp_max(x[e]);
              mine = lane == e ? top : mine;
            }
            if (lane < 16) sm.part[quarter][c0 + lane] = mine;
          }
          named_bar_sync(my_bar, kSharers);
          auto move = [&](int c, float was, float& alpha) {      // the new reference
            float top = fmaxf(sm.part[0][c], sm.part[1][c]);
            if (kParts == 4) top = fmaxf(top, fmaxf(sm.part[2][c], sm.part[3][c]));
            const float now = top == -INFINITY ? was : fmaxf(was, top * scale);
            alpha = now == was ? 1.f : cosa::ex2_approx(was - now);
            return now;
          };
          float alpha = 1.f;               // kRowLanes: the row's
          if constexpr (S::kRowLanes) {
            ref = move(at, ref, alpha);
            weights();
          } else if (owns) {
            sm.base[own] = -move(own, -sm.base[own], sm.alpha[own]);
          }
          named_bar_sync(my_bar, kSharers);
          if (t > pc.t0) {
            if constexpr (S::kRowLanes) l[0] *= alpha;
            else
#pragma unroll
              for (int i = 0; i < NC; ++i) l[i] *= sm.alpha[c0 + i];
            fail = !warp_wait(&sm.pv_done[(tile - 1) & 1], ((tile - 1) / 2) & 1, abort_flag, a.status);
            if (!fail) {
              tc_fence_after();
              constexpr int kTimes = S::kRowLanes ? kWidth / 16 : S::kBlocks;
#pragma unroll 1
              for (int m = 0; m < kTimes; ++m) {
                const uint32_t o = tmem + lanes + S::kTmemO + (S::kRowLanes ? g * kWidth + m * 16 : m * N + c0);
                uint32_t v[16];
                cosa::tmem_ld16(o, v);
                cosa::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * (S::kRowLanes ? alpha : sm.alpha[c0 + e]));
                cosa::tmem_st16(o, v);
              }
              cosa::tmem_wait_st();
            }
          }
        }
        // P's buffer is free once the product before (or before that) has read it
        constexpr int kBack = S::kPBufs;
        if (!fail && tile >= kBack)
          fail = !warp_wait(&sm.pv_done[(tile - kBack) & 1], ((tile - kBack) / 2) & 1, abort_flag, a.status);
        if (!fail) {
          if constexpr (S::kRowLanes) {
            l[0] += sum;
            tc_fence_after();
            cosa::tmem_st32(tmem + lanes + S::kTmemP + (tile & 1) * (kTile / 2) + g * (kSlotsOf / 2), w);
            cosa::tmem_wait_st();
          } else {
            // exp2(x * scale - reference), summed, and as bf16 to P^T
            uint8_t* p = S::kAlias ? sm.rope[0] : sm.p[S::kPBufs == 2 ? tile & 1 : 0];
#pragma unroll
            for (int h = 0; h < 16; h += 8) {
              uint32_t y[4];
#pragma unroll
              for (int e = h; e < h + 8; e += 4) {
                const float4 b = *reinterpret_cast<const float4*>(&sm.base[c0 + e]);
                fma2(x[e], x[e + 1], x[e], x[e + 1], scale, b.x, b.y);
                fma2(x[e + 2], x[e + 3], x[e + 2], x[e + 3], scale, b.z, b.w);
#pragma unroll
                for (int k = e; k < e + 4; ++k) x[k] = cosa::ex2_approx(x[k]);
                cosa::add2_acc(l[e], l[e + 1], x[e], x[e + 1]);
                cosa::add2_acc(l[e + 2], l[e + 3], x[e + 2], x[e + 3]);
                y[(e - h) / 2] = cosa::pack_bf16x2(x[e], x[e + 1]);
                y[(e - h) / 2 + 1] = cosa::pack_bf16x2(x[e + 2], x[e + 3]);
              }
              *reinterpret_cast<uint4*>(p + p_offset<S::kPRow>(at, (c0 + h) / 8)) = make_uint4(y[0], y[1], y[2], y[3]);
            }
            fence_proxy_async_smem();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sm.p_full[S::kPBufs == 2 ? tile & 1 : 0]);
            mbar_arrive(&sm.s_empty[sb]);
          }
        }
        // a wait that ran out has set the abort flag: the next wait ends too, and its vote stops the group
      }
      if (!ok) break;
      // ---------------- the piece's end ----------------
      if constexpr (S::kRowLanes) {
        sm.part[g][at] = l[0];
        if (owns) sm.base[at] = -ref;
      } else {
        float mine = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          float s = l[i];
#pragma unroll
          for (int m = 1; m < 32; m *= 2) s += __shfl_xor_sync(kAll, s, m);
          mine = lane == i ? s : mine;
        }
        if (lane < NC) sm.part[quarter][c0 + lane] = mine;
      }
      bool fail = false;
      if (pc.t0 < pc.t1) fail = !warp_wait(&sm.pv_done[(tile - 1) & 1], ((tile - 1) / 2) & 1, abort_flag, a.status);
      if (named_bar_red_or(my_bar, kSharers, fail)) { ok = false; break; }
      if (a.cluster > 1) break;      // its one item is joined below
      if (owns) {
        const int c = own;
        const float sum = sm.part[0][c] + sm.part[1][c] + (kParts == 4 ? sm.part[2][c] + sm.part[3][c] : 0.f), m = -sm.base[c];
        if (pc.slot >= 0) {
          float* ml = a.part_ml + (static_cast<int64_t>(pc.slot) * N + c) * 2;
          ml[0] = m == kNone ? -INFINITY : m;
          ml[1] = sum;
        } else {
          sm.alpha[c] = sum == 0.f ? 0.f : 1.f / sum;
          if (a.lse && sm.row[c] >= 0) a.lse[sm.row[c]] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
        }
      }
      named_bar_sync(my_bar, kSharers);
      const bool odd_values = pc.t0 < pc.t1 && *reinterpret_cast<volatile int*>(&sm.odd_values);
      if (pc.t0 < pc.t1 || pc.slot < 0)
        outputs(odd_values, [&](const auto& o, int c, int d) {
          if (pc.slot >= 0) {
            float* to = a.part_o + (static_cast<int64_t>(pc.slot) * N + c) * DV + d;
            if constexpr (S::kRowLanes) {
              *reinterpret_cast<float4*>(to) = make_float4(o[0], o[1], o[2], o[3]);
              *reinterpret_cast<float4*>(to + 4) = make_float4(o[4], o[5], o[6], o[7]);
            } else
#pragma unroll
              for (int e = 0; e < 16; ++e) to[e * DV] = o[e];
          } else if constexpr (S::kRowLanes) {
            const float f = sm.alpha[c];
            if (sm.row[c] >= 0)
              *reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(sm.row[c]) * DV + d) =
                  make_uint4(cosa::pack_bf16x2(o[0] * f, o[1] * f), cosa::pack_bf16x2(o[2] * f, o[3] * f), cosa::pack_bf16x2(o[4] * f, o[5] * f),
                             cosa::pack_bf16x2(o[6] * f, o[7] * f));
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int row = sm.row[c + e];
              if (row >= 0) a.out[static_cast<int64_t>(row) * DV + d] = static_cast<uint16_t>(cosa::pack_bf16x2(o[e] * sm.alpha[c + e], 0.f));
            }
          }
        });
      tc_fence_before();
      if (odd_values) {        // the other threads have read it
        if (!meet()) { ok = false; break; }
        if (tid == 0) sm.odd_values = 0;
      }
    }
    if (a.cluster > 1) {
      // The cluster joins its item: the references and sums go to all of its CTAs, then each has a share of the values, to which the
      // others send theirs, weighted.  Every thread takes all three barriers: behind the first every CTA has started, so that its
      // shared memory may be written (one without tiles would be here before), behind the second the references are there and
      // the rings are free to receive, behind the third the shares are whole.
      const bool mine = works && ok;
      const int rank = cta % a.cluster, width = DV / a.cluster;
      cluster_wait();
      if (mine && owns) {
        const int c = own;
        const float sum = sm.part[0][c] + sm.part[1][c] + (kParts == 4 ? sm.part[2][c] + sm.part[3][c] : 0.f), m = -sm.base[c];
        for (int k = 0; k < a.cluster; ++k) store_remote(&sm.ml[rank][c], k, make_float2(m == kNone ? -INFINITY : m, sum));
      }
      cluster_barrier();
      float* parts = reinterpret_cast<float*>(sm.ring);      // [cluster][N][width]
      if (mine) {
        if (tid < N) {
          float m = -INFINITY, sum = 0.f;
#pragma unroll 8
          for (int k = 0; k < a.cluster; ++k) m = fmaxf(m, sm.ml[k][tid].x);
#pragma unroll 8
          for (int k = 0; k < a.cluster; ++k) {
            const float2 x = sm.ml[k][tid];
            sum += x.x == -INFINITY && x.y == 0.f ? 0.f : x.y * (x.x == -INFINITY ? 1.f : exp2f(x.x - m));
          }
          const float own = sm.ml[rank][tid].x;
          sm.alpha[tid] = sum == 0.f || own == -INFINITY ? (sum != sum ? sum : 0.f) : exp2f(own - m) / sum;
          if (a.lse && rank == 0 && sm.row[tid] >= 0) a.lse[sm.row[tid]] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
        }
        if (meet()) {
          const bool odd_values = pc.t0 < pc.t1 && *reinterpret_cast<volatile int*>(&sm.odd_values);
          outputs(odd_values, [&](const auto& o, int c, int d) {
            const uint32_t to = remote(parts + (rank * N + c) * width + d % width, d / width);      // (8 values: of one share)
            if constexpr (S::kRowLanes) {
              const float f = sm.alpha[c];
              if (sm.row[c] < 0) return;
              store_remote(to, o[0] * f, o[1] * f, o[2] * f, o[3] * f);
              store_remote(to + 16, o[4] * f, o[5] * f, o[6] * f, o[7] * f);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) store_remote(to + e * width * 4, o[e] * sm.alpha[c + e]);
            }
          });
        }
      }
      cluster_barrier();
      if (mine) {
        for (int e = tid; e < N * width / 2; e += kSoftmax) {
          const int c = e / (width / 2), d = e % (width / 2) * 2, row = sm.row[c];
          if (row < 0) continue;
          float x = 0.f, y = 0.f;
#pragma unroll 8
          for (int k = 0; k < a.cluster; ++k) {
            const float2 p = *reinterpret_cast<const float2*>(parts + (k * N + c) * width + d);
            x += p.x;
            y += p.y;
          }
          *reinterpret_cast<uint32_t*>(a.out + static_cast<int64_t>(row) * DV + rank * width + d) = cosa::pack_bf16x2(x, y);
        }
      }
    }
  }
  if (a.cluster > 1 && warp < 4) {
    cluster_wait();
    cluster_barrier();
    cluster_barrier();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    cosa::tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the items that several CTAs had: out = sum 2^(m_i - m) o_i / sum 2^(m_i - m) l_i.  blockIdx.x is an entry of
// `joins`; a block has eight rows of 128 values, or (kWide, where an item has many parts) one row, which its sixteen warps share.
constexpr int kJoinThreads = 256, kWideThreads = 512;

template <int N, int DV, bool kWide>
__global__ void __launch_bounds__(kWide ? kWideThreads : kJoinThreads) join_kernel(const __grid_constant__ Args a) {
  constexpr int kSeg = DV < 128 ? DV : 128, kVec = kSeg / 32;
  constexpr int kWarps = kWide ? kWideThreads / 32 : 1;          // that share a row
  constexpr int kAhead = kWide ? (kCtas + kWarps - 1) / kWarps : 4;      // parts of a warp in flight
  using Vec = typename std::conditional<kVec == 4, float4, float2>::type;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  cosa_kv::wait_for_stream();
  const Join j = a.joins[blockIdx.x];
  // (the bounds hold whatever another call might have made of the workspace; without sign, so that the sum does not wrap)
  if (j.parts < 2 || j.parts > kCtas || j.first < 0 || j.first >= 2 * kCtas || j.next < 0 || j.step < 0 ||
      j.step > 2 * kCtas || static_cast<uint32_t>(j.next) + j.step * (j.parts - 2) >= 2u * kCtas)
    return;
  const int parts = j.parts, seg = blockIdx.z;
  const int c = kWide ? blockIdx.y : blockIdx.y * 8 + warp;      // row of the tile
  const int64_t row = static_cast<int64_t>(j.row_tile) * N + c;
  if (row >= j.rows) return;                                     // (kWide: the whole block)
  auto slot = [&](int i) { return i == 0 ? j.first : j.next + j.step * (i - 1); };
  const float* base = a.part_o + static_cast<int64_t>(c) * DV + seg * kSeg + lane * kVec;
  // (volatile: else the compiler moves each load to its use)
  auto load = [&](int i) {
    Vec x{};
    const float* at = base + static_cast<int64_t>(slot(i)) * N * DV;
    if (i < parts) {
      if constexpr (kVec == 4) asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "l"(at));
      else asm volatile("ld.global.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "l"(at));
    }
    return x;
  };
  const int first = kWide ? warp : 0;
  // all loads at once: the first values of the parts, and their references and sums (a part to a lane)
  Vec v[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) v[k] = load(first + k * kWarps);
  constexpr int kLane = (kCtas + 31) / 32;
  float2 ml[kLane];
  float m = -INFINITY, sum = 0.f;
#pragma unroll
  for (int k = 0; k < kLane; ++k) {
    const int i = lane + 32 * k;
    ml[k] = i < parts ? *reinterpret_cast<const float2*>(a.part_ml + (static_cast<int64_t>(slot(i)) * N + c) * 2) : make_float2(-INFINITY, 0.f);
    m = fmaxf(m, ml[k].x);
  }
#pragma unroll
  for (int k = 1; k < 32; k *= 2) m = fmaxf(m, __shfl_xor_sync(kAll, m, k));
#pragma unroll
  for (int k = 0; k < kLane; ++k) {
    const bool none = ml[k].x == -INFINITY;                     // a part that saw nothing may have no values
    sum += none ? ml[k].y : exp2f(ml[k].x - m) * ml[k].y;
    ml[k].x = none ? -1.f : exp2f(ml[k].x - m);                  // its weight
  }
#pragma unroll
  for (int k = 1; k < 32; k *= 2) sum += __shfl_xor_sync(kAll, sum, k);
  float o[kVec] = {};
  auto add = [&](int i, const Vec& x) {
    float f = 0.f;
#pragma unroll
    for (int k = 0; k < kLane; ++k) {
      const float g = __shfl_sync(kAll, ml[k].x, i % 32);
      f = i / 32 == k ? g : f;
    }
    if (i >= parts || f < 0.f) return;
    const float* y = reinterpret_cast<const float*>(&x);
#pragma unroll
    for (int e = 0; e < kVec; ++e) o[e] = fmaf(f, y[e], o[e]);
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) add(first + k * kWarps, v[k]);
  for (int i = first + kAhead * kWarps; i < parts; i += kWarps) add(i, load(i));
  if constexpr (kWide) {
    __shared__ float sums[kWarps][kSeg];
#pragma unroll
    for (int e = 0; e < kVec; ++e) sums[warp][lane * kVec + e] = o[e];
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      o[e] = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) o[e] += sums[k][lane * kVec + e];
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t to = (j.tok0 + row / a.group) * a.num_q_heads + j.head * a.group + row % a.group;
  if (to < 0 || to >= static_cast<int64_t>(a.total_tokens) * a.num_q_heads) return;
  uint16_t* dst = a.out + to * DV + seg * kSeg + lane * kVec;
  if constexpr (kVec == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(cosa::pack_bf16x2(o[0] * inv, o[1] * inv), cosa::pack_bf16x2(o[2] * inv, o[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = cosa::pack_bf16x2(o[0] * inv, o[1] * inv);
  if (a.lse && seg == 0 && lane == 0) a.lse[to] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
}

// 24 requests of 52 rows: 168 us as 64 columns, 159 a row to a lane; of 24 rows: 152 as 32 columns, 156 a row to a lane.
int rows_of_tile(const PagedLaunch& L) {
  const int64_t rows = static_cast<int64_t>(L.max_new_tokens) * (L.num_q_heads / L.num_kv_heads);
  return rows <= 16 ? 16 : rows <= 32 ? 32 : L.latent_dim ? 64 : 128;
}

// Row tiles of the same keys that CTAs walk together, a CTA to a row tile, so that a tile of the cache is read from HBM once; the most
// that a request has (up to 8) if the average one has more than one less, since a CTA idles through a request with fewer.
int row_tiles_together(const PagedLaunch& L) {
  if (rows_of_tile(L) < 128) return 1;
  const int64_t n = rows_of_tile(L), group = L.num_q_heads / L.num_kv_heads;
  const int64_t most = (L.max_new_tokens * group + n - 1) / n, rounds = (most + 7) / 8;
  return L.total_tokens * group > L.num_reqs * (most - 1) * n ? static_cast<int>((most + rounds - 1) / rounds) : 1;
}

// At most so many (request, kv head, row tile): what the tokens fill and a part of a row tile for every request, or of `together`.
int64_t most_items(const PagedLaunch& L, int together) {
  return L.num_kv_heads * (L.total_tokens * static_cast<int64_t>(L.num_q_heads / L.num_kv_heads) / rows_of_tile(L) + L.num_reqs * static_cast<int64_t>(together));
}

template <class S>
cudaError_t launch_shape(const PagedLaunch& L, cudaStream_t stream) {
  Args a{};
  a.q = L.q;
  a.q_rope = L.q_rope;
  a.k_cache = L.k_cache;
  a.v_cache = L.v_cache;
  a.cu_seqlens = L.cu_seqlens;
  a.page_table = L.page_table;
  a.kv_len = L.kv_len;
  a.tree_mask = L.tree_mask;
  a.out = L.out;
  a.lse = L.lse;
  a.part_o = static_cast<float*>(L.workspace);
  a.part_ml = a.part_o + static_cast<size_t>(2 * kCtas) * S::N * S::DV;
  a.joins = reinterpret_cast<Join*>(a.part_ml + static_cast<size_t>(2 * kCtas) * S::N * 2);
  const int64_t group = L.num_q_heads / L.num_kv_heads, items = most_items(L, 1);
  a.status = L.status;
  a.q_stride = L.q_stride;
  a.q_head_stride = L.q_head_stride;
  a.q_rope_stride = L.q_rope_stride;
  a.q_rope_head_stride = L.q_rope_head_stride;
  a.num_reqs = L.num_reqs;
  a.num_q_heads = L.num_q_heads;
  a.num_kv_heads = L.num_kv_heads;
  a.group = static_cast<int>(group);
  a.page_shift = L.page_shift;
  a.total_tokens = L.total_tokens;
  a.max_seqlen = L.max_seqlen;
  a.num_pages = L.num_pages;
  a.max_pages_per_req = L.max_pages_per_req;
  a.scale_log2 = L.scale_log2;
  a.stall = L.stall;
  // the caches as (64 values, row of a page, 64-value column, head); a copy has the rows of a page
  CUtensorMap kmap, vmap;
  const uint64_t rows = static_cast<uint64_t>(L.num_pages) * L.page_size, pitch = static_cast<uint64_t>(S::kLatent ? 1 : L.num_kv_heads) * S::DK * 2;
  const uint64_t dims[4] = {64, rows, S::DK / 64, static_cast<uint64_t>(S::kLatent ? 1 : L.num_kv_heads)};
  const uint64_t strides[3] = {pitch, 128, S::DK * 2};
  const uint32_t box[4] = {64, static_cast<uint32_t>(L.page_size), 1, 1};
  if (!encode_bf16(&kmap, L.k_cache, dims, strides, box)) return cudaErrorInvalidValue;
  if (S::kLatent) vmap = kmap;
  else if (!encode_bf16(&vmap, L.v_cache, dims, strides, box)) return cudaErrorInvalidValue;

  const size_t smem = sizeof(Smem<S>) + 1024;
  static_assert(sizeof(Smem<S>) + 1024 <= 227 * 1024, "shared memory");
  auto* kernel = paged_kernel<S>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  a.cluster = 1;
  // How the items are shared, by the tiles that a CTA then has at most (lengths are known to the device only: max_seqlen's): all tiles
  // in one list, cut anywhere, and a second kernel to join (about kJoin tiles' time); whole items to a CTA; or an item to a cluster.
  // One token each, list / whole / cluster: 1 context of 900 (32 heads over 8 of 128) 10.3 / 11.7 / 8.9 us, 4 of 900 13.4 / 12.1 / 10.9,
  // 64 of 300 33.0 / 30.4 / -, 4 of 4000 22.3 / 28.3 / -; latent 512 of 16 heads: 9 of 900 14.6 / 26.2 / 13.2, 150 of 900 46.0 / 41.4 / -,
  // 200 of 900 62 / 69 / -.  Not always the best: one latent token after 900 11.8 / 25.9 / 12.6, 64 tokens after 900 17.3 / 16.4 / 18.5.
  // (19 clusters of eight, the most that there are, run at once: a call of them whose waits run out takes one wait's time.)
  // All of these have equal lengths, and what the rule knows is max_seqlen and an upper bound of the items.  A batch of other lengths can wait
  // for few long items where it takes whole ones or clusters (counted in tiles: 31 requests, one of 128K and thirty of 1000, 2050 to a CTA
  // where the list has 68), and where rows fill their row tile exactly the bound is twice the items, so that half of the card may idle.
  constexpr double kJoin = S::kLatent ? 2.5 : 5;
  const double tiles = (L.max_seqlen + kTile - 1) / kTile;
  double best = items * (tiles + 1) / kCtas + kJoin;
  if (std::ceil(static_cast<double>(items) / kCtas) * (tiles + 1) <= best) {
    best = std::ceil(static_cast<double>(items) / kCtas) * (tiles + 1);
    a.whole = 1;
  }
  for (int c = 2; c <= kMaxCluster; c *= 2)
    if (items * c <= kCtas && std::ceil(tiles / c) + 1 < best) {
      best = std::ceil(tiles / c) + 1;
      a.whole = 1;
      a.cluster = c;
    }
  a.together = a.cluster > 1 ? 1 : row_tiles_together(L);
  a.walkers = kCtas / a.together;
  const int64_t joins = most_items(L, a.together);
  a.join_items = joins <= kCtas ? static_cast<int>(joins) : 0;
  const unsigned ctas = static_cast<unsigned>(a.cluster > 1 ? items * a.cluster : kCtas);
  e = cosa_kv::launch_after(kernel, dim3(ctas), S::kThreads, smem, stream, a.cluster, kmap, vmap, a);
  if (e != cudaSuccess || a.whole) return e;
  const unsigned segs = S::DV < 128 ? 1 : S::DV / 128, x = static_cast<unsigned>(a.join_items ? a.join_items : kCtas);
  if (a.join_items && a.join_items <= 16)
    return cosa_kv::launch_after(join_kernel<S::N, S::DV, true>, dim3(x, S::N, segs), kWideThreads, 0, stream, 1, a);
  return cosa_kv::launch_after(join_kernel<S::N, S::DV, false>, dim3(x, S::N / 8, segs), kJoinThreads, 0, stream, 1, a);
}

template <int DK, int DV, bool LATENT>
cudaError_t launch_width(const PagedLaunch& L, cudaStream_t stream) {
  switch (rows_of_tile(L)) {
    case 16: return launch_shape<Shape<DK, DV, LATENT, 16>>(L, stream);
    case 32: return launch_shape<Shape<DK, DV, LATENT, 32>>(L, stream);
    default: return launch_shape<Shape<DK, DV, LATENT, LATENT ? 64 : 128>>(L, stream);
  }
}

}  // namespace

bool paged_fits(const PagedLaunch& L) { return most_items(L, row_tiles_together(L)) <= INT32_MAX / (int64_t{L.max_seqlen} / kTile + 2); }

size_t paged_workspace_bytes(const PagedLaunch& L) {
  const size_t dv = static_cast<size_t>(L.latent_dim ? L.latent_dim : L.head_dim);
  return static_cast<size_t>(2 * kCtas) * rows_of_tile(L) * (dv + 2) * sizeof(float) + kCtas * sizeof(Join);
}

cudaError_t launch_paged(const PagedLaunch& L, cudaStream_t stream) {
  if (L.latent_dim == 512) return launch_width<576, 512, true>(L, stream);
  if (L.latent_dim == 256) return launch_width<320, 256, true>(L, stream);
  return L.head_dim == 128 ? launch_width<128, 128, false>(L, stream) : launch_width<64, 64, false>(L, stream);
}

}  // namespace cosa_attn
