// K and V into the 4-bit cache and back (layout: include/cosa_kv.h).
//
// Per group of 32 values:  s = bf16(max|x| / 7),  c = clamp(rint(x / s), -7, 7).  Four lanes have a row (token,
// head): lane c of them holds values 32 g + 8 c .. + 7 of every group g, of K and of V, which are 16 (d = 128) or
// 8 (d = 64) neighbouring bytes of the row's K codes and of its V codes; the four lanes of a group share its
// largest magnitude by two shuffles.  Both directions are memory bound: 4 d bytes of bf16 and
// 9/8 d bytes of cache per token and kv head.
//
// Measured: 32K tokens of 8 heads of 128 stored in 34 us (172 MB at 5.1 TB/s, 75 % of the measured copy rate; the issue slots
// are 69 % busy with the rounding) and loaded in 28 us (6.1 TB/s); 243K tokens of four ragged requests loaded in 224 us
// (6.4 TB/s, 94 %).  One lane for eight values, with divisions and 2- and 4-byte stores, took 81 us and 43 us for the 32K.
#include <algorithm>
#include <cstdint>

#include "cosa_kv.h"
#include "kv_internal.h"
#include "kv_layout.cuh"

namespace cosa_kv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;     // tokens of a CTA (a storage tile: its slots share their pages)

// Codes of eight values, lowest nibble first: nibble n of each half has the magnitude of value n, and the sign of
// value n ^ 2 in its high bit.
//
// rint(x / s) without a division: x / s is formed to 2^-21 by the reciprocal and rounded to a multiple of 2^-10 by
// being added to 1.5 * 2^13.  Significands of 8 bits make a quotient that lies on a border k + 1/2 or at least 1/512
// from it (2 X 2^e - (2 k + 1) S is a whole multiple of 1/2 where it is not zero, over 2 S <= 510), so this first
// rounding puts every tie on its border exactly and moves nothing across one.  A second addition, to 1.5 * 2^23
// in all, rounds to even and leaves the code in the low bits; the eight words are summed with weights 16^i.
__device__ __forceinline__ uint32_t codes8(const uint4& u, float inv) {
  float x[8];
  unpack8(u, x);
  uint32_t sum = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    sum += __float_as_uint(fmaf(x[i], inv, 12288.0f) + (12582912.0f - 12288.0f)) << (4 * i);
  // sum_i (0x4B400000 + c_i) 16^i: without the constant, and with 8 in each nibble, the nibbles are c + 8
  uint32_t bias = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) bias += 0x4B400000u << (4 * i);
  const uint32_t c = (sum - bias + 0x88888888u) ^ 0x88888888u;       // two's complement in each nibble
  const uint32_t neg = (c >> 3) & 0x11111111u;
  const uint32_t mag = (c ^ (neg * 15u)) + neg;                       // no carry: the codes are -7 .. 7
  return mag | __byte_perm(neg << 3, 0, 0x2301);                      // the bytes of a half hold nibbles 0, 1 and 2, 3
}

// The same by the division, for scales whose reciprocal or codes leave the range (near the ends of bf16's).
__device__ __noinline__ uint32_t codes8_slow(uint4 u, float s) {
  float x[8];
  unpack8(u, x);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = static_cast<int>(fminf(fmaxf(rintf(x[i] / s), -7.f), 7.f));
    w |= static_cast<uint32_t>(abs(c)) << (4 * i);
    if (c < 0) w |= 8u << (4 * (i ^ 2));
  }
  return w;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The larger magnitudes of two pairs of bf16 numbers (NaN above every number; the signs mean nothing).
__device__ __forceinline__ uint32_t max_abs2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// Codes of eight values of a group whose largest magnitude has the bits m, and the bits of its scale.
__device__ __forceinline__ uint32_t quantise8(const uint4& u, uint32_t m, uint32_t& scale) {
  if (m >= 0x7F80u) {
    scale = 0x7FC0u;
    return 0u;
  }
  // max|x| / 7 by the reciprocal: the quotient of an 8-bit significand is never halfway between two bf16 numbers (7 times
  // an odd 9-bit one is odd and above 255), nor nearer to it than 2^-12 of itself, so the product's 2^-23 does not matter
  scale = cosa::pack_bf16x2(__uint_as_float(m << 16) * (1.0f / 7.0f), 0.f) & 0xFFFFu;
  if (scale >= 0x0400u && scale < 0x7C00u) return codes8(u, rcp_approx(__uint_as_float(scale << 16)));     // 2^-119 <= s < 2^121
  // near the ends of the range, subnormal scales among them
  scale = cosa::pack_bf16x2(__uint_as_float(m << 16) / 7.0f, 0.f) & 0xFFFFu;
  return scale == 0u ? 0u : codes8_slow(u, __uint_as_float(scale << 16));
}

// Codes of a lane's values of K and V, a word per group, and the bits of the groups' scales.  Every lane of the warp calls
// it: the four lanes of a group find its largest magnitude, of K in the low half of a word and of V in the high half.
template <int G>
__device__ __forceinline__ void quantise(const uint4 (&ku)[G], const uint4 (&vu)[G], uint32_t (&kw)[G], uint32_t (&ks)[G],
                                         uint32_t (&vw)[G], uint32_t (&vs)[G]) {
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const uint32_t k = max_abs2(max_abs2(ku[g].x, ku[g].y), max_abs2(ku[g].z, ku[g].w));
    const uint32_t v = max_abs2(max_abs2(vu[g].x, vu[g].y), max_abs2(vu[g].z, vu[g].w));
    uint32_t m = max_abs2(__byte_perm(k, v, 0x5410), __byte_perm(k, v, 0x7632));
    m = max_abs2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max_abs2(m, __shfl_xor_sync(0xffffffffu, m, 2)) & 0x7FFF7FFFu;
    kw[g] = quantise8(ku[g], m & 0xFFFFu, ks[g]);
    vw[g] = quantise8(vu[g], m >> 16, vs[g]);
  }
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("sub.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// Eight values from their codes and `scale` (the bf16 scale in both halves).  The two magnitudes of a byte become the
// bf16 numbers 128 + m (low bits of the significand) and 8 + m (high bits), less 128 and 8; the product with the scale is
// rounded once.
__device__ __forceinline__ uint4 dequantise8(uint32_t w, uint32_t scale) {
  uint32_t y[4];
  const uint32_t w4 = w << 4;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t x = (__byte_perm(w, 0, k | (4 << 4) | (k << 8) | (4 << 12)) & 0x00700007u) | 0x41004300u;
    // signs of values 2k and 2k + 1: bits 3 and 7 of byte k ^ 1
    const uint32_t sign = __byte_perm(w4, w, ((k ^ 1) << 4) | ((4 + (k ^ 1)) << 12)) & 0x80008000u;
    y[k] = mul_bf16x2(sub_bf16x2(x, 0x41004300u), scale) ^ sign;
  }
  return make_uint4(y[0], y[1], y[2], y[3]);
}

// A lane's share of a row of K codes is one piece of the row; of a row of V codes too.
template <int D>
__device__ __forceinline__ void store_piece(uint8_t* at, const uint32_t (&w)[Tile<D>::G]) {
  if constexpr (Tile<D>::G == 4)
    *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
  else
    *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
}

template <int D>
__device__ __forceinline__ void load_piece(const uint8_t* at, uint32_t (&w)[Tile<D>::G]) {
  if constexpr (Tile<D>::G == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(at);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(at);
    w[0] = u.x; w[1] = u.y;
  }
}

// Between a word per group and the V order: 16-bit words i * G + g for i = 2c, then for i = 2c + 1.
template <int G>
__device__ __forceinline__ void to_v_order(const uint32_t (&w)[G], uint32_t (&v)[G]) {
#pragma unroll
  for (int g = 0; g < G; g += 2) {
    v[g / 2] = __byte_perm(w[g], w[g + 1], 0x5410);
    v[G / 2 + g / 2] = __byte_perm(w[g], w[g + 1], 0x7632);
  }
}
template <int G>
__device__ __forceinline__ void from_v_order(const uint32_t (&v)[G], uint32_t (&w)[G]) {
#pragma unroll
  for (int g = 0; g < G; g += 2) {
    w[g] = __byte_perm(v[g / 2], v[G / 2 + g / 2], 0x5410);
    w[g + 1] = __byte_perm(v[g / 2], v[G / 2 + g / 2], 0x7632);
  }
}

// A row's codes and scales into token t of its tile (lane c of the row's four).
template <int D>
__device__ __forceinline__ void put(uint8_t* tile, int t, int c, const uint32_t (&kw)[Tile<D>::G], const uint32_t (&ks)[Tile<D>::G],
                                    const uint32_t (&vw)[Tile<D>::G], const uint32_t (&vs)[Tile<D>::G]) {
  using T = Tile<D>;
  constexpr int G = T::G;
  store_piece<D>(tile + t * T::kRow + c * 4 * G, kw);
  uint32_t v[G];
  to_v_order<G>(vw, v);
  store_piece<D>(tile + T::kVCodes + v_row(t) * T::kRow + c * 4 * G, v);
  if (c < 2) {                                 // lane 0 writes the K scales, lane 1 the V scales
    uint8_t* at = tile + (c ? T::kVScales : T::kKScales) + t * G * 2;
    uint32_t two[G / 2];
#pragma unroll
    for (int g = 0; g < G; g += 2) two[g / 2] = c ? vs[g] | (vs[g + 1] << 16) : ks[g] | (ks[g + 1] << 16);
    if constexpr (G == 4)
      *reinterpret_cast<uint2*>(at) = make_uint2(two[0], two[1]);
    else
      *reinterpret_cast<uint32_t*>(at) = two[0];
  }
}

template <int G>
__device__ __forceinline__ void load_row(const uint16_t* src, int c, bool in, uint4 (&u)[G]) {
#pragma unroll
  for (int g = 0; g < G; ++g) u[g] = in ? *reinterpret_cast<const uint4*>(src + 32 * g + 8 * c) : make_uint4(0, 0, 0, 0);
}

// Slots first .. end - 1 of request b; a contradiction gives an empty range and the status.
__device__ __forceinline__ Range slots_of(const ConvertLaunch& L, int b, int len, int from) {
  Range r{from, len, true};
  if (from < 0 || len < 0 || len > L.max_seqlen) r = Range{0, 0, false};
  return r;
}

__device__ __forceinline__ int page_of(const int32_t* table, const ConvertLaunch& L, int b, int slot, int pages) {
  const int phys = table[static_cast<size_t>(b) * L.max_pages_per_req + (slot >> L.page_shift)];
  return phys >= 0 && phys < pages ? phys : -1;
}

// Rows packed by cu_seqlens; a CTA takes `tokens` tokens of the batch.
template <int D>
__global__ void __launch_bounds__(kThreads) store_rows_kernel(const ConvertLaunch L, const int tokens) {
  constexpr int G = Tile<D>::G;
  __shared__ int s_slot[kMaxTokens], s_phys[kMaxTokens];
  const int tid = threadIdx.x;
  wait_for_stream();
  const int t0 = blockIdx.x * tokens;
  const int last = L.cu_seqlens[L.num_reqs];
  if (blockIdx.x == 0 && tid == 0 && (L.cu_seqlens[0] != 0 || last > L.total_tokens))
    cosa::report_status(L.status, cosa::kStatusBadInput);
  const int ntok = min(tokens, min(last, L.total_tokens) - t0);
  if (ntok <= 0) return;
  for (int j = tid / 32; j < ntok; j += blockDim.x / 32) {
    const int t = t0 + j, lane = tid % 32;
    int b = 0;
    for (int i = lane; i < L.num_reqs; i += 32) b += L.cu_seqlens[i + 1] <= t;
    b = __reduce_add_sync(0xffffffffu, b);
    if (lane == 0) {
      const int off = b < L.num_reqs ? t - L.cu_seqlens[b] : -1;
      const int64_t slot = off < 0 ? -1 : static_cast<int64_t>(off) + (L.start ? L.start[b] : 0);
      const bool fits = slot >= 0 && slot < L.max_seqlen;
      if (!fits) cosa::report_status(L.status, cosa::kStatusBadInput);
      s_slot[j] = fits ? static_cast<int>(slot) : 0;
      s_phys[j] = fits ? page_of(L.page_table, L, b, static_cast<int>(slot), L.num_kv4_pages) : -1;
    }
  }
  __syncthreads();
  const int c = tid % 4;
  const int rows = ntok * L.num_kv_heads;
  for (int r0 = 0; r0 < rows; r0 += blockDim.x / 4) {     // uniform: the shuffles need every lane
    const int r = r0 + tid / 4;
    const bool in = r < rows;
    const int j = in ? r / L.num_kv_heads : 0;
    const int h = in ? r - j * L.num_kv_heads : 0;
    const int64_t t = t0 + j;
    uint4 ku[G], vu[G];
    load_row<G>(L.k + t * L.k_stride + static_cast<int64_t>(h) * D, c, in, ku);
    load_row<G>(L.v + t * L.v_stride + static_cast<int64_t>(h) * D, c, in, vu);
    uint32_t kw[G], ks[G], vw[G], vs[G];
    quantise<G>(ku, vu, kw, ks, vw, vs);
    if (in && s_phys[j] >= 0)
      put<D>(L.cache + tile_offset<D>(s_phys[j], h, s_slot[j], L.num_kv_heads, L.page_shift), s_slot[j] % kTile, c, kw, ks,
             vw, vs);
  }
}

// Pages to pages: the CTAs of request blockIdx.y take `tokens` slots at a time.  LOAD: from the cache to bf16 pages.
template <int D, bool LOAD>
__global__ void __launch_bounds__(kThreads) pages_kernel(const ConvertLaunch L, const int tokens) {
  using T = Tile<D>;
  constexpr int G = T::G;
  const int tid = threadIdx.x;
  const int b = blockIdx.y;
  wait_for_stream();
  const Range range = slots_of(L, b, L.kv_len[b], L.start ? L.start[b] : 0);
  if (!range.ok && blockIdx.x == 0 && tid == 0) cosa::report_status(L.status, cosa::kStatusBadInput);
  const int c = tid % 4;
  const int rows = tokens * L.num_kv_heads;
  // from the tile boundary at or before the first slot
  for (int64_t s0 = range.first / kTile * kTile + static_cast<int64_t>(blockIdx.x) * tokens; s0 < range.end;
       s0 += static_cast<int64_t>(gridDim.x) * tokens) {
    const int slot0 = static_cast<int>(s0);
    const int p4 = page_of(L.page_table, L, b, slot0, L.num_kv4_pages);
    const int p16 = page_of(L.other_table, L, b, slot0, L.num_pages);
    if (p4 < 0 || p16 < 0) continue;
    for (int r0 = 0; r0 < rows; r0 += blockDim.x / 4) {     // uniform: the shuffles need every lane
      const int r = r0 + tid / 4;
      const int j = r < rows ? r / L.num_kv_heads : 0;
      const int h = r < rows ? r - j * L.num_kv_heads : 0;
      const int slot = slot0 + j;
      const bool in = r < rows && slot >= range.first && slot < range.end;
      const size_t at = ((static_cast<size_t>(p16) * L.page_size + (slot & ((1 << L.page_shift) - 1))) * L.num_kv_heads + h) * D;
      uint8_t* tile = L.cache + tile_offset<D>(p4, h, slot, L.num_kv_heads, L.page_shift);
      const int t = slot % kTile;
      if (LOAD) {
        if (!in) continue;
        uint32_t kw[G], v[G], vw[G];
        load_piece<D>(tile + t * T::kRow + c * 4 * G, kw);
        load_piece<D>(tile + T::kVCodes + v_row(t) * T::kRow + c * 4 * G, v);
        from_v_order<G>(v, vw);
        const uint32_t* ks = reinterpret_cast<const uint32_t*>(tile + T::kKScales + t * G * 2);
        const uint32_t* vs = reinterpret_cast<const uint32_t*>(tile + T::kVScales + t * G * 2);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const uint32_t both = g % 2 ? 0x3232 : 0x1010;      // the group's scale in both halves
          *reinterpret_cast<uint4*>(L.k_cache + at + 32 * g + 8 * c) = dequantise8(kw[g], __byte_perm(ks[g / 2], 0, both));
          *reinterpret_cast<uint4*>(L.v_cache + at + 32 * g + 8 * c) = dequantise8(vw[g], __byte_perm(vs[g / 2], 0, both));
        }
      } else {
        uint4 ku[G], vu[G];
        load_row<G>(L.k + at, c, in, ku);
        load_row<G>(L.v + at, c, in, vu);
        uint32_t kw[G], ks[G], vw[G], vs[G];
        quantise<G>(ku, vu, kw, ks, vw, vs);
        if (in) put<D>(tile, t, c, kw, ks, vw, vs);
      }
    }
  }
}

}  // namespace

namespace {

// Four threads per row: a CTA of tokens that fill 256 of them, 16 where the heads are few.  8 heads of 128, CTAs of 8 tokens
// instead of 16: 5000 rows stored in 7.5 us instead of 8.3, 32K loaded in 28.0 us instead of 29.1 (but 200K rows stored in
// 189 us instead of 180); 2 heads of 64, 16 instead of 8: 128K loaded in 12.6 us instead of 13.2.
struct Shape {
  int tokens, threads;
  explicit Shape(int heads)
      : tokens(heads >= 8 ? 8 : kMaxTokens), threads((std::min(kThreads, 4 * tokens * heads) + 31) / 32 * 32) {}
};

// CTAs per request: one for each group of tokens, but no more than 32 per SM over the batch, so that requests much
// shorter than max_seqlen (or a late `start`) leave few CTAs without work (0.6 ns each).  With no bound 32 requests of 1000 tokens
// in tables for 128K load in 265 us instead of 28.  With 32 / 64 / 128 per SM: 4 requests of 64K load in 215 / 207 / 203 us and
// are stored in 207 / 210 / 213, those 32 load in 27.7 / 28.9 / 31.3 us and are stored in 31.6 / 34.6 / 39.9.
dim3 pages_grid(const ConvertLaunch& L, int tokens) {
  const int64_t most = std::max<int64_t>(1, 32 * 152 / L.num_reqs);
  return dim3(static_cast<unsigned>(std::min<int64_t>(most, (static_cast<int64_t>(L.max_seqlen) + tokens - 1) / tokens)),
              static_cast<unsigned>(L.num_reqs));
}

template <bool LOAD>
cudaError_t launch_pages(const ConvertLaunch& L, cudaStream_t stream) {
  const Shape s(L.num_kv_heads);
  return launch_after(L.head_dim == 128 ? pages_kernel<128, LOAD> : pages_kernel<64, LOAD>, pages_grid(L, s.tokens), s.threads, 0,
                      stream, 1, L, s.tokens);
}

}  // namespace

cudaError_t launch_store_rows(const ConvertLaunch& L, cudaStream_t stream) {
  const Shape s(L.num_kv_heads);
  // few rows: a token per CTA (8 heads: 64 tokens 3.4 us instead of 3.8, 1000 4.8 instead of 5.0; with 2 heads of 64 5000 tokens
  // would take 6.6 us instead of 4.5)
  const int tokens = L.total_tokens <= 8 * 152 ? 1 : s.tokens;
  const int threads = std::min(s.threads, (4 * tokens * L.num_kv_heads + 31) / 32 * 32);
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(L.total_tokens) + tokens - 1) / tokens);
  return launch_after(L.head_dim == 128 ? store_rows_kernel<128> : store_rows_kernel<64>, dim3(grid), threads, 0, stream, 1, L,
                      tokens);
}

cudaError_t launch_store_pages(const ConvertLaunch& L, cudaStream_t stream) { return launch_pages<false>(L, stream); }

cudaError_t launch_load(const ConvertLaunch& L, cudaStream_t stream) { return launch_pages<true>(L, stream); }

}  // namespace cosa_kv
