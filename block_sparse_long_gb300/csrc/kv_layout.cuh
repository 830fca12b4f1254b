// The 4-bit cache layout (include/cosa_kv.h) and the small device helpers its kernels share.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace cosa_kv {

constexpr int kTile = 16;    // tokens of a storage tile
constexpr int kGroup = 32;   // values that share a scale

// Byte offsets inside a tile of 16 tokens of one kv head.
template <int D>
struct Tile {
  static constexpr int G = D / kGroup;          // scales per token
  static constexpr int kRow = D / 2;            // bytes of a token's codes
  static constexpr int kVCodes = kTile * kRow;
  static constexpr int kKScales = 2 * kTile * kRow;
  static constexpr int kVScales = kKScales + kTile * G * 2;
  static constexpr int kBytes = kVScales + kTile * G * 2;   // 18 D
};

// Row of token t of a tile among its V codes: tokens 2c and 2c + 1, which a lane of the second matrix
// product takes together, are eight rows apart, so that the four lanes' rows are neighbours (no bank conflicts).
__device__ __forceinline__ int v_row(int t) { return (t & 1) * 8 + (t >> 1); }

// First byte of the tile of `slot` of (physical page, kv head).
template <int D>
__device__ __forceinline__ size_t tile_offset(int phys, int kvh, int slot, int num_kv_heads, int page_shift) {
  const int tile = (slot & ((1 << page_shift) - 1)) / kTile;
  return (((static_cast<size_t>(phys) * num_kv_heads + kvh) << (page_shift - 4)) + tile) * Tile<D>::kBytes;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Eight bf16 values to fp32 and back (rounded to nearest even).
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
  x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z); x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(cosa::pack_bf16x2(x[0], x[1]), cosa::pack_bf16x2(x[2], x[3]), cosa::pack_bf16x2(x[4], x[5]),
                    cosa::pack_bf16x2(x[6], x[7]));
}

// Kernels of this library are launched while the kernel before them on the stream still runs (its last CTAs, or all of
// it where it allows), so that their launch costs no time of its own.  wait_for_stream() ends when that kernel has ended
// and its writes are visible; every thread calls it before anything else.  let_next_start() allows it to the next one.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

struct Range {
  int first, end;
  bool ok;
};

}  // namespace cosa_kv
