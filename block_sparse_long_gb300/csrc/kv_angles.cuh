// Angles of position rotations, reduced to half turns (for sincospif) before they are rounded to fp32.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace cosa_kv {

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

}  // namespace cosa_kv
