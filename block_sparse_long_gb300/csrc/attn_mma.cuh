// What both attention kernels of libcosa_attn use of the tensor core: descriptors in halves, products issued by one elected
// lane of a warp that runs as a whole, rings of barriers.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace cosa_attn {

constexpr unsigned kAll = 0xffffffffu;

// Shared-memory matrix descriptors in two halves; layout 2, 4, 6: 128-, 64-, 32-byte swizzle.  Offsets add to the low half.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr & 0x3FFFFu) >> 4 | (lbo >> 4) << 16; }
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo, int layout) { return sbo >> 4 | 1u << 14 | static_cast<uint32_t>(layout) << 29; }

// Issuing warps run as a whole and one elected lane issues: so their loop counters and descriptors are uniform, and a product
// costs them few instructions beside the softmax warps of the same scheduler (with the whole loop in one lane a product
// took 80 to 140 cycles to issue, twice what it takes to run).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// D[tmem] (+)= A[smem] * B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}

// A place in a ring of kCount barriers, and the parity of its use.
template <int kCount>
struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == kCount) at = 0, phase ^= 1;
  }
  __device__ __forceinline__ void back() {
    if (--at < 0) at = kCount - 1, phase ^= 1;
  }
};

// A bounded wait of a whole warp, which agrees on the outcome.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  return __all_sync(kAll, cosa::wait_parity_bounded(bar, parity, abort_flag, status));
}

// Whether a wait of this call has run out already: a CTA that starts then does nothing, since its waits would take as long again.
__device__ __forceinline__ bool gave_up(const int* status) {
  return status != nullptr && *static_cast<const volatile int*>(status) == cosa::kStatusDeviceTimeout;
}

// Of eight bf16 values: nonzero if one is not finite (its exponent, all ones, carries into the sign's place), and zeros for those.
__device__ __forceinline__ uint32_t odd(const uint4& x) {
  constexpr uint32_t kExp = 0x7F807F80u, kOne = 0x00800080u;
  return (((x.x & kExp) + kOne) | ((x.y & kExp) + kOne) | ((x.z & kExp) + kOne) | ((x.w & kExp) + kOne)) & 0x80008000u;
}
__device__ __forceinline__ uint32_t finite(uint32_t two) {
  const uint32_t bad = (((two & 0x7F807F80u) + 0x00800080u) & 0x80008000u) >> 15;      // 1 in the half that is not
  return two & ~(bad * 0xFFFFu);
}
__device__ __forceinline__ uint4 finite(const uint4& x) { return make_uint4(finite(x.x), finite(x.y), finite(x.z), finite(x.w)); }

}  // namespace cosa_attn
