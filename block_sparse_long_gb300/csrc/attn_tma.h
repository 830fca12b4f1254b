// Tensor maps of libcosa_attn: bf16 tensors of four dimensions, 128-byte swizzle.
#pragma once

#include <cstdint>
#include <cuda.h>

namespace cosa_attn {

// dims and box from the innermost, strides in bytes of dimensions 1 to 3.  False if the driver refuses.
bool encode_bf16(CUtensorMap* map, const void* base, const uint64_t (&dims)[4], const uint64_t (&strides)[3], const uint32_t (&box)[4]);

}  // namespace cosa_attn
