// Scales of the 8-bit forms (blocks of 32 of the optimizer states, blocks of
// 128 of matrices), device code shared by their units.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace zdp {

__device__ __forceinline__ uint32_t bits_of(float x) { return __builtin_bit_cast(uint32_t, x); }
__device__ __forceinline__ float float_of(uint32_t x) { return __builtin_bit_cast(float, x); }

// Scale byte of a block whose largest magnitude has the bits `big`: the
// exponent, one more where the mantissa passes 448 = 1.75 * 2^8.  255 for a
// block that holds an inf or a NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t big) {
    int e = static_cast<int>((big + 0x1FFFFFu) >> 23) - 8;
    e = e < 1 ? 1 : e;
    return big >= 0x7F800000u ? 255u : static_cast<uint32_t>(e);
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
    const uint32_t bits = byte == 255u ? 0x7FC00000u : byte == 0u ? 0x00400000u : byte << 23;
    return __builtin_bit_cast(float, bits);
}

}  // namespace zdp
