// A value rounded to a 16-bit type, nearest, ties to even, as the bits of its word.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

__device__ __forceinline__ uint32_t f16_bits(float f) { return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f); }

__device__ __forceinline__ uint32_t bf16_bits(float f) {
  const uint32_t b = __float_as_uint(f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return (b >> 16) | 0x40u;  // NaN stays NaN
  return (b + (((b >> 16) & 1u) + 0x7FFFu)) >> 16;
}

}  // namespace moe
