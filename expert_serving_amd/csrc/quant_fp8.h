// The E4M3 code of a value and the scale of its block, shared by every kernel that
// makes 8-bit floating-point blocks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kFp8Block = 128;      // elements that share a scale along a product's K
constexpr float kFp8Max = 448.0f;   // the largest E4M3 value

// |v| as a word: the largest of a block's words is that of its largest magnitude, or
// of a NaN where the block holds one, whose scale is then a NaN too.
__device__ __forceinline__ uint32_t f8_magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// What a block of maximum magnitude amax needs for its codes 448 v / amax.
struct F8Block {
  float pre;   // power of two that keeps 448 v and 1 / amax inside fp32's normal range
  float amax;  // amax * pre
  float rcp;   // 1 / (amax * pre); 0 for a block of zeros, whose codes are then 0
};

__device__ __forceinline__ F8Block f8_block(float amax) {
  F8Block r;
  r.pre = amax > 1e30f ? 0x1p-16f : (amax < 1e-20f ? 0x1p60f : 1.0f);
  r.amax = amax * r.pre;
  r.rcp = r.amax > 0.f ? 1.0f / r.amax : 0.f;
  return r;
}

__device__ __forceinline__ float f8_scale(float amax) { return amax / kFp8Max; }

// 448 v / amax to its last bit (ties of the codes' rounding occur in earnest: a
// maximum whose significand is a multiple of 7 leaves many), as a product with the
// reciprocal that the remainder corrects once; within +-448.
__device__ __forceinline__ float f8_quotient(float v, const F8Block& b) {
  const float x = v * b.pre;
  const float t = kFp8Max * x;
  const float q0 = t * b.rcp;
  const float rest = fmaf(-q0, b.amax, t) + fmaf(kFp8Max, x, -t);
  return fminf(fmaxf(fmaf(rest, b.rcp, q0), -kFp8Max), kFp8Max);
}

// The same for values that carry roundings of their own (h of an FFN), where the last
// bit of the quotient decides nothing that they do not: one product.  The powers of two
// are f8_block's: the reciprocal instruction returns 0 for a maximum above 2^126.
struct F8Near {
  float pre, factor;  // 448 / (amax * pre); 0 for a block of zeros
};
__device__ __forceinline__ F8Near f8_near(float amax) {
  F8Near r;
  r.pre = amax > 1e30f ? 0x1p-16f : (amax < 1e-20f ? 0x1p60f : 1.0f);
  const float x = amax * r.pre;
  r.factor = x > 0.f ? kFp8Max * __builtin_amdgcn_rcpf(x) : 0.f;
  return r;
}
__device__ __forceinline__ float f8_code(float v, const F8Near& b) {
  return __builtin_amdgcn_fmed3f((v * b.pre) * b.factor, -kFp8Max, kFp8Max);
}

// A scale 2^e m with m in [1, 2): the word with its exponent in the top byte, which the
// matrix units take as E8M0 (a scale below fp32's normal range counts as 2^-127 m), and
// m, from the scale's word or from that one.
__device__ __forceinline__ int f8_exponent(uint32_t scale) { return (int)(scale << 1); }
__device__ __forceinline__ float f8_unit(uint32_t scale) { return __uint_as_float((scale & 0x007FFFFFu) | 0x3F800000u); }
__device__ __forceinline__ float f8_unit_of(int e) { return f8_unit((uint32_t)e >> 1); }

// four quotients to four E4M3 bytes, nearest, ties to even
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d) {
  int p = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  p = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, p, true);
  return (uint32_t)p;
}

}  // namespace moe
