// The int8 code of a value, shared by every kernel that quantises rows.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// |v| as a word.  The largest of a row's words is that of its largest magnitude,
// or of a NaN where the row holds one (a NaN's is above infinity's), so that a row
// that is not finite gets a scale that is not: products of its unspecified codes
// are then no plausible numbers.
__device__ __forceinline__ uint32_t i8_magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// What a row of maximum magnitude amax needs for its codes 127 v / amax.
struct I8Row {
  float pre;   // power of two that keeps 127 v and 1 / amax inside fp32's normal range
  float amax;  // amax * pre
  float rcp;   // 1 / (amax * pre); 0 for a row of zeros, whose codes are then 0
};

__device__ __forceinline__ I8Row i8_row(float amax) {
  I8Row r;
  r.pre = amax > 1e30f ? 0x1p-16f : (amax < 1e-20f ? 0x1p60f : 1.0f);
  r.amax = amax * r.pre;
  r.rcp = r.amax > 0.f ? 1.0f / r.amax : 0.f;
  return r;
}

// rint(127 v / amax), ties to even, in [-127, 127].  Half of the maximum is a
// tie (63.5) and occurs in earnest, so the quotient has to be right to its last
// bit: a product with the reciprocal, corrected once by the remainder of the
// unrounded 127 v (both exact in fused multiply-adds).  Six operations where
// a division takes about ten.  For bf16 and fp16 v every quotient that is no
// tie is at least 9e-7 away from one, so the codes are those of exact arithmetic.
__device__ __forceinline__ int i8_code(float v, const I8Row& r) {
  const float x = v * r.pre;
  const float t = 127.0f * x;
  const float q0 = t * r.rcp;
  const float rest = fmaf(-q0, r.amax, t) + fmaf(127.0f, x, -t);
  const float q = fmaf(rest, r.rcp, q0);
  return (int)rintf(fminf(fmaxf(q, -127.0f), 127.0f));
}

__device__ __forceinline__ uint32_t i8_pack4(int a, int b, int c, int d) {
  return ((uint32_t)a & 0xFFu) | (((uint32_t)b & 0xFFu) << 8) | (((uint32_t)c & 0xFFu) << 16) | ((uint32_t)d << 24);
}

}  // namespace moe
