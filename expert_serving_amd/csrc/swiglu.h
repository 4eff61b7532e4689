// silu(g) * u for the int8 experts, whose h decides 8-bit codes.
#pragma once

#include <hip/hip_runtime.h>

namespace moe {

// v with values outside fp16's range taken as the largest in it; a NaN stays
// one (the minimum and maximum alone would make a number of it).
__device__ __forceinline__ float clamp_half(float v) {
  const float c = fminf(fmaxf(v, -65504.f), 65504.f);
  return v == v ? c : v;
}

// silu(g) = g / (1 + e^-g).  The rounding of -g * log2 e is carried into the
// exponential (without it the result is off by |g| roundings, with it by one
// or two), and the reciprocal is the hardware's, about one rounding.
__device__ __forceinline__ float silu_mul_exact(float g, float u) {
  // past 256 the exponential is 0 or infinite; a larger g would overflow its product
  // with log2 e, and the remainder of that would be a NaN
  const float x = __builtin_amdgcn_fmed3f(g, -256.f, 256.f);
  const float a = -1.442695041f * x;
  // log2 e = fp32(1.442695041) + 1.92596e-8
  const float lo = fmaf(-1.442695041f, x, -a) + -1.92596e-8f * x;
  const float e = __builtin_amdgcn_exp2f(a);
  const float d = 1.0f + fmaf(e, 0.69314718f * lo, e);
  // e = inf (g < -88): the reciprocal of inf is 0 and the result a zero
  return g * __builtin_amdgcn_rcpf(e < 3.0e38f ? d : __builtin_inff()) * u;
}

}  // namespace moe
