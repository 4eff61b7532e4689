// Products of 8-bit floating-point rows and expert weights with an fp32 scale per
// block of 128 (the launchers and their operands: moe_internal.h).
#include "moe_internal.h"
#include "quant_fp8.h"
#include "swiglu.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t f16_bits(float f) { return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f); }
__device__ __forceinline__ uint32_t bf16_bits(float f) {
  const uint32_t b = __float_as_uint(f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return (b >> 16) | 0x40u;  // NaN stays NaN
  return (b + (((b >> 16) & 1u) + 0x7FFFu)) >> 16;
}

// the 32 codes of a lane for v_mfma_scale_f32_32x32x64_f8f6f4, from two 16-byte parts
__device__ __forceinline__ i32x8 cat8(u32x4 lo, u32x4 hi) {
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}
__device__ __forceinline__ f32x16 mfma8(i32x8 a, i32x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 127, 0, 127);
}

// 64 x 64 outputs per block of four wavefronts, a quarter each, operands straight from
// memory.  A block of K = 128 is two MFMAs into a sum of its own, which the scales'
// product then adds to the running one.
template <bool DUAL>
__global__ __launch_bounds__(256) void k_gemm_fp8(const Fp8Args a) {
  int expert = 0, row0 = blockIdx.y * kFp8TileRows, rows;
  if (a.sched) {
    if ((int)blockIdx.y >= *a.count) return;
    const MTile t = a.sched[blockIdx.y];
    expert = t.expert, row0 = t.row0, rows = t.rows;
  } else {
    rows = min(kFp8TileRows, a.static_rows - row0);
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lr = lane & 31, lk = (lane >> 5) * 16;
  const int m0 = 32 * (wave & 1), n0 = blockIdx.x * 64 + 32 * (wave >> 1);
  if (m0 >= rows || n0 >= a.N) return;
  const int K = a.K, blocks = K / kFp8Block;
  const int r = row0 + min(m0 + lr, rows - 1), n = min(n0 + lr, a.N - 1);
  const uint8_t* pa = a.A + (size_t)r * K + lk;
  const uint8_t* pb0 = a.B0 + ((size_t)expert * a.N + n) * K + lk;
  const uint8_t* pb1 = DUAL ? a.B1 + ((size_t)expert * a.N + n) * K + lk : pb0;
  const float* sa = a.sa + (size_t)r * a.sa_row;
  const size_t sbo = ((size_t)expert * ((a.N + kFp8Block - 1) / kFp8Block) + n0 / kFp8Block) * blocks;
  f32x16 acc0, acc1;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc0[i] = acc1[i] = 0.f;
  auto load = [](const uint8_t* p) {
    return cat8(*reinterpret_cast<const u32x4*>(p), *reinterpret_cast<const u32x4*>(p + 32));
  };
  for (int b = 0; b < blocks; ++b) {
    const float s = sa[(size_t)b * a.sa_group];
    f32x16 t0, t1;
#pragma unroll
    for (int i = 0; i < 16; ++i) t0[i] = t1[i] = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const i32x8 x = load(pa + (size_t)b * kFp8Block + 64 * h);
      t0 = mfma8(load(pb0 + (size_t)b * kFp8Block + 64 * h), x, t0);
      if constexpr (DUAL) t1 = mfma8(load(pb1 + (size_t)b * kFp8Block + 64 * h), x, t1);
    }
    const float c0 = s * a.sb0[sbo + b], c1 = DUAL ? s * a.sb1[sbo + b] : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      acc0[i] = fmaf(t0[i], c0, acc0[i]);
      if constexpr (DUAL) acc1[i] = fmaf(t1[i], c1, acc1[i]);
    }
  }
  if (m0 + lr >= rows) return;
  bool range = false;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int col = n0 + 8 * q + 4 * (lane >> 5);
    if (col >= a.N) continue;
    const size_t o = (size_t)r * a.N + col;
    f32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = DUAL ? silu_mul_exact(acc0[4 * q + i], acc1[4 * q + i]) : acc0[4 * q + i];
    if (DUAL) {
#pragma unroll
      for (int i = 0; i < 4; ++i) range |= !(fabsf(v[i]) <= 3.402823466e38f);
      *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + o) = v;
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (a.y_dtype == MOE_F16) {
          range |= !(fabsf(v[i]) <= 65504.f);
          w[i] = f16_bits(v[i]);
        } else {
          w[i] = bf16_bits(v[i]);
        }
      }
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o) = uint2{w[0] | (w[1] << 16), w[2] | (w[3] << 16)};
    }
  }
  if (range && a.flags) atomicOr(a.flags, (uint32_t)(DUAL ? MOE_FLAG_H_RANGE : MOE_FLAG_Y_RANGE));
}

}  // namespace

hipError_t launch_gemm_fp8(const Fp8Args& a, bool dual, int max_tiles, hipStream_t st) {
  const int tiles = a.sched ? max_tiles : (a.static_rows + kFp8TileRows - 1) / kFp8TileRows;
  if (tiles <= 0) return hipSuccess;
  if (tiles > 65535) return hipErrorInvalidValue;
  const dim3 grid((a.N + 63) / 64, tiles);
  if (dual)
    hipLaunchKernelGGL(k_gemm_fp8<true>, grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(k_gemm_fp8<false>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace moe
