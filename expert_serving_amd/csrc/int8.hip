// The reductions of the int8 expert path behind a split K: SwiGLU over int32
// partial sums, and the sum of a down projection's fp32 shares.  Both read each
// part once, from the caches where a few rows wrote it: 4.2 us for one token over
// 8 experts of 7168 x 2048 behind 41 us of gate and up, 4.3 behind 22 us of the
// down projection, which is the launch.  Unsplit, one token's rows would leave
// three quarters of the compute units idle.
#include "moe_internal.h"
#include "swiglu.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t f32_to_f16_bits(float f) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f);
}
__device__ __forceinline__ uint32_t f32_to_bf16_rne(float f) {
  const uint32_t b = __float_as_uint(f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return (b >> 16) | 0x40u;  // NaN stays NaN
  return (b + (((b >> 16) & 1u) + 0x7FFFu)) >> 16;
}

constexpr int kPartRows = 4;  // rows of a tile per block (gridDim.z blocks take the others)

// h of the rows of one 32-row tile and 1024 columns: gate and up sums are the
// exact int32 sums of their parts.  The row tile gives the expert, whose scales
// the four columns of a thread share over the rows.
__global__ __launch_bounds__(256) void k_swiglu_parts_i8(const int32_t* __restrict__ parts, int nparts,
                                                         long long part_elems, int N,
                                                         const int32_t* __restrict__ a_rows,
                                                         const float* __restrict__ sa, const float* __restrict__ sbg,
                                                         const float* __restrict__ sbu,
                                                         const MTile* __restrict__ sched,
                                                         const int32_t* __restrict__ count, int static_rows,
                                                         uint16_t* __restrict__ h, uint32_t* __restrict__ flags) {
  int expert = 0, row0 = blockIdx.x * 32, rows;
  if (sched) {
    if ((int)blockIdx.x >= *count) return;
    const MTile t = sched[blockIdx.x];
    expert = t.expert, row0 = t.row0, rows = t.rows;
  } else {
    rows = min(32, static_rows - row0);
  }
  const int c = (blockIdx.y * 256 + threadIdx.x) * 4;
  if (c >= N) return;
  const f32x4 g4 = *reinterpret_cast<const f32x4*>(sbg + (size_t)expert * N + c);
  const f32x4 u4 = *reinterpret_cast<const f32x4*>(sbu + (size_t)expert * N + c);
  bool overflow = false;
  for (int r = blockIdx.z; r < rows; r += gridDim.z) {
    const int row = row0 + r;
    const float s = sa[a_rows ? a_rows[row] : row];
    const int32_t* g = parts + (size_t)row * N + c;
    const int32_t* u = g + (size_t)nparts * part_elems;
    i32x4 gs = *reinterpret_cast<const i32x4*>(g), us = *reinterpret_cast<const i32x4*>(u);
    for (int p = 1; p < nparts; ++p) {
      gs += *reinterpret_cast<const i32x4*>(g + p * part_elems);
      us += *reinterpret_cast<const i32x4*>(u + p * part_elems);
    }
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v = silu_mul_exact((float)gs[q] * (s * g4[q]), (float)us[q] * (s * u4[q]));
      overflow |= !(fabsf(v) <= 65504.f);
      w[q] = f32_to_f16_bits(clamp_half(v));
    }
    *reinterpret_cast<uint2*>(h + (size_t)row * N + c) = uint2{w[0] | (w[1] << 16), w[2] | (w[3] << 16)};
  }
  if (overflow && flags) atomicOr(flags, (uint32_t)MOE_FLAG_H_RANGE);
}

__global__ __launch_bounds__(256) void k_sum_parts(const float* __restrict__ parts, int nparts, long long part_elems,
                                                   int N, const int32_t* __restrict__ rows_dev, int y_dtype,
                                                   void* __restrict__ y, uint32_t* __restrict__ flags) {
  const int r = blockIdx.x;
  if (rows_dev && r >= *rows_dev) return;
  const int c = (blockIdx.y * 256 + threadIdx.x) * 4;
  if (c >= N) return;
  const size_t o = (size_t)r * N + c;
  f32x4 v = *reinterpret_cast<const f32x4*>(parts + o);
  for (int p = 1; p < nparts; ++p) v += *reinterpret_cast<const f32x4*>(parts + p * part_elems + o);
  if (y_dtype == MOE_F32) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(y) + o) = v;
    return;
  }
  uint32_t w[4];
  bool overflow = false;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (y_dtype == MOE_F16) {
      overflow |= !(fabsf(v[q]) <= 65504.f);
      w[q] = f32_to_f16_bits(v[q]);
    } else {
      w[q] = f32_to_bf16_rne(v[q]);
    }
  }
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + o) = uint2{w[0] | (w[1] << 16), w[2] | (w[3] << 16)};
  if (overflow && flags) atomicOr(flags, (uint32_t)MOE_FLAG_Y_RANGE);
}

}  // namespace

hipError_t launch_swiglu_parts_i8(const int32_t* parts, int nparts, long long part_elems, int N,
                                  const int32_t* a_rows, const float* sa, const float* sbg, const float* sbu,
                                  const MTile* sched, const int32_t* count, int max_tiles, int static_rows,
                                  void* h, uint32_t* flags, hipStream_t st) {
  const int tiles = sched ? max_tiles : (static_rows + 31) / 32;
  if (tiles <= 0) return hipSuccess;
  if (N % 4) return hipErrorInvalidValue;
  hipLaunchKernelGGL(k_swiglu_parts_i8, dim3(tiles, (N + 1023) / 1024, 32 / kPartRows), dim3(256), 0, st, parts,
                     nparts, part_elems, N, a_rows, sa, sbg, sbu, sched, count, static_rows,
                     static_cast<uint16_t*>(h), flags);
  return hipGetLastError();
}

hipError_t launch_sum_parts(const float* parts, int nparts, long long part_elems, int N, const int32_t* rows_dev,
                            int max_rows, int y_dtype, void* y, uint32_t* flags, hipStream_t st) {
  if (max_rows <= 0) return hipSuccess;
  if (N % 4) return hipErrorInvalidValue;
  hipLaunchKernelGGL(k_sum_parts, dim3(max_rows, (N + 1023) / 1024), dim3(256), 0, st, parts, nparts, part_elems, N,
                     rows_dev, y_dtype, y, flags);
  return hipGetLastError();
}

}  // namespace moe
