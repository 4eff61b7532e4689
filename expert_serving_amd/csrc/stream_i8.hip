// Few rows against int8 weights: products bound by reading the weights once.
//
// The LDS tiles of the grouped GEMM need several hundred blocks of many K
// stages each to reach the memory's rate; a decode step of few experts has
// neither, and splitting K over blocks costs a second launch for the partial
// sums.  Here every wavefront takes its weights from memory straight into
// MFMA operands -- no LDS, no barrier until the end -- and the eight wavefronts
// of a block split K between them:
//   * one block: 32 output columns (of both matrices for gate/up) and the up
//     to 32 rows of a row tile, as two 16-row halves; the second half is
//     skipped where the tile has at most 16 rows;
//   * step s of 128 codes belongs to wavefront s % 8, so the block reads
//     1 KB runs of every weight row; lane l holds row l % 16 of a fragment and
//     bytes 16 * (l / 16) .. + 15 of each 64-byte half of the step, one operand
//     of v_mfma_i32_16x16x64_i8 each, so that a load touches every 64-byte
//     sector once.  Weights and rows use the same split of K over lanes and
//     operands, so each product pairs equal k;
//   * the eight int32 partial sums meet in LDS (exact in any order), and
//     the epilogue scales, applies SwiGLU and stores four columns per thread.
#include "moe_internal.h"
#include "swiglu.h"

namespace moe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8;
constexpr int kCols = 32;             // output columns of a block
constexpr int kStep = 128;            // codes of a step
constexpr int kAccStride = kCols + 4;  // ints per row of a partial tile in LDS (padded: 16 rows, distinct banks)

__device__ __forceinline__ uint32_t f16_bits(float f) { return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f); }
__device__ __forceinline__ uint32_t bf16_bits(float f) {
  const uint32_t b = __float_as_uint(f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return (b >> 16) | 0x40u;  // NaN stays NaN
  return (b + (((b >> 16) & 1u) + 0x7FFFu)) >> 16;
}

// MH: 16-row halves of the tile (1 or 2)
template <bool DUAL, int MH>
__device__ __forceinline__ void stream_tile(int32_t* __restrict__ smem, const uint8_t* __restrict__ A,
                                            const int32_t* __restrict__ a_rows, const float* __restrict__ sa,
                                            const uint8_t* __restrict__ B0, const uint8_t* __restrict__ B1,
                                            const float* __restrict__ sb0, const float* __restrict__ sb1, int N, int K,
                                            int y_dtype, void* __restrict__ Out, int expert, int row0, int rows,
                                            int n0, uint32_t* __restrict__ flags) {
  constexpr int NB = DUAL ? 2 : 1;
  constexpr int D = 2;  // steps in flight per wavefront
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lk = (lane >> 4) * 16;
  const int steps = K / kStep;
  const int mine = wave < steps ? (steps - wave + kWaves - 1) / kWaves : 0;

  const uint8_t* wp[NB][2];
  const uint8_t* ap[MH];
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    const size_t o = ((size_t)expert * N + min(n0 + 16 * f + lr, N - 1)) * K + (size_t)wave * kStep + lk;
    wp[0][f] = B0 + o;
    if constexpr (DUAL) wp[NB - 1][f] = B1 + o;
  }
#pragma unroll
  for (int h = 0; h < MH; ++h) {
    const int r = row0 + min(16 * h + lr, rows - 1);
    ap[h] = A + (size_t)(a_rows ? a_rows[r] : r) * K + (size_t)wave * kStep + lk;
  }
  i32x4 acc[NB][2][MH];
#pragma unroll
  for (int m = 0; m < NB; ++m)
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int h = 0; h < MH; ++h) acc[m][f][h] = i32x4{0, 0, 0, 0};

  u32x4 wv[D][NB][2][2], av[D][MH][2];
  auto issue = [&](int d, int s) {  // step s of this wavefront (clamped: re-read, not used)
    const size_t o = (size_t)min(s, mine - 1) * (kWaves * kStep);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int m = 0; m < NB; ++m)
#pragma unroll
        for (int f = 0; f < 2; ++f)
          wv[d][m][f][q] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wp[m][f] + o + 64 * q));
#pragma unroll
      for (int h = 0; h < MH; ++h) av[d][h][q] = *reinterpret_cast<const u32x4*>(ap[h] + o + 64 * q);
    }
  };
  auto multiply = [&](int d) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int m = 0; m < NB; ++m)
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int h = 0; h < MH; ++h)
            acc[m][f][h] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, wv[d][m][f][q]),
                                                                 __builtin_bit_cast(i32x4, av[d][h][q]),
                                                                 acc[m][f][h], 0, 0, 0);
  };
  if (mine > 0) {
#pragma unroll
    for (int d = 0; d < D; ++d) issue(d, d);
    const int full = mine - mine % D;
    for (int s = 0; s < full; s += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        // the fences keep the next loads below the products that free their
        // registers
        multiply(d);
        __builtin_amdgcn_sched_barrier(0);
        if (s + d + D < mine) issue(d, s + d + D);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (d < mine - full) multiply(d);
  }

  // lane l of fragment (f, h): row 16 h + l % 16, columns 16 f + 4 (l / 16) .. + 3
#pragma unroll
  for (int m = 0; m < NB; ++m)
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int h = 0; h < MH; ++h)
        *reinterpret_cast<i32x4*>(smem + ((wave * NB + m) * (16 * MH) + 16 * h + lr) * kAccStride + 16 * f +
                                  4 * (lane >> 4)) = acc[m][f][h];
  __syncthreads();
  const int r = tid >> 3, c = (tid & 7) * 4, n = n0 + c;
  if (r >= rows || n >= N) return;  // (512 threads cover 64 rows; rows <= 16 MH)
  i32x4 sum[NB];
#pragma unroll
  for (int m = 0; m < NB; ++m) {
    sum[m] = i32x4{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      sum[m] += *reinterpret_cast<const i32x4*>(smem + ((w * NB + m) * (16 * MH) + r) * kAccStride + c);
  }
  const int row = row0 + r;
  const size_t o = (size_t)row * N + n;
  const f32x4 b0 = *reinterpret_cast<const f32x4*>(sb0 + (size_t)expert * N + n);
  bool overflow = false;
  if constexpr (DUAL) {
    const f32x4 b1 = *reinterpret_cast<const f32x4*>(sb1 + (size_t)expert * N + n);
    const float s = sa[a_rows ? a_rows[row] : row];
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v = silu_mul_exact((float)sum[0][q] * (s * b0[q]), (float)sum[NB - 1][q] * (s * b1[q]));
      overflow |= !(fabsf(v) <= 65504.f);
      w[q] = f16_bits(fminf(fmaxf(v, -65504.f), 65504.f));
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(Out) + o) = uint2{w[0] | (w[1] << 16), w[2] | (w[3] << 16)};
    if (overflow && flags) atomicOr(flags, (uint32_t)MOE_FLAG_H_RANGE);
  } else {
    const float s = sa[row];
    f32x4 v;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = (float)sum[0][q] * (s * b0[q]);
    if (y_dtype == MOE_F32) {
      *reinterpret_cast<f32x4*>(static_cast<float*>(Out) + o) = v;
      return;
    }
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (y_dtype == MOE_F16) {
        overflow |= !(fabsf(v[q]) <= 65504.f);
        w[q] = f16_bits(v[q]);
      } else {
        w[q] = bf16_bits(v[q]);
      }
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(Out) + o) = uint2{w[0] | (w[1] << 16), w[2] | (w[3] << 16)};
    if (overflow && flags) atomicOr(flags, (uint32_t)MOE_FLAG_Y_RANGE);
  }
}

// blockIdx.x: column strip, blockIdx.y: row tile.  sched null: rows of one
// expert, *rows_dev (nullable) of the static_rows exist.
template <bool DUAL>
__global__ __launch_bounds__(64 * kWaves) void k_stream_i8(
    const uint8_t* __restrict__ A, const int32_t* __restrict__ a_rows, const float* __restrict__ sa,
    const uint8_t* __restrict__ B0, const uint8_t* __restrict__ B1, const float* __restrict__ sb0,
    const float* __restrict__ sb1, int N, int K, int y_dtype, void* __restrict__ Out,
    const MTile* __restrict__ sched, const int32_t* __restrict__ count, const int32_t* __restrict__ rows_dev,
    int static_rows, uint32_t* __restrict__ flags) {
  extern __shared__ __attribute__((aligned(16))) int32_t smem[];
  int expert = 0, row0 = blockIdx.y * 32, rows;
  if (sched) {
    if ((int)blockIdx.y >= *count) return;
    const MTile t = sched[blockIdx.y];
    expert = t.expert, row0 = t.row0, rows = t.rows;
  } else {
    rows = min(32, (rows_dev ? min(*rows_dev, static_rows) : static_rows) - row0);
  }
  if (rows <= 0) return;
  const int n0 = blockIdx.x * kCols;
  if (rows <= 16)
    stream_tile<DUAL, 1>(smem, A, a_rows, sa, B0, B1, sb0, sb1, N, K, y_dtype, Out, expert, row0, rows, n0, flags);
  else
    stream_tile<DUAL, 2>(smem, A, a_rows, sa, B0, B1, sb0, sb1, N, K, y_dtype, Out, expert, row0, rows, n0, flags);
}

}  // namespace

hipError_t launch_stream_i8(const void* A, const int32_t* a_rows, const float* sa, const void* B0, const float* sb0,
                            const void* B1, const float* sb1, int N, int K, int y_dtype, void* out,
                            const MTile* sched, const int32_t* count, int max_tiles, const int32_t* rows_dev,
                            int static_rows, uint32_t* flags, hipStream_t st) {
  const int tiles = sched ? max_tiles : (static_rows + 31) / 32;
  if (tiles <= 0) return hipSuccess;
  if (tiles > 65535) return hipErrorInvalidValue;
  const bool dual = B1 != nullptr;
  const int lds = kWaves * (dual ? 2 : 1) * 32 * kAccStride * 4;  // 73728 or 36864 bytes
  const dim3 grid((N + kCols - 1) / kCols, tiles), block(64 * kWaves);
  const uint8_t *a = static_cast<const uint8_t*>(A), *b0 = static_cast<const uint8_t*>(B0),
                *b1 = static_cast<const uint8_t*>(B1);
  if (dual) {
    static std::atomic<uint64_t> set_on{0};
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(&k_stream_i8<true>), lds, set_on);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_stream_i8<true>, grid, block, lds, st, a, a_rows, sa, b0, b1, sb0, sb1, N, K, y_dtype, out,
                       sched, count, rows_dev, static_rows, flags);
  } else {
    hipLaunchKernelGGL(k_stream_i8<false>, grid, block, lds, st, a, a_rows, sa, b0, b1, sb0, sb1, N, K, y_dtype, out,
                       sched, count, rows_dev, static_rows, flags);
  }
  return hipGetLastError();
}

}  // namespace moe
