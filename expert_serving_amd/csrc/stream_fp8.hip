// Few rows against 8-bit floating-point weights with a scale per block of 128:
// products bound by reading the weights once.
//
// As for int8 weights, every wavefront takes its weights from memory straight into
// MFMA operands, with no LDS and no barrier until the end, and the eight wavefronts of
// a block split K between them.  A step of 128 codes is one block of scales and one
// v_mfma_scale_f32_16x16x128_f8f6f4: the matrix units apply the powers of two of the
// row's and the weight block's scale (E8M0 operands), and the sum of the block enters
// the running sum times the product of the two scales' significands, one fused
// multiply-add per sum.
//   * one block: 16 F output columns (of both matrices for gate/up) and the up to 32
//     rows of a row tile, as two 16-row halves, the second skipped where the tile has
//     at most 16;
//   * step s belongs to wavefront s % 8; lane l holds row l % 16 of a fragment and
//     bytes 16 (l / 16) .. + 15 of each 64-byte half of the step, so that a load
//     touches every 64-byte sector once.  Rows and weights use the same split of K over
//     lanes and bytes, so each product pairs equal k;
//   * the eight partial sums meet in LDS and are added in order.
// Gate and up of few rows multiply the codes as fp16, which holds each, on
// v_mfma_f32_16x16x32_f16 instead: the 8-bit units drop what lies 2^-13 below a group's
// largest product, and an h off by 1.4e-5 for that now and then rounds to the next of its 8-bit
// codes, half a step from where it was.  Large batches average over such codes, in the
// row of one token a single one showed (2-norm error of y 4.3e-3 instead of the 1.6e-3 that
// bf16 leaves).  16 conversions and four multiplications for one: 0 to 8 % of the FFN, for which
// the memory sets the time.
// D = 2 steps are under way per wavefront (a third adds 12 % to the product of 17 rows below,
// a fourth 3 %: fewer blocks per compute unit).
//
// Measured (device time of calls in a row): product of 17 rows x 14336 x 4096 15 us, weights
// at 3.9 TB/s; of 128 rows, 8 experts, 4096 x 14336 88 us, 5.3 TB/s; of 1 row x 4096 x 4096
// 8 us; FFN of 1 token over 128 experts of 2048 x 768 16 us for 38 MB, which is the
// latency of two launches, a tile search, a chain of loads and a join each.
#include "half_bits.h"
#include "moe_internal.h"
#include "quant_fp8.h"
#include "swiglu.h"

namespace moe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 8;
constexpr int kStep = 128;  // codes of a step
constexpr int kTileRows = 32;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00020000);
}

struct Tile {
  int expert, row0, rows;
};

// Row tile `index` of the experts' rows, 32 rows each counted from the expert's first;
// rows 0 behind the last tile.  Uniform over the wavefront, which scans the experts'
// offsets: one load and some thirty instructions, where a launch for a tile list costs
// 3 us.
__device__ __forceinline__ Tile find_tile(const Fp8Args& a, int E, int index, int lane) {
  if (!a.offsets) return Tile{0, index * kTileRows, min(kTileRows, a.static_rows - index * kTileRows)};
  const int per = (E + 63) >> 6;  // experts per lane, at most 8
  const int e0 = lane * per;
  int tiles = 0;
  int at[9];
#pragma unroll
  for (int i = 0; i < 9; ++i)
    if (i <= per) at[i] = a.offsets[min(e0 + i, E)];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < per) tiles += (at[i + 1] - at[i] + kTileRows - 1) / kTileRows;
  int upto = tiles;  // tiles of the lanes up to this one
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(upto, off, 64);
    if (lane >= off) upto += o;
  }
  const uint64_t behind = __ballot(upto > index);
  if (behind == 0) return Tile{0, 0, 0};
  const int owner = __builtin_ctzll(behind);
  int left = index - (upto - tiles), e = 0, row0 = 0, rows = 0;
  bool found = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i < per && !found) {
      const int n = at[i + 1] - at[i], t = (n + kTileRows - 1) / kTileRows;
      if (left < t) {
        found = true;
        e = e0 + i;
        row0 = at[i] + left * kTileRows;
        rows = min(kTileRows, n - left * kTileRows);
      }
      left -= t;
    }
  }
  return Tile{__builtin_amdgcn_readlane(e, owner), __builtin_amdgcn_readlane(row0, owner),
              __builtin_amdgcn_readlane(rows, owner)};
}

// F: 16-column fragments of the block, MH: 16-row halves of the tile (1 or 2).
// QUANT: the rows are fp32 h, quantised on the way: a step's 128 columns are one block.
template <bool DUAL, int F, int MH, bool QUANT>
__device__ __forceinline__ void stream_tile(float* __restrict__ smem, const Fp8Args& a, const Tile t, int n0) {
  constexpr int NB = DUAL ? 2 : 1;
  constexpr int D = 2;  // steps in flight per wavefront
  constexpr int kCols = 16 * F;
  constexpr int kStride = kCols + 4;  // floats per row of a partial tile (padded: 16 rows, distinct banks)
  const int N = a.N, K = a.K;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lk = (lane >> 4) * 16;
  const int steps = K / kStep;
  const int mine = wave < steps ? (steps - wave + kWaves - 1) / kWaves : 0;

  // Buffer loads: a resource for each expert's matrix, the tile's rows and their scales,
  // a 32-bit offset per fragment (an expert's matrix and 32 rows of at most 2^20 values
  // are below 2^31 bytes) and the step's in a scalar register.
  const size_t eb = (size_t)t.expert * N * K;
  const __amdgpu_buffer_rsrc_t rw[2] = {resource(a.B0 + eb, (uint32_t)N * (uint32_t)K),
                                        resource((DUAL ? a.B1 : a.B0) + eb, (uint32_t)N * (uint32_t)K)};
  constexpr int kBytes = QUANT ? 4 : 1;
  const __amdgpu_buffer_rsrc_t ra = resource(a.A + (size_t)t.row0 * K * kBytes, (uint32_t)t.rows * (uint32_t)K * kBytes);
  int wo[F], ao[MH];
#pragma unroll
  for (int f = 0; f < F; ++f) wo[f] = min(n0 + 16 * f + lr, N - 1) * K + wave * kStep + lk;
  // (their scales row-major, as every caller of a stream has them)
  const __amdgpu_buffer_rsrc_t rs = resource(a.sa + (size_t)t.row0 * steps, (uint32_t)t.rows * (uint32_t)steps * 4);
  int so_row[MH];
#pragma unroll
  for (int h = 0; h < MH; ++h) {
    const int r = min(16 * h + lr, t.rows - 1);
    ao[h] = (r * K + wave * kStep + lk) * kBytes;
    so_row[h] = (r * steps + wave) * 4;
  }
  // (a block's columns lie in one block of 128 weight rows: 16 F divides 128)
  const size_t so = ((size_t)t.expert * ((N + kFp8Block - 1) / kFp8Block) + n0 / kFp8Block) * steps + wave;
  typedef const __attribute__((address_space(4))) float* scalar_ptr;  // uniform: scalar loads
  const scalar_ptr sw[2] = {(scalar_ptr)(a.sb0 + so), (scalar_ptr)((DUAL ? a.sb1 : a.sb0) + so)};
  f32x4 acc[NB][F][MH];
#pragma unroll
  for (int m = 0; m < NB; ++m)
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int h = 0; h < MH; ++h) acc[m][f][h] = f32x4{0.f, 0.f, 0.f, 0.f};

  u32x4 wv[D][NB][F][2], av[D][MH][2];
  uint32_t sr[D][MH], sb[D][NB];
  bool range = false;
  auto issue = [&](int d, int s) {  // step s of this wavefront (past the last: re-read, not used)
    const int at = min(s, mine - 1) * kWaves;
    const int o = at * kStep;
#pragma unroll
    for (int m = 0; m < NB; ++m) sb[d][m] = __float_as_uint(sw[m][at]);
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int m = 0; m < NB; ++m)
#pragma unroll
        for (int f = 0; f < F; ++f) wv[d][m][f][q] = __builtin_amdgcn_raw_buffer_load_b128(rw[m], wo[f], o + 64 * q, 0);
#pragma unroll
    for (int h = 0; h < MH; ++h) {
      if constexpr (QUANT) {
        f32x4 v[2][4];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[q][i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, ao[h] + 16 * i, (o + 64 * q) * 4, 0));
        uint32_t top = 0u;
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) top = max(top, f8_magnitude(v[q][i][j]));
        top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
        const float amax = __uint_as_float(top);
        range |= !(amax <= 3.402823466e38f);
        const F8Near blk = f8_near(amax);
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            av[d][h][q][i] = f8_pack4(f8_code(v[q][i][0], blk), f8_code(v[q][i][1], blk), f8_code(v[q][i][2], blk),
                                      f8_code(v[q][i][3], blk));
        sr[d][h] = __float_as_uint(f8_scale(amax));
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) av[d][h][q] = __builtin_amdgcn_raw_buffer_load_b128(ra, ao[h], o + 64 * q, 0);
        sr[d][h] = __builtin_amdgcn_raw_buffer_load_b32(rs, so_row[h], at * 4, 0);
      }
    }
  };
  auto operand = [](const u32x4 (&p)[2]) {
    return i32x8{(int)p[0][0], (int)p[0][1], (int)p[0][2], (int)p[0][3],
                 (int)p[1][0], (int)p[1][1], (int)p[1][2], (int)p[1][3]};
  };
  auto halves = [](uint32_t a, uint32_t b) {
    f16x8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = i < 2 ? a : b;
      const f16x2 p = i & 1 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, true)
                            : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, false);
      r[2 * i] = p[0], r[2 * i + 1] = p[1];
    }
    return r;
  };
  // significand of a scale, NaN for one that is not finite, and its exponent + 127; the exponents
  // of the two scales meet before they are applied, as they do in the 8-bit units: neither alone
  // leaves the range
  auto unit = [](uint32_t scale) { return (scale & 0x7F800000u) == 0x7F800000u ? __uint_as_float(0x7FC00000u) : f8_unit(scale); };
  auto power = [](uint32_t scale) { return (int)((scale >> 23) & 0xFFu); };
  auto multiply_wide = [&](int d) {
#pragma unroll
    for (int h = 0; h < MH; ++h) {
      f16x8 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = halves(av[d][h][i >> 1][2 * (i & 1)], av[d][h][i >> 1][2 * (i & 1) + 1]);
      const float ux = unit(sr[d][h]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < NB; ++m) {
        const float u = ux * unit(sb[d][m]);
        const int e = power(sr[d][h]) + power(sb[d][m]) - 254;
#pragma unroll
        for (int f = 0; f < F; ++f) {
          f32x4 p{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            p = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                halves(wv[d][m][f][i >> 1][2 * (i & 1)], wv[d][m][f][i >> 1][2 * (i & 1) + 1]), x[i], p, 0, 0, 0);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[m][f][h][q] = fmaf(__builtin_ldexpf(p[q], e), u, acc[m][f][h][q]);
          __builtin_amdgcn_sched_barrier(0);  // (few block sums at a time: registers)
        }
      }
    }
  };
  auto multiply = [&](int d) {
    if constexpr (DUAL) return multiply_wide(d);
#pragma unroll
    for (int m = 0; m < NB; ++m) {
      const float um = f8_unit(sb[d][m]);
      const int em = f8_exponent(sb[d][m]);
#pragma unroll
      for (int h = 0; h < MH; ++h) {
        const float u = f8_unit(sr[d][h]) * um;
        const int eh = f8_exponent(sr[d][h]);
#pragma unroll
        for (int f = 0; f < F; ++f) {
          const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              operand(wv[d][m][f]), operand(av[d][h]), f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 3, em, 3, eh);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[m][f][h][q] = fmaf(p[q], u, acc[m][f][h][q]);
        }
        __builtin_amdgcn_sched_barrier(0);  // (few block sums at a time: registers)
      }
    }
  };
  if (mine > 0) {
#pragma unroll
    for (int d = 0; d < D; ++d) issue(d, d);
    // no branch around a load inside the loop: its result would be copied at the join,
    // and the copy waits for it
    int s = 0;
    for (; s + 2 * D <= mine; s += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        // the fences keep the next loads below the products that free their registers
        multiply(d);
        __builtin_amdgcn_sched_barrier(0);
        issue(d, s + d + D);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (s + d < mine) multiply(d);
      if (s + d + D < mine) issue(d, s + d + D);
    }
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (s + d + D < mine) multiply(d);
  }
  if (QUANT && range && n0 == 0 && a.flags) atomicOr(a.flags, (uint32_t)MOE_FLAG_H_RANGE);

  // lane l of fragment (f, h): row 16 h + l % 16, columns 16 f + 4 (l / 16) .. + 3
#pragma unroll
  for (int m = 0; m < NB; ++m)
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int h = 0; h < MH; ++h)
        *reinterpret_cast<f32x4*>(smem + ((wave * NB + m) * (16 * MH) + 16 * h + lr) * kStride + 16 * f +
                                  4 * (lane >> 4)) = acc[m][f][h];
  __syncthreads();
  // a thread takes four columns of a row: 128 / F rows of the 16 MH at a time
  const int r = tid / (4 * F), c = (tid % (4 * F)) * 4, n = n0 + c;
  if (r >= t.rows || n >= N) return;
  f32x4 sum[NB];
#pragma unroll
  for (int m = 0; m < NB; ++m) {
    sum[m] = *reinterpret_cast<const f32x4*>(smem + (m * (16 * MH) + r) * kStride + c);
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
      sum[m] += *reinterpret_cast<const f32x4*>(smem + ((w * NB + m) * (16 * MH) + r) * kStride + c);
  }
  const size_t o = (size_t)(t.row0 + r) * N + n;
  if constexpr (DUAL) {
    f32x4 v;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = silu_mul_exact(sum[0][q], sum[NB - 1][q]);
    *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + o) = v;
  } else {
    bool overflow = false;
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (a.y_dtype == MOE_F16) {
        overflow |= !(fabsf(sum[0][q]) <= 65504.f);
        w[q] = f16_bits(sum[0][q]);
      } else {
        w[q] = bf16_bits(sum[0][q]);
      }
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o) = uint2{w[0] | (w[1] << 16), w[2] | (w[3] << 16)};
    if (overflow && a.flags) atomicOr(a.flags, (uint32_t)MOE_FLAG_Y_RANGE);
  }
}

// blockIdx.x: column strip, blockIdx.y: row tile.  MH 1: no tile has more than 16 rows.
template <bool DUAL, int F, int MH, bool QUANT>
__global__ __launch_bounds__(64 * kWaves) void k_stream_fp8(const Fp8Args a, int E, int clear_flags) {
  extern __shared__ __attribute__((aligned(16))) float smem[];
  if (clear_flags && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.flags = 0u;
  const Tile t = find_tile(a, E, blockIdx.y, threadIdx.x & 63);
  if (t.rows <= 0) return;
  const int n0 = blockIdx.x * (16 * F);
  if (MH == 1 || t.rows <= 16)
    stream_tile<DUAL, F, 1, QUANT>(smem, a, t, n0);
  else if constexpr (MH == 2)
    stream_tile<DUAL, F, 2, QUANT>(smem, a, t, n0);
}

template <bool DUAL, int F, int MH, bool QUANT>
hipError_t launch(const Fp8Args& a, int E, bool clear_flags, int tiles, hipStream_t st) {
  constexpr int lds = kWaves * (DUAL ? 2 : 1) * 16 * MH * (16 * F + 4) * 4;  // at most 73728 bytes
  static std::atomic<uint64_t> set_on{0};
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(&k_stream_fp8<DUAL, F, MH, QUANT>), lds, set_on);
  if (e != hipSuccess) return e;
  const dim3 grid((a.N + 16 * F - 1) / (16 * F), tiles);
  hipLaunchKernelGGL((k_stream_fp8<DUAL, F, MH, QUANT>), grid, dim3(64 * kWaves), lds, st, a, E, clear_flags ? 1 : 0);
  return hipGetLastError();
}

// Blocks below which 32 columns per block are better than 64, which leave compute units
// idle.  Measured, 64 against 32 columns: product of 1 row x 4096 x 4096 (64 wide blocks)
// 11.6 against 8.0 us, x 8192 (128) 11.8 against 7.8, x 12288 (192) 12.2 against 11.9, of 28672 x 8192
// (448) 42 against 56; of 17 rows x 8192 x 4096 (128) 14.3 against 11.0, x 14336 (224) 14.7
// against 17.7; of 64 rows, 16 experts, 4096 x 1024 25 against 28.
constexpr int kWideBlocks = 192;

}  // namespace

hipError_t launch_stream_fp8(const Fp8Args& a, bool dual, bool quantise, int E, int max_tiles, int max_rows,
                             bool clear_flags, hipStream_t st) {
  const int tiles = a.offsets ? max_tiles : (a.static_rows + kTileRows - 1) / kTileRows;
  if (tiles <= 0) return hipSuccess;
  if (tiles > 65535) return hipErrorInvalidValue;
  const bool few = max_rows <= 16;
  if (dual) return few ? launch<true, 2, 1, false>(a, E, clear_flags, tiles, st)
                       : launch<true, 2, 2, false>(a, E, clear_flags, tiles, st);
  const bool wide = (long long)tiles * ((a.N + 63) / 64) >= kWideBlocks;
  if (quantise) {  // fp32 rows, at most 16 per tile
    if (!few) return hipErrorInvalidValue;
    return wide ? launch<false, 4, 1, true>(a, E, clear_flags, tiles, st)
                : launch<false, 2, 1, true>(a, E, clear_flags, tiles, st);
  }
  if (few) return wide ? launch<false, 4, 1, false>(a, E, clear_flags, tiles, st)
                       : launch<false, 2, 1, false>(a, E, clear_flags, tiles, st);
  return wide ? launch<false, 4, 2, false>(a, E, clear_flags, tiles, st)
              : launch<false, 2, 2, false>(a, E, clear_flags, tiles, st);
}

}  // namespace moe
