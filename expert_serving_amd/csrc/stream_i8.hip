// Few rows against int8 weights: products bound by reading the weights once.
//
// The LDS tiles of the grouped GEMM need several hundred blocks of many K
// stages each to reach the memory's rate; a decode step of few experts has
// neither, and splitting K over blocks costs a second launch for the partial
// sums.  Here every wavefront takes its weights from memory straight into
// MFMA operands -- no LDS, no barrier until the end -- and the eight wavefronts
// of a block split K between them:
//   * one block: 16 F output columns (of both matrices for gate/up) and the up
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
// The compute units' fill rate bounds it: 58.7 MB of weights for 17 rows take
// 11.4 us as bare loads in this pattern and 16.4 us with the rows' own loads at 32
// columns per block, 15.0 us at 64, so 64 weight rows per block are taken
// wherever they leave enough blocks.  (Non-temporal weight loads: 1 us slower.)
//
// The row tiles are found in the kernel: every wavefront scans the experts'
// offsets, one load and some thirty instructions, where a launch for a tile
// list costs 3 us.
#include "moe_internal.h"
#include "quant_int8.h"
#include "swiglu.h"

namespace moe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 8;
constexpr int kStep = 128;  // codes of a step
constexpr int kTileRows = 32;

__device__ __forceinline__ uint32_t f16_bits(float f) { return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f); }
__device__ __forceinline__ uint32_t bf16_bits(float f) {
  const uint32_t b = __float_as_uint(f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return (b >> 16) | 0x40u;  // NaN stays NaN
  return (b + (((b >> 16) & 1u) + 0x7FFFu)) >> 16;
}

struct StreamArgs {
  const uint8_t* A;          // codes, or fp16 rows (QUANT)
  const int32_t* a_rows;     // rows of A of the tile's rows; null: themselves
  const float* sa;           // scales by row of A
  const uint8_t* B0;
  const uint8_t* B1;
  const float* sb0;
  const float* sb1;
  int N, K, y_dtype;
  void* out;
  const int32_t* offsets;    // [E + 1]; null: rows [0, static_rows) of one expert
  int E, static_rows;
  uint32_t* flags;
  int clear_flags;
};

struct Tile {
  int expert, row0, rows;
};

// Row tile `index` of the experts' rows, 32 rows each counted from the
// expert's first; rows 0 behind the last tile.  Uniform over the wavefront.
__device__ __forceinline__ Tile find_tile(const StreamArgs& a, int index, int lane) {
  if (!a.offsets) return Tile{0, index * kTileRows, min(kTileRows, a.static_rows - index * kTileRows)};
  const int per = (a.E + 63) >> 6;  // experts per lane, at most 8
  const int e0 = lane * per;
  int tiles = 0;
  int at[9];
#pragma unroll
  for (int i = 0; i < 9; ++i)
    if (i <= per) at[i] = a.offsets[min(e0 + i, a.E)];
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

// Four fp16 words (8 values) to 8 codes, with values out of range taken as the
// largest in it (a row with a NaN has the scale NaN, whatever its codes).
__device__ __forceinline__ void codes8(const u32x4 w, const I8Row& r, uint32_t& lo, uint32_t& hi) {
  int c[8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t x = w[q];
    const f16x2 h = __builtin_bit_cast(f16x2, x);
    c[2 * q] = i8_code(fminf(fmaxf((float)h[0], -65504.f), 65504.f), r);
    c[2 * q + 1] = i8_code(fminf(fmaxf((float)h[1], -65504.f), 65504.f), r);
  }
  lo = i8_pack4(c[0], c[1], c[2], c[3]);
  hi = i8_pack4(c[4], c[5], c[6], c[7]);
}

// F: 16-column fragments of the block, MH: 16-row halves of the tile (1 or 2).
// QUANT: the rows are fp16 and quantised here, every block for itself: a row's
// maximum from one pass over it, its codes from a second (both from the cache).
template <bool DUAL, int F, int MH, bool QUANT>
__device__ __forceinline__ void stream_tile(int32_t* __restrict__ smem, const StreamArgs& a, const Tile t, int n0) {
  constexpr int NB = DUAL ? 2 : 1;
  constexpr int D = 2;  // steps in flight per wavefront
  constexpr int kCols = 16 * F;
  constexpr int kStride = kCols + 4;  // ints per row of a partial tile (padded: 16 rows, distinct banks)
  const int N = a.N, K = a.K;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lk = (lane >> 4) * 16;
  const int steps = K / kStep;
  const int mine = wave < steps ? (steps - wave + kWaves - 1) / kWaves : 0;

  const uint8_t* wp[NB][F];
  const uint8_t* ap[MH];
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const size_t o = ((size_t)t.expert * N + min(n0 + 16 * f + lr, N - 1)) * K + (size_t)wave * kStep + lk;
    wp[0][f] = a.B0 + o;
    if constexpr (DUAL) wp[NB - 1][f] = a.B1 + o;
  }
#pragma unroll
  for (int h = 0; h < MH; ++h) {
    const int r = t.row0 + min(16 * h + lr, t.rows - 1);
    ap[h] = a.A + ((size_t)(a.a_rows ? a.a_rows[r] : r) * K + (size_t)wave * kStep + lk) * (QUANT ? 2 : 1);
  }
  i32x4 acc[NB][F][MH];
#pragma unroll
  for (int m = 0; m < NB; ++m)
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int h = 0; h < MH; ++h) acc[m][f][h] = i32x4{0, 0, 0, 0};

  // QUANT: the row's maximum, over this wavefront's steps, the four lanes of a
  // row, and the wavefronts
  __shared__ uint32_t s_top[QUANT ? kWaves : 1][16];
  I8Row q8{};
  if constexpr (QUANT) {
    u16x2 tops = {0, 0};  // magnitudes of halves order as words do
    for (int s = 0; s < mine; ++s)
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // two operands of 16 values
        const u32x4 w = *reinterpret_cast<const u32x4*>(ap[0] + ((size_t)s * (kWaves * kStep) + 64 * (q >> 1)) * 2 +
                                                        16 * (q & 1));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          tops = __builtin_elementwise_max(tops, __builtin_bit_cast(u16x2, (uint32_t)(w[i] & 0x7FFF7FFFu)));
      }
    const uint16_t half = tops[0] > tops[1] ? tops[0] : tops[1];
    uint32_t top = i8_magnitude((float)__builtin_bit_cast(_Float16, half));
    top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
    if (lane < 16) s_top[wave][lane] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = max(top, s_top[w][lr]);
    const float amax = __uint_as_float(top);
    if (!(amax <= 65504.f) && n0 == 0 && a.flags) atomicOr(a.flags, (uint32_t)MOE_FLAG_H_RANGE);
    q8 = i8_row(clamp_half(amax));
  }

  u32x4 wv[D][NB][F][2], av[D][MH][2];
  auto issue = [&](int d, int s) {  // step s of this wavefront (past the last: re-read, not used)
    const size_t o = (size_t)min(s, mine - 1) * (kWaves * kStep);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int m = 0; m < NB; ++m)
#pragma unroll
        for (int f = 0; f < F; ++f) wv[d][m][f][q] = *reinterpret_cast<const u32x4*>(wp[m][f] + o + 64 * q);
#pragma unroll
      for (int h = 0; h < MH; ++h) {
        if constexpr (QUANT) {
          const uint8_t* p = ap[h] + (o + 64 * q) * 2;
          uint32_t w0, w1, w2, w3;
          codes8(*reinterpret_cast<const u32x4*>(p), q8, w0, w1);
          codes8(*reinterpret_cast<const u32x4*>(p + 16), q8, w2, w3);
          av[d][h][q] = u32x4{w0, w1, w2, w3};
        } else {
          av[d][h][q] = *reinterpret_cast<const u32x4*>(ap[h] + o + 64 * q);
        }
      }
    }
  };
  auto multiply = [&](int d) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int m = 0; m < NB; ++m)
#pragma unroll
        for (int f = 0; f < F; ++f)
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
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int h = 0; h < MH; ++h)
        *reinterpret_cast<i32x4*>(smem + ((wave * NB + m) * (16 * MH) + 16 * h + lr) * kStride + 16 * f +
                                  4 * (lane >> 4)) = acc[m][f][h];
  __syncthreads();
  // a thread takes four columns of a row: 128 / F rows of the 16 MH at a time
  const int r = tid / (4 * F), c = (tid % (4 * F)) * 4, n = n0 + c;
  if (r >= t.rows || n >= N) return;
  i32x4 sum[NB];
#pragma unroll
  for (int m = 0; m < NB; ++m) {
    sum[m] = i32x4{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      sum[m] += *reinterpret_cast<const i32x4*>(smem + ((w * NB + m) * (16 * MH) + r) * kStride + c);
  }
  const int row = t.row0 + r;
  const size_t o = (size_t)row * N + n;
  const f32x4 b0 = *reinterpret_cast<const f32x4*>(a.sb0 + (size_t)t.expert * N + n);
  bool overflow = false;
  if constexpr (DUAL) {
    // A value out of fp16's range, also one that would round to the largest in it,
    // becomes infinite (a NaN stays): the quantisation of the row takes it back to
    // the largest one and sets the flag, which this launch may be clearing.
    const f32x4 b1 = *reinterpret_cast<const f32x4*>(a.sb1 + (size_t)t.expert * N + n);
    const float s = a.sa[a.a_rows ? a.a_rows[row] : row];
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float v = silu_mul_exact((float)sum[0][q] * (s * b0[q]), (float)sum[NB - 1][q] * (s * b1[q]));
      w[q] = f16_bits(fabsf(v) <= 65504.f ? v : v * __builtin_inff());
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o) = uint2{w[0] | (w[1] << 16), w[2] | (w[3] << 16)};
  } else {
    float s;
    if constexpr (QUANT) {
      uint32_t top = 0u;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = max(top, s_top[w][r]);
      s = clamp_half(__uint_as_float(top)) / 127.0f;
    } else {
      s = a.sa[row];
    }
    f32x4 v;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = (float)sum[0][q] * (s * b0[q]);
    if (a.y_dtype == MOE_F32) {
      *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + o) = v;
      return;
    }
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (a.y_dtype == MOE_F16) {
        overflow |= !(fabsf(v[q]) <= 65504.f);
        w[q] = f16_bits(v[q]);
      } else {
        w[q] = bf16_bits(v[q]);
      }
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o) = uint2{w[0] | (w[1] << 16), w[2] | (w[3] << 16)};
    if (overflow && a.flags) atomicOr(a.flags, (uint32_t)MOE_FLAG_Y_RANGE);
  }
}

// blockIdx.x: column strip, blockIdx.y: row tile.  MH 1: no tile has more than
// 16 rows.
template <bool DUAL, int F, int MH, bool QUANT>
__global__ __launch_bounds__(64 * kWaves) void k_stream_i8(const StreamArgs a) {
  extern __shared__ __attribute__((aligned(16))) int32_t smem[];
  if (a.clear_flags && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.flags = 0u;
  const Tile t = find_tile(a, blockIdx.y, threadIdx.x & 63);
  if (t.rows <= 0) return;
  const int n0 = blockIdx.x * (16 * F);
  if (MH == 1 || t.rows <= 16)
    stream_tile<DUAL, F, 1, QUANT>(smem, a, t, n0);
  else if constexpr (MH == 2)
    stream_tile<DUAL, F, 2, QUANT>(smem, a, t, n0);
}

template <bool DUAL, int F, int MH, bool QUANT>
hipError_t launch(const StreamArgs& a, int tiles, hipStream_t st) {
  constexpr int lds = kWaves * (DUAL ? 2 : 1) * 16 * MH * (16 * F + 4) * 4;  // at most 73728 bytes
  static std::atomic<uint64_t> set_on{0};
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(&k_stream_i8<DUAL, F, MH, QUANT>), lds, set_on);
  if (e != hipSuccess) return e;
  const dim3 grid((a.N + 16 * F - 1) / (16 * F), tiles);
  hipLaunchKernelGGL((k_stream_i8<DUAL, F, MH, QUANT>), grid, dim3(64 * kWaves), lds, st, a);
  return hipGetLastError();
}

// blocks below which 32 columns per block are better than 64: they leave
// compute units idle
constexpr int kWideBlocks = 192;

}  // namespace

hipError_t launch_stream_gateup_i8(const void* A, const int32_t* a_rows, const float* sa, const moe_int8_ffn& w,
                                   int N, int K, void* h, const int32_t* offsets, int E, int max_tiles,
                                   int max_rows, int static_rows, uint32_t* flags, bool clear_flags, hipStream_t st) {
  const int tiles = offsets ? max_tiles : (static_rows + kTileRows - 1) / kTileRows;
  if (tiles <= 0) return hipSuccess;
  if (tiles > 65535) return hipErrorInvalidValue;
  const StreamArgs a{static_cast<const uint8_t*>(A), a_rows, sa, reinterpret_cast<const uint8_t*>(w.gate),
                     reinterpret_cast<const uint8_t*>(w.up), w.gate_scales, w.up_scales, N, K, MOE_F16, h, offsets, E,
                     static_rows, flags, clear_flags ? 1 : 0};
  return max_rows <= 16 ? launch<true, 2, 1, false>(a, tiles, st) : launch<true, 2, 2, false>(a, tiles, st);
}

hipError_t launch_stream_i8(const void* A, const float* sa, const void* B, const float* sb, int N, int K, int y_dtype,
                            void* y, const int32_t* offsets, int E, int max_tiles, int max_rows, int static_rows,
                            uint32_t* flags, bool clear_flags, hipStream_t st) {
  const int tiles = offsets ? max_tiles : (static_rows + kTileRows - 1) / kTileRows;
  if (tiles <= 0) return hipSuccess;
  if (tiles > 65535) return hipErrorInvalidValue;
  const StreamArgs a{static_cast<const uint8_t*>(A), nullptr, sa, static_cast<const uint8_t*>(B), nullptr, sb, nullptr,
                     N, K, y_dtype, y, offsets, E, static_rows, flags, clear_flags ? 1 : 0};
  const bool wide = (long long)tiles * ((N + 63) / 64) >= kWideBlocks;
  if (!sa) {  // fp16 rows, at most 16 per tile
    if (max_rows > 16) return hipErrorInvalidValue;
    return wide ? launch<false, 4, 1, true>(a, tiles, st) : launch<false, 2, 1, true>(a, tiles, st);
  }
  if (max_rows <= 16) return wide ? launch<false, 4, 1, false>(a, tiles, st) : launch<false, 2, 1, false>(a, tiles, st);
  return wide ? launch<false, 4, 2, false>(a, tiles, st) : launch<false, 2, 2, false>(a, tiles, st);
}

}  // namespace moe
