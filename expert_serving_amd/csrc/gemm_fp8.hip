// Products of 8-bit floating-point rows and expert weights with an fp32 scale per
// block of 128 along K (and per 128 weight rows): y = sum over blocks b of
// sa[r][b] sb[n / 128][b] sum_k a[r][k] w[n][k], and the SwiGLU of two of them.
//
// The scales change from block to block, so they cannot wait for the epilogue.  A
// block's sum on its own would take registers for it beside the running sums, which a
// 256 x 256 tile does not have.  So the running sums are held in units: a scale is
// 2^e m with m in [1, 2); the matrix units apply 2^e themselves (E8M0 operands of
// v_mfma_scale_f32_32x32x64_f8f6f4, 2^e of the token row and of the weight block), and
// before the first MFMA of a block every sum is multiplied by the ratio of the last
// block's m_row m_weight to this one's, a factor between 1/4 and 4 that cannot leave
// fp32's range.  One multiplication per sum and block either way; the ratio carries
// three roundings, so that a sum over K / 128 blocks is off by a few times K / 128
// half steps of fp32, far below the 2^-13 that the units' alignment of products costs.
//
// One block of 8 wavefronts (two per SIMD) makes a tile of up to 256 token rows (in
// steps of 64) x 256 weight rows (gate/up: 128 of each matrix), weights as the MFMA's
// first operand, so that a lane's 16 sums of a fragment belong to one token row.  A stage
// is K = 128 in one of two (for low tiles three) LDS buffers: rows of 128 bytes, 16-byte
// chunk c of row r at c ^ ((r >> 1) & 7), filled straight from memory (8 rows x 128 bytes
// per wavefront load).  A stage has two steps of K = 64.  In the first the fragments of
// the second are read, which is the last use of the buffer; a barrier; in the second
// the fragments of the next stage are read and the loads of the stage after it issued.
//
// Measured: product of 4096 rows x 4096 x 14336 240 us, 2.0 PFLOP/s (a library product
// with one scale per matrix: 2.5); of 8192 rows, 8 experts, 500 us; FFN of 8192 tokens, top
// 8 of 256 experts, 7168 x 2048, 3.9 ms, 1.5 PFLOP/s.  A stage takes 3300 to 3650 cycles
// where its MFMAs alone take 2048: a multiplication per sum and block takes the wavefront's
// issue slots (8 MFMAs 517 cycles, with their 128 multiplications 740), and a stage's loads
// are under way for about as long as the stage.  MFMA duty 46 to 55 % at 1.7 to 1.8 GHz, the
// power limit's.  FFN of 64 tokens over 8 experts of 4096 x 14336 295 us: weights at 4.8 TB/s.
#include <type_traits>

#include "moe_internal.h"
#include "quant_fp8.h"
#include "swiglu.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef const __attribute__((address_space(1))) void* gbl_ptr_t;

constexpr int kBufferRsrcWord3 = 0x00020000;  // raw buffer of gfx9-family GPUs, 32-bit data format
constexpr int kStage = 128;                   // codes (bytes) of K per stage
constexpr int kChunkStages = 8;               // stages whose scales lie in LDS together

// the 32 codes of a lane for v_mfma_scale_f32_32x32x64_f8f6f4, from two 16-byte parts
__device__ __forceinline__ i32x8 cat8(u32x4 lo, u32x4 hi) {
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

__device__ __forceinline__ void raw_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// s_waitcnt for this wavefront's LDS reads, and for all but its last N loads
template <int N>
__device__ __forceinline__ void wait_lds_and_loads() {
  static_assert(N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4));
}

// The tiles of a launch, taken by blocks that stay: every XCD has an equal contiguous
// share of them (blocks go to XCD blockIdx % 8 in turn, and neighbouring tiles share rows
// and weights in its L2), a block whose XCD has none left helps the others, and the
// quarter tiles of the last row tiles (see k_schedule_fp8) come behind all others.
// Tiles differ in height, so equal counts alone leave XCDs idle: FFN of 8192 rows over 8
// experts, 4096 x 14336, a third of the gate/up launch.
struct Queue {
  int32_t* next;    // [8] of the XCDs, [1] of the quarter tiles
  int whole, all;   // tiles without quarters, and all
  __device__ __forceinline__ int share(int x) const { return min(whole, (x + 1) * ((whole + 7) >> 3)); }
  // tile of the own XCD's v-th turn, or one of another's; -1: none left
  __device__ __forceinline__ int tile(int x, int v) const {
    const int per = (whole + 7) >> 3;
    if (x * per + v < share(x)) return x * per + v;
    for (int i = 1; i < 8; ++i) {
      const int y = (x + i) & 7, n = share(y) - y * per;
      if (__hip_atomic_load(next + y, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) >= n) continue;
      const int u = atomicAdd(next + y, 1);
      if (u < n) return y * per + u;
    }
    const int u = whole + atomicAdd(next + 8, 1);
    return u < all ? u : -1;
  }
};

__device__ __forceinline__ f32x16 mfma_scaled(i32x8 w, i32x8 x, f32x16 c, int ew, int ex) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, c, 0, 0, 3, ew, 3, ex);
}

// LDS buffers of a tile: as many as fit beside the scales (half a compute unit's LDS for
// BN 128).  The few rows of a low tile stream their weights, and what is under way
// decides how fast: with three instead of two FFN of 64 tokens over 8 experts of 4096 x 14336
// 350 -> 286 us, product of 128 rows over them 132 -> 115.
constexpr int tile_stages(int BM, int BN) { return BN == 128 ? (BM <= 64 ? 3 : 2) : (BM <= 128 ? 3 : 2); }
constexpr int tile_lds(int BM, int BN) {
  return tile_stages(BM, BN) * (BM + BN) * kStage + 2 * kChunkStages * (BM + 64) * 4;
}

constexpr int max_of(int a, int b) { return a > b ? a : b; }

// BM token rows x BN weight rows (DUAL: BN / 2 of each matrix).  The first thread takes
// its XCD's next turn (v) a few stages before the end.
template <int BM, int BN, bool DUAL>
__device__ __forceinline__ void tile_fp8(uint8_t* smem, const Fp8Args& a, const MTile t, int ni, int32_t* turn, int& v) {
  constexpr int FM = BM / 64, FN = BN / 128;   // fragments of a wavefront: 2 x 4 wavefronts
  constexpr int WM = BM / 2, WN = DUAL ? BN / 8 : BN / 4;  // its rows and columns (of each matrix)
  constexpr int NI = FM + BN / 64;             // 8-row loads per wavefront and stage
  constexpr int BUF = (BM + BN) * kStage, NS = tile_stages(BM, BN);
  constexpr int COLS = DUAL ? BN / 2 : BN;     // output columns
  static_assert(!DUAL || BN == 256, "a block of h columns per tile");
  const int N = a.N, K = a.K, S = K / kStage;
  const int rows = t.rows, n0 = ni * COLS;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  const int fr = lane & 31, fk = lane >> 5;

  // ---- loads ----
  const uint8_t* A0 = a.A + (size_t)t.row0 * K;
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(A0), 0,
                                                                      (uint32_t)rows * (uint32_t)K, kBufferRsrcWord3);
  const size_t eb = (size_t)t.expert * N * K;
  const __amdgpu_buffer_rsrc_t rb0 = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.B0 + eb), 0,
                                                                       (uint32_t)N * (uint32_t)K, kBufferRsrcWord3);
  const __amdgpu_buffer_rsrc_t rb1 = DUAL ? __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.B1 + eb), 0,
                                                                              (uint32_t)N * (uint32_t)K, kBufferRsrcWord3)
                                          : rb0;
  // lane l of a load fills position l % 8 of row l / 8, which holds chunk
  // (l % 8) ^ ((row >> 1) & 7); the row's own eight start at a multiple of 8 rows
  // that is odd or even with the wavefront
  const int chunk = (lane & 7) ^ ((4 * wave + (lane >> 4)) & 7);
  int va[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i) va[i] = min(8 * (wave + 8 * i) + (lane >> 3), rows - 1) * K + chunk * 16;
  const int vb = (lane >> 3) * K + chunk * 16;
  auto load = [&](int buf, int s, int i) {  // load i of stage s
    uint8_t* dst = smem + buf * BUF + 8 * (wave + 8 * i) * kStage;
    if (i < FM) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)dst, 16, va[i < FM ? i : 0], s * kStage, 0, 0);
    } else {
      const int w0 = 8 * (wave + 8 * (i - FM));  // weight row of the tile; N is a multiple of 8
      const int col = min(n0 + (DUAL ? w0 & (COLS - 1) : w0), N - 8);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(DUAL && w0 >= COLS ? rb1 : rb0, (lds_ptr_t)dst, 16, vb,
                                               col * K + s * kStage, 0, 0);
    }
  };
  // the scales of stages 8 c .. 8 c + 7: wavefront w those of stage 8 c + w, BM token
  // rows, then the weight blocks of the tile (two, in turn over the lanes)
  float* const s_row = reinterpret_cast<float*>(smem + NS * BUF);  // [2][8][BM]
  float* const s_wgt = s_row + 2 * kChunkStages * BM;             // [2][8][64]
  const int nblocks = (N + kFp8Block - 1) / kFp8Block;
  const float* const swl = (DUAL && (lane & 1) ? a.sb1 : a.sb0) +
                           ((size_t)t.expert * nblocks +
                            min(n0 / kFp8Block + (DUAL ? 0 : lane & 1), nblocks - 1)) * S;
  auto load_scales = [&](int c) {
    const int g = min(kChunkStages * c + wave, S - 1), at = (c & 1) * kChunkStages + wave;
    const float* p = a.sa + (size_t)t.row0 * a.sa_row + (size_t)g * a.sa_group;
#pragma unroll
    for (int i = 0; i < FM; ++i)
      __builtin_amdgcn_global_load_lds((gbl_ptr_t)(p + (size_t)min(64 * i + lane, rows - 1) * a.sa_row),
                                       (lds_ptr_t)(s_row + at * BM + 64 * i), 4, 0, 0);
    __builtin_amdgcn_global_load_lds((gbl_ptr_t)(swl + g), (lds_ptr_t)(s_wgt + at * 64), 4, 0, 0);
  };

  // ---- fragments ----
  // row r of the stage, chunks 4 h + fk and 4 h + 2 + fk: (r >> 1) & 7 is that of fr,
  // since fragments start at multiples of 32 rows
  const int swz = (fr >> 1) & 7;
  const uint8_t* const fa = smem + (wm * WM + fr) * kStage;
  const uint8_t* const fb = smem + (BM + wn * WN + fr) * kStage;
  auto frag = [&](const uint8_t* row, int h) {
    return cat8(*reinterpret_cast<const u32x4*>(row + (((4 * h + fk) ^ swz) << 4)),
                *reinterpret_cast<const u32x4*>(row + (((4 * h + 2 + fk) ^ swz) << 4)));
  };
  auto frag_a = [&](int buf, int h, int b) { return frag(fa + buf * BUF + b * 32 * kStage, h); };
  auto frag_b = [&](int buf, int h, int f) { return frag(fb + buf * BUF + f * (DUAL ? COLS : 32) * kStage, h); };

  f32x16 acc[FN][FM];
#pragma unroll
  for (int f = 0; f < FN; ++f)
#pragma unroll
    for (int b = 0; b < FM; ++b)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[f][b][q] = 0.f;
  i32x8 xa[FM], wf[2][FN];
  // exponent words of the current stage's scales, and the change of the sums' units
  // that its first step makes
  int et[FM], ew[FN];
  float rt[FM], rw[FN];
  auto read_scales = [&](int s, uint32_t (&nt)[FM], uint32_t (&nw)[FN]) {
    const int at = ((s / kChunkStages) & 1) * kChunkStages + s % kChunkStages;
#pragma unroll
    for (int b = 0; b < FM; ++b) nt[b] = __float_as_uint(s_row[at * BM + wm * WM + b * 32 + fr]);
#pragma unroll
    for (int f = 0; f < FN; ++f) nw[f] = __float_as_uint(s_wgt[at * 64 + (DUAL ? f : (wn * WN) / kFp8Block)]);
  };
  auto next_units = [&](const uint32_t (&nt)[FM], const uint32_t (&nw)[FN]) {
#pragma unroll
    for (int b = 0; b < FM; ++b) {
      rt[b] = f8_unit_of(et[b]) * __builtin_amdgcn_rcpf(f8_unit_of(f8_exponent(nt[b])));
      et[b] = f8_exponent(nt[b]);
    }
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      rw[f] = f8_unit_of(ew[f]) * __builtin_amdgcn_rcpf(f8_unit_of(f8_exponent(nw[f])));
      ew[f] = f8_exponent(nw[f]);
    }
  };

#pragma unroll
  for (int b = 0; b < FM; ++b) et[b] = 0;
#pragma unroll
  for (int f = 0; f < FN; ++f) ew[f] = 0;
  load_scales(0);
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int i = 0; i < NI; ++i) load(s, min(s, S - 1), i);
  wait_lds_and_loads<NI * (NS - 1)>();
  raw_barrier();
  {
    uint32_t nt[FM], nw[FN];
    read_scales(0, nt, nw);
    next_units(nt, nw);
  }
#pragma unroll
  for (int f = 0; f < FN; ++f) wf[0][f] = frag_b(0, 0, f);
#pragma unroll
  for (int b = 0; b < FM; ++b) xa[b] = frag_a(0, 0, b);

  // no branch inside a stage: loads past the last one read it again, into the buffer
  // that is not read any more
  int cur = 0;  // buffer of stage s
  for (int c = 0; c < S; c += kChunkStages) {
    load_scales(c / kChunkStages + 1);
    if (BN == 256 && c + kChunkStages >= S && tid == 0) v = atomicAdd(turn, 1);
    for (int s = c; s < min(c + kChunkStages, S); ++s) {
      const int after = cur + 1 == NS ? 0 : cur + 1;
      // first step: the sums to this stage's units, the multiplications of one fragment
      // beside the MFMA of the one before
#pragma unroll
      for (int f = 0; f < FN; ++f) wf[1][f] = frag_b(cur, 1, f);
#pragma unroll
      for (int b = 0; b < FM; ++b) {
#pragma unroll
        for (int f = 0; f < FN; ++f) {
          const float r = rt[b] * rw[f];
#pragma unroll
          for (int q = 0; q < 16; ++q) acc[f][b][q] *= r;
          acc[f][b] = mfma_scaled(wf[0][f], xa[b], acc[f][b], ew[f], et[b]);
          __builtin_amdgcn_sched_barrier(0);
        }
        xa[b] = frag_a(cur, 1, b);
      }
      // every wavefront has this buffer's last fragments, and its loads of the next
      // stage have landed (those of later ones may be under way; a chunk's scales among
      // them only make the wait longer)
      wait_lds_and_loads<NI * (NS - 2)>();
      raw_barrier();
      __builtin_amdgcn_sched_barrier(0);
      uint32_t nt[FM], nw[FN];
      read_scales(min(s + 1, S - 1), nt, nw);
#pragma unroll
      for (int f = 0; f < FN; ++f) wf[0][f] = frag_b(after, 0, f);
#pragma unroll
      for (int b = 0; b < FM; ++b) {
#pragma unroll
        for (int f = 0; f < FN; ++f) {
          acc[f][b] = mfma_scaled(wf[1][f], xa[b], acc[f][b], ew[f], et[b]);
          __builtin_amdgcn_sched_barrier(0);
        }
        xa[b] = frag_a(after, 0, b);
#pragma unroll
        for (int i = b * NI / FM; i < (b + 1) * NI / FM; ++i) load(cur, min(s + NS, S - 1), i);
      }
      next_units(nt, nw);
      cur = after;
    }
  }
  __builtin_amdgcn_s_waitcnt(0);
  raw_barrier();

  // ---- epilogue: sum q of fragment (f, b) is column 32 f + 8 (q / 4) + 4 fk + q % 4 of
  // the wavefront (DUAL: of matrix f), token row 32 b + fr ----
  bool range = false;
  if constexpr (DUAL) {
    // h, its codes by blocks of 128 columns: the tile's.  A wavefront holds 32 of them;
    // their maxima meet in LDS.
    uint32_t* const s_top = reinterpret_cast<uint32_t*>(smem);  // [4][BM]
    float h[FM][16];
#pragma unroll
    for (int b = 0; b < FM; ++b) {
      uint32_t top = 0u;
      const float u0 = f8_unit_of(et[b]) * f8_unit_of(ew[0]), u1 = f8_unit_of(et[b]) * f8_unit_of(ew[1]);
      const bool in = n0 + wn * WN < N;   // (N is a multiple of 128)
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        h[b][q] = silu_mul_exact(acc[0][b][q] * u0, acc[1][b][q] * u1);
        top = max(top, f8_magnitude(h[b][q]));
      }
      const auto both = __builtin_amdgcn_permlane32_swap(top, top, false, false);
      top = max(top, (uint32_t)(fk ? both[0] : both[1]));
      if (fk == 0) s_top[wn * BM + wm * WM + b * 32 + fr] = in ? top : 0u;
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < FM; ++b) {
      const int m = wm * WM + b * 32 + fr;
      const uint32_t top = max(max(s_top[m], s_top[BM + m]), max(s_top[2 * BM + m], s_top[3 * BM + m]));
      const float amax = __uint_as_float(top);
      const F8Near blk = f8_near(amax);
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = f8_pack4(f8_code(h[b][4 * q], blk), f8_code(h[b][4 * q + 1], blk), f8_code(h[b][4 * q + 2], blk),
                        f8_code(h[b][4 * q + 3], blk));
      const auto s02 = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
      const auto s13 = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
      if (m >= rows) continue;
      range |= !(amax <= 3.402823466e38f);
      *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(a.out) + (size_t)(t.row0 + m) * N + n0 + wn * WN + 16 * fk) =
          u32x4{s02[0], s02[1], s13[0], s13[1]};
      if (wn == 0 && fk == 0) a.out_scales[(size_t)(n0 / kFp8Block) * a.out_group + t.row0 + m] = f8_scale(amax);
    }
  } else {
    // through LDS (16-byte chunks swizzled by row), stored as whole runs of a row
    constexpr int WC = FN * 32, CH = WC / 8;
    uint16_t* const part = reinterpret_cast<uint16_t*>(smem) + wave * (WM * WC);
    auto place = [&](int row, int ch) { return row * WC + ((ch ^ (CH == 8 ? row & 7 : (row >> 1) & 3)) << 3); };
    auto lay = [&](auto f16) {
#pragma unroll
      for (int b = 0; b < FM; ++b) {
        const bool real = wm * WM + b * 32 + fr < rows;
#pragma unroll
        for (int f = 0; f < FN; ++f) {
          const float u = f8_unit_of(et[b]) * f8_unit_of(ew[f]);
#pragma unroll
          for (int qi = 0; qi < 4; ++qi) {
            f32x4 v;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = acc[f][b][4 * qi + q] * u;
            u32x2 w;
            if constexpr (f16.value) {
              const bool in = n0 + wn * WC + f * 32 + 8 * qi < N;
#pragma unroll
              for (int q = 0; q < 4; ++q) range |= real && in && !(fabsf(v[q]) <= 65504.f);
              w = __builtin_bit_cast(u32x2, __builtin_convertvector(v, f16x4));
            } else {
              w = __builtin_bit_cast(u32x2, __builtin_convertvector(v, bf16x4));
            }
            *reinterpret_cast<u32x2*>(part + place(b * 32 + fr, f * 4 + qi) + 4 * fk) = w;
          }
        }
      }
    };
    if (a.y_dtype == MOE_F16) lay(std::true_type{});
    else lay(std::false_type{});
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    constexpr int RPL = 64 / CH;
#pragma unroll
    for (int i = 0; i < WM / RPL; ++i) {
      const int r = i * RPL + lane / CH, ch = lane % CH;
      const u32x4 v = *reinterpret_cast<const u32x4*>(part + place(r, ch));
      const int m = wm * WM + r, n = n0 + wn * WC + 8 * ch;
      if (m < rows && n < N)
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + (size_t)(t.row0 + m) * N + n) = v;
    }
  }
  if (range && a.flags) atomicOr(a.flags, (uint32_t)(DUAL ? MOE_FLAG_H_RANGE : MOE_FLAG_Y_RANGE));
}

// Tile L of the schedule's row tiles x cols columns: the tiles of an expert's
// neighbouring row tiles come column by column, so that an XCD reads a weight column once
// for all of them.
__device__ __forceinline__ MTile tile_at(const MTile* __restrict__ sched, int L, int cols, int& col) {
  const int at = L / cols, group = sched[at].group;
  const int first = at - (group & 0xFF), size = group >> 8;
  const int r = L - first * cols;
  col = r / size;
  MTile t = sched[first + (r - col * size)];
  t.expert = __builtin_amdgcn_readfirstlane(t.expert);
  t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
  t.rows = __builtin_amdgcn_readfirstlane(t.rows);
  col = __builtin_amdgcn_readfirstlane(col);
  return t;
}

// Row tiles of up to 256 rows, each at the height its rows need, 256 weight rows.  One
// block per compute unit; a block's first tile is its own, the others it draws: against a
// launch of a block per tile, whose XCDs end at different times, FFN of 8192 rows over 8
// experts, 4096 x 14336, 1905 -> 1690 us, of 8192 tokens over 256 experts 4270 -> 4100.
template <bool DUAL>
__global__ __launch_bounds__(512) void k_gemm_fp8(const Fp8Args a, int cols) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  constexpr int BN = 256;
  const int x = blockIdx.x & 7;
  int32_t* const next = a.count + (DUAL ? kFp8QueueUp : kFp8QueueDown);
  const Queue queue{next, a.count[1] * cols, a.count[0] * cols};
  int32_t* const s_tile = reinterpret_cast<int32_t*>(smem);
  int v = blockIdx.x >> 3;  // (the queues begin behind the blocks' own turns)
  for (;;) {
    if (threadIdx.x == 0) *s_tile = queue.tile(x, v);
    __syncthreads();
    const int L = __builtin_amdgcn_readfirstlane(*s_tile);
    __syncthreads();  // (the tile's loads overwrite it)
    if (L < 0) return;
    int ni;
    const MTile t = tile_at(a.sched, L, cols, ni);
    if (t.rows <= 0) {  // (a quarter behind a short tile)
      if (threadIdx.x == 0) v = atomicAdd(next + x, 1);
    } else if (t.rows <= 64) {
      tile_fp8<64, BN, DUAL>(smem, a, t, ni, next + x, v);
    } else if (t.rows <= 128) {
      tile_fp8<128, BN, DUAL>(smem, a, t, ni, next + x, v);
    } else if (t.rows <= 192) {
      tile_fp8<192, BN, DUAL>(smem, a, t, ni, next + x, v);
    } else {
      tile_fp8<256, BN, DUAL>(smem, a, t, ni, next + x, v);
    }
    __syncthreads();
  }
}

// The same on 128 weight rows, a row tile taken as two of up to 128: for launches of few
// tiles, one each of blocks that fit a compute unit twice (blocks that draw their tiles pile
// up two on a compute unit while others idle: 62 instead of 34 us for 1024 rows x 4096 x 4096).
__global__ __launch_bounds__(512, 4) void k_gemm_fp8_halves(const Fp8Args a, int cols) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int real = a.count[0] * 2 * cols, per = (real + 7) >> 3, slot = blockIdx.x >> 3;
  const int L = (blockIdx.x & 7) * per + slot;  // (an XCD's share, as in a queue)
  if (slot >= per || L >= real) return;
  int col, none = 0;
  MTile t = tile_at(a.sched, L, 2 * cols, col);
  t.row0 += 128 * (col & 1);
  t.rows = min(t.rows - 128 * (col & 1), 128);
  if (t.rows <= 0) return;
  if (t.rows <= 64) tile_fp8<64, 128, false>(smem, a, t, col >> 1, nullptr, none);
  else tile_fp8<128, 128, false>(smem, a, t, col >> 1, nullptr, none);
}

template <typename F>
hipError_t launch_tiles(F* kernel, int lds, std::atomic<uint64_t>& set_on, long long grid, const Fp8Args& a, int cols,
                        hipStream_t st) {
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), lds, set_on);
  if (e != hipSuccess) return e;
  if (grid > 0x7fffff) return hipErrorInvalidValue;  // (2^32 threads of one axis)
  hipLaunchKernelGGL(*kernel, dim3((unsigned)grid), dim3(512), lds, st, a, cols);
  return hipGetLastError();
}

// Row tiles of up to 256 rows in expert order, the queues at their beginning and the flag
// word cleared.  fill_cols > 0: the column tiles of a launch; when a few rounds of its tiles on
// all compute units would end with one that keeps at most a quarter of them busy, that
// round's row tiles are cut into kFillSplit (some parts without rows).
// offsets null: rows [0, static_rows) of one expert.
__global__ __launch_bounds__(512) void k_schedule_fp8(const int32_t* __restrict__ offsets, int E, int static_rows,
                                                      MTile* __restrict__ sched, int max_tiles,
                                                      int32_t* __restrict__ count, uint32_t* __restrict__ flags,
                                                      int fill_cols) {
  __shared__ int s_wave[8];
  const int tid = threadIdx.x, lane = tid & 63;
  if (tid == 0) *flags = 0u;
  if (tid >= 2 && tid < kFp8CountWords)
    count[tid] = (tid - kFp8QueueUp) < 8u || (tid - kFp8QueueDown) < 8u ? kUnits / 8 : 0;
  int r0 = 0, kept = 0;
  if (tid < E) {
    r0 = offsets ? offsets[tid] : 0;
    kept = (offsets ? offsets[tid + 1] : static_rows) - r0;
  }
  const int nb = (kept + 255) / 256;
  int upto = nb;  // tiles of the experts up to this one
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(upto, off, 64);
    if (lane >= off) upto += o;
  }
  if (lane == 63) s_wave[tid >> 6] = upto;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    if (w < (tid >> 6)) upto += s_wave[w];
    total += s_wave[w];
  }
  int whole = total;
  if (fill_cols > 0) {
    const long long blocks = (long long)total * fill_cols;
    const int rest = (int)(blocks % kUnits), turn = (rest + fill_cols - 1) / fill_cols;
    if (rest > 0 && blocks > kUnits && blocks < 5 * kUnits && turn * fill_cols * kFillSplit <= kUnits)
      whole = total - turn;
  }
  const int begin = upto - nb, uncut = min(max(whole - begin, 0), nb);
  for (int i = 0; i < nb; ++i) {
    const int slot = begin + i;
    if (i < uncut) {
      const int g = i / kTileGroup * kTileGroup;
      if (slot < max_tiles)
        sched[slot] = MTile{tid, r0 + 256 * i, min(256, kept - 256 * i), tile_group(i - g, min(kTileGroup, uncut - g))};
    } else {
      constexpr int part = 256 / kFillSplit;
      for (int q = 0; q < kFillSplit; ++q) {
        const int at = whole + (slot - whole) * kFillSplit + q;
        if (at < max_tiles)
          sched[at] = MTile{tid, r0 + 256 * i + q * part, max(0, min(part, kept - 256 * i - q * part)),
                            tile_group(q, kFillSplit)};
      }
    }
  }
  if (tid == 0) {
    count[0] = min(whole + (total - whole) * kFillSplit, max_tiles);
    count[1] = min(whole, max_tiles);
  }
}

}  // namespace

hipError_t launch_schedule_fp8(const int32_t* offsets, int E, int static_rows, MTile* sched, int max_tiles,
                               int32_t* count, uint32_t* flags, int fill_cols, hipStream_t st) {
  hipLaunchKernelGGL(k_schedule_fp8, dim3(1), dim3(512), 0, st, offsets, E, static_rows, sched, max_tiles, count,
                     flags, fill_cols);
  return hipGetLastError();
}

hipError_t launch_gemm_fp8(const Fp8Args& a, bool dual, bool halves, int row_tiles, hipStream_t st) {
  static std::atomic<uint64_t> set_up{0}, set_down{0}, set_halves{0};
  constexpr int lds = max_of(tile_lds(128, 256), tile_lds(256, 256));  // (64 and 192 rows take less)
  constexpr int lds_halves = max_of(tile_lds(64, 128), tile_lds(128, 128));
  static_assert(lds <= 160 * 1024 && lds_halves <= 80 * 1024, "LDS");
  if (dual) return launch_tiles(k_gemm_fp8<true>, lds, set_up, kUnits, a, (a.N + 127) / 128, st);
  if (!halves) return launch_tiles(k_gemm_fp8<false>, lds, set_down, kUnits, a, (a.N + 255) / 256, st);
  const int cols = (a.N + 127) / 128;
  return launch_tiles(k_gemm_fp8_halves, lds_halves, set_halves, ((long long)row_tiles * 2 * cols + 7) / 8 * 8, a, cols, st);
}

}  // namespace moe
