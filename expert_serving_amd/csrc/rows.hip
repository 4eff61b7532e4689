// Token rows to expert order and back: rows times a weight per slot or quantised to
// 8-bit floating-point blocks on the way to their experts, and the gradients of the
// dispatch and of the gate-weighted combine ("Expert Parallelism: MoE model parallel
// split", section 3 and section 12 Q2: k copies of a token's hidden state out, k
// outputs back).
//
// All are bound by memory: a token's row is read once for its k slots, an expert's row
// once, each written once.  Every row belongs to one slot, so nothing is added with
// atomics: sums over a token's slots run in slot order inside a thread.
//
// Measured (device time of calls in a row; a copy of this memory runs at 4.9 TB/s): 8192 tokens x
// 7168 of bf16, top 8: to codes 130 us, 4.6 TB/s; gradient of the dispatch 211 us, 5.0 TB/s; gradient of the combine with both
// outputs 428 us, 4.9 TB/s; 4099 x 4096 with weights, top 2: 22.7 us, 4.4 TB/s.  One token: 5 us, the
// launch and one chain of loads.
#include <type_traits>

#include "half_bits.h"
#include "moe_internal.h"
#include "quant_fp8.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int type_bytes(int dt) { return dt == MOE_F32 ? 4 : 2; }

// two 16-bit values of a word
template <int DT>
__device__ __forceinline__ void widen2(uint32_t x, float& a, float& b) {
  if constexpr (DT == MOE_BF16) {
    a = __uint_as_float(x << 16);
    b = __uint_as_float(x & 0xFFFF0000u);
  } else {
    const f16x2 h = __builtin_bit_cast(f16x2, x);
    a = (float)h[0];
    b = (float)h[1];
  }
}

// N consecutive values (N 4 or 8, element i a multiple of N) as they lie in memory
template <int DT, int N>
struct Raw {
  static constexpr int kWords = N * type_bytes(DT) / 4;
  uint32_t w[kWords];
};

template <int DT, int N>
__device__ __forceinline__ Raw<DT, N> load_raw(const void* p, size_t i) {
  constexpr int W = Raw<DT, N>::kWords;
  const char* s = static_cast<const char*>(p) + i * type_bytes(DT);
  Raw<DT, N> r;
  if constexpr (W >= 4) {
#pragma unroll
    for (int q = 0; q < W; q += 4) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(s + 4 * q);
      r.w[q] = v[0], r.w[q + 1] = v[1], r.w[q + 2] = v[2], r.w[q + 3] = v[3];
    }
  } else {
    const u32x2 v = *reinterpret_cast<const u32x2*>(s);
    r.w[0] = v[0], r.w[1] = v[1];
  }
  return r;
}

template <int DT, int N>
__device__ __forceinline__ void store_raw(void* p, size_t i, const Raw<DT, N>& r) {
  constexpr int W = Raw<DT, N>::kWords;
  char* d = static_cast<char*>(p) + i * type_bytes(DT);
  if constexpr (W >= 4) {
#pragma unroll
    for (int q = 0; q < W; q += 4)
      *reinterpret_cast<u32x4*>(d + 4 * q) = u32x4{r.w[q], r.w[q + 1], r.w[q + 2], r.w[q + 3]};
  } else {
    *reinterpret_cast<u32x2*>(d) = u32x2{r.w[0], r.w[1]};
  }
}

template <int DT, int N>
__device__ __forceinline__ void widen(const Raw<DT, N>& r, float* f) {
#pragma unroll
  for (int q = 0; q < Raw<DT, N>::kWords; ++q) {
    const uint32_t x = r.w[q];
    if constexpr (DT == MOE_F32) f[q] = __uint_as_float(x);
    else widen2<DT>(x, f[2 * q], f[2 * q + 1]);
  }
}

template <int DT, int N>
__device__ __forceinline__ Raw<DT, N> narrow(const float* f) {
  Raw<DT, N> r;
#pragma unroll
  for (int q = 0; q < Raw<DT, N>::kWords; ++q) {
    if constexpr (DT == MOE_F32) r.w[q] = __float_as_uint(f[q]);
    else if constexpr (DT == MOE_BF16) r.w[q] = bf16_bits(f[2 * q]) | (bf16_bits(f[2 * q + 1]) << 16);
    else r.w[q] = f16_bits(f[2 * q]) | (f16_bits(f[2 * q + 1]) << 16);
  }
  return r;
}

constexpr int granule(int dt) { return dt == MOE_F32 ? 4 : 8; }  // values of 16 bytes

// the row of slot (t, j), or -1 where it has none inside [0, num_rows)
__device__ __forceinline__ int slot_row(const int32_t* __restrict__ row_of_slot, int t, int j, int k, int num_rows) {
  if (j >= k) return -1;
  const int r = row_of_slot[(size_t)t * k + j];
  return (uint32_t)r < (uint32_t)num_rows ? r : -1;
}

// ---- rows to expert order -------------------------------------------------------

// One thread per 16 bytes of a token's row, over all tokens.
template <int DT, int KM, bool WEIGHTED>
__global__ __launch_bounds__(256) void k_dispatch_rows(int items, int granules, int H, int k, const void* __restrict__ x,
                                                       const int32_t* __restrict__ row_of_slot,
                                                       const float* __restrict__ weights, int num_rows,
                                                       void* __restrict__ out) {
  constexpr int G = granule(DT);
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= items) return;
  const int t = i / granules, c = (i - t * granules) * G;
  int row[KM];
  float w[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    row[j] = slot_row(row_of_slot, t, j, k, num_rows);
    if constexpr (WEIGHTED) w[j] = j < k ? weights[(size_t)t * k + j] : 0.f;
  }
  const Raw<DT, G> v = load_raw<DT, G>(x, (size_t)t * H + c);
  float f[G];
  if constexpr (WEIGHTED) widen<DT, G>(v, f);
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    if (row[j] < 0) continue;
    Raw<DT, G> o = v;
    if constexpr (WEIGHTED) {
      float p[G];
#pragma unroll
      for (int q = 0; q < G; ++q) p[q] = f[q] * w[j];
      o = narrow<DT, G>(p);
    }
    store_raw<DT, G>(out, (size_t)row[j] * H + c, o);
  }
}

// 16 values of element 16 i of a matrix to codes; the eight lanes of a block share its
// maximum.  Returns the block's scale.
template <int DT>
__device__ __forceinline__ float quantise16(const void* __restrict__ src, size_t i, u32x4& codes) {
  float f[16];
  const Raw<DT, 8> a = load_raw<DT, 8>(src, 16 * i), b = load_raw<DT, 8>(src, 16 * i + 8);
  widen<DT, 8>(a, f);
  widen<DT, 8>(b, f + 8);
  uint32_t top = 0u;
#pragma unroll
  for (int q = 0; q < 16; ++q) top = max(top, f8_magnitude(f[q]));
#pragma unroll
  for (int off = 1; off < 8; off <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
  const float amax = __uint_as_float(top);
  const F8Block blk = f8_block(amax);
#pragma unroll
  for (int q = 0; q < 16; ++q) f[q] = f8_quotient(f[q], blk);
#pragma unroll
  for (int q = 0; q < 4; ++q) codes[q] = f8_pack4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
  return f8_scale(amax);
}

// A thread takes 16 columns of a token's row: eight lanes one block of 128 (rows are
// whole blocks, so those eight lanes are in range together).
template <int DT, int KM>
__global__ __launch_bounds__(256) void k_dispatch_rows_fp8(int items, int H, int k, const void* __restrict__ x,
                                                           const int32_t* __restrict__ row_of_slot, int num_rows,
                                                           uint8_t* __restrict__ codes, float* __restrict__ scales) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= items) return;
  const int per_row = H / 16, t = i / per_row, c = i - t * per_row;
  int row[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) row[j] = slot_row(row_of_slot, t, j, k, num_rows);
  u32x4 w;
  const float scale = quantise16<DT>(x, (size_t)i, w);
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    if (row[j] < 0) continue;
    *reinterpret_cast<u32x4*>(codes + (size_t)row[j] * H + 16 * c) = w;
    if ((c & 7) == 0) scales[(size_t)row[j] * (H / kFp8Block) + (c >> 3)] = scale;
  }
}

// The same on a matrix of whole blocks, in its own order: block b of 128 elements has
// scale b.  8192 x 14336 of bf16 59 us, 6.0 TB/s (two thirds of it reads).
template <int DT>
__global__ __launch_bounds__(256) void k_quant_fp8(long long items, int per_row, const int32_t* __restrict__ rows_dev,
                                                   const void* __restrict__ src, uint8_t* __restrict__ codes,
                                                   float* __restrict__ scales, uint32_t* __restrict__ h_flags) {
  const long long step = (long long)gridDim.x * 256;
  if (rows_dev) items = min(items, (long long)*rows_dev * per_row);
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < items; i += step) {
    u32x4 w;
    const float scale = quantise16<DT>(src, (size_t)i, w);
    *reinterpret_cast<u32x4*>(codes + 16 * i) = w;
    if ((i & 7) == 0) {
      scales[i >> 3] = scale;
      if (h_flags && !(scale <= 3.402823466e38f)) atomicOr(h_flags, (uint32_t)MOE_FLAG_H_RANGE);
    }
  }
}

// One block per 128 x 128 block of a weight matrix (fewer rows at its end); a thread
// holds 64 values, 16 columns of four rows.  Done once per weight; bound by memory: 8 x
// 14336 x 4096 of bf16 259 us, 5.4 TB/s, 128 x 768 x 2048 117 us, 1 x 4096 x 4096 11.5 us.
template <int DT>
__global__ __launch_bounds__(256) void k_quant_fp8_weights(int n, int k, const void* __restrict__ src,
                                                           uint8_t* __restrict__ codes, float* __restrict__ scales) {
  const int kb = blockIdx.x, nb = blockIdx.y, e = blockIdx.z;
  const int c = (threadIdx.x & 7) * 16;
  float f[4][16];
  uint32_t top = 0u;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int r = nb * kFp8Block + (threadIdx.x >> 3) + 32 * q;
    if (r >= n) continue;
    const size_t i = ((size_t)e * n + r) * k + (size_t)kb * kFp8Block + c;
    widen<DT, 8>(load_raw<DT, 8>(src, i), f[q]);
    widen<DT, 8>(load_raw<DT, 8>(src, i + 8), f[q] + 8);
#pragma unroll
    for (int j = 0; j < 16; ++j) top = max(top, f8_magnitude(f[q][j]));
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
  __shared__ uint32_t s_top[4];
  if ((threadIdx.x & 63) == 0) s_top[threadIdx.x >> 6] = top;
  __syncthreads();
  const float amax = __uint_as_float(max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3])));
  const F8Block blk = f8_block(amax);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int r = nb * kFp8Block + (threadIdx.x >> 3) + 32 * q;
    if (r >= n) continue;
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = f8_pack4(f8_quotient(f[q][4 * j], blk), f8_quotient(f[q][4 * j + 1], blk),
                      f8_quotient(f[q][4 * j + 2], blk), f8_quotient(f[q][4 * j + 3], blk));
    *reinterpret_cast<u32x4*>(codes + ((size_t)e * n + r) * k + (size_t)kb * kFp8Block + c) = w;
  }
  if (threadIdx.x == 0) scales[((size_t)e * gridDim.y + nb) * gridDim.x + kb] = f8_scale(amax);
}

// ---- gradients ------------------------------------------------------------------

// Blocks of one token each in a grid whose first axis stays below 2^32 threads.
constexpr int kGridTokens = 1 << 21;
inline dim3 token_grid(int tokens) {
  return dim3(tokens < kGridTokens ? tokens : kGridTokens, (unsigned)((tokens + (long long)kGridTokens - 1) / kGridTokens));
}
__device__ __forceinline__ int grid_token() {
  const uint32_t t = blockIdx.y * (uint32_t)kGridTokens + blockIdx.x;
  return t < 0x7FFFFFFFu ? (int)t : 0x7FFFFFFF;
}

// One token per block; a thread takes granule g % NT of the token's k rows (row type
// DR) and, where it needs them, of the token's own row (type DT).
//   BACK (gradient of the dispatch): sum_out[t] = sum_j weight_j row_j;
//   else (gradient of the combine):  row_out_j = weight_j token[t];
//   DOT: dots[t][j] = <row_j, token[t]>, summed over the thread's granules, its
//        wavefront and the block's wavefronts, always in that order.
// KM bounds k, so that a granule's loads of all rows are in flight together.  A slot
// without a row loads the row of a slot that has one and does not use it.  rows may be
// out: a thread loads a granule of every row before it stores the first.
template <int DR, int DT, int KM, bool BACK, bool DOT, bool WEIGHTED, int NT>
__global__ __launch_bounds__(NT) void k_slots(int T, int H, int k, const void* rows,
                                              const int32_t* __restrict__ row_of_slot, int num_rows,
                                              const float* __restrict__ weights, const void* __restrict__ token,
                                              void* out, float* __restrict__ dots) {
  constexpr int G = granule(DR);
  constexpr bool READ_ROWS = BACK || DOT, READ_TOKEN = !BACK || DOT;
  const int t = grid_token();
  if (t >= T) return;
  int row[KM], at[KM], any = -1;
  float w[KM], dot[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    row[j] = slot_row(row_of_slot, t, j, k, num_rows);
    w[j] = WEIGHTED && row[j] >= 0 ? weights[(size_t)t * k + j] : 1.f;
    dot[j] = 0.f;
    if (row[j] >= 0) any = row[j];
  }
#pragma unroll
  for (int j = 0; j < KM; ++j) at[j] = row[j] >= 0 ? row[j] : any;
  const int granules = H / G;
  for (int g = threadIdx.x; g < granules; g += NT) {
    const size_t c = (size_t)g * G;
    Raw<DR, G> raw[KM];
    float f[G];
    if constexpr (READ_ROWS) {
      if (any >= 0) {
#pragma unroll
        for (int j = 0; j < KM; ++j) raw[j] = load_raw<DR, G>(rows, (size_t)at[j] * H + c);
      }
    }
    if constexpr (READ_TOKEN) widen<DT, G>(load_raw<DT, G>(token, (size_t)t * H + c), f);
    float sum[G];
#pragma unroll
    for (int q = 0; q < G; ++q) sum[q] = 0.f;
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      if (row[j] < 0) continue;
      float v[G];
      if constexpr (READ_ROWS) widen<DR, G>(raw[j], v);
      if constexpr (DOT) {
#pragma unroll
        for (int q = 0; q < G; ++q) dot[j] = fmaf(v[q], f[q], dot[j]);
      }
      if constexpr (BACK) {
#pragma unroll
        for (int q = 0; q < G; ++q) sum[q] = WEIGHTED ? fmaf(w[j], v[q], sum[q]) : sum[q] + v[q];
      } else {
        if (out) {
          float p[G];
#pragma unroll
          for (int q = 0; q < G; ++q) p[q] = w[j] * f[q];
          store_raw<DR, G>(out, (size_t)row[j] * H + c, narrow<DR, G>(p));
        }
      }
    }
    if constexpr (BACK) {
      if (out) store_raw<DR, G>(out, (size_t)t * H + c, narrow<DR, G>(sum));
    }
  }
  if constexpr (DOT) {
    // a step gives half of the lanes half of the slots each: KM + 5 - log2 KM exchanges in
    // place of 6 KM (gradient of the combine of 64 x 2048 fp32, 8 slots: 7.3 -> 6.8 us), lane l ends with slot l / (64 / KM)
    __shared__ float s_dot[NT / 64][KM];
    const int lane = threadIdx.x & 63;
    int off = 32;
#pragma unroll
    for (int half = KM / 2; half >= 1; half /= 2, off /= 2) {
      const bool upper = lane & off;
#pragma unroll
      for (int j = 0; j < half; ++j) {
        const float keep = upper ? dot[j + half] : dot[j], give = upper ? dot[j] : dot[j + half];
        dot[j] = keep + __shfl_xor(give, off, 64);
      }
    }
#pragma unroll
    for (; off >= 1; off /= 2) dot[0] += __shfl_xor(dot[0], off, 64);
    if (lane % (64 / KM) == 0) s_dot[threadIdx.x >> 6][lane / (64 / KM)] = dot[0];
    __syncthreads();
    if ((int)threadIdx.x < k) {
      float s = s_dot[0][threadIdx.x];
#pragma unroll
      for (int v = 1; v < NT / 64; ++v) s += s_dot[v][threadIdx.x];
      dots[(size_t)t * k + threadIdx.x] = s;
    }
  }
}

template <int DR, int DT, int KM, bool BACK, bool DOT, bool WEIGHTED>
hipError_t launch_slots_nt(int T, int H, int k, const void* rows, const int32_t* row_of_slot, int num_rows,
                           const float* weights, const void* token, void* out, float* dots, hipStream_t st) {
  const int granules = H / granule(DR);
#define MOE_SLOTS(NT)                                                                                         \
  hipLaunchKernelGGL((k_slots<DR, DT, KM, BACK, DOT, WEIGHTED, NT>), token_grid(T), dim3(NT), 0, st, T, H, k, \
                     rows, row_of_slot, num_rows, weights, token, out, dots)
  // Threads per token.  A short row leaves the many threads' dot products to join with
  // nothing to do, few tokens leave compute units to the threads of one, and a long row keeps
  // 512 busy.  Measured, gradient of the combine with both outputs, 64 / 256 / 512 threads: 4096
  // tokens x 512, 8 slots (64 granules) 16.3 / 22.4 / 37.1 us, x 1024 (128) 25.7 / 28.0 / 38.8, x 2048
  // (256) 51.8 / 48.0 / 55.4; 8192 x 7168 (896) 411 / 409 / 406; 1 x 7168 36.6 / 13.6 / 10.0; 64 x
  // 2048 of fp32 (512) 17.2 / 8.3 / 7.1.
  if (granules <= 128) MOE_SLOTS(64);
  else if (granules >= 512 || T <= kUnits) MOE_SLOTS(512);
  else MOE_SLOTS(256);
#undef MOE_SLOTS
  return hipGetLastError();
}

// f(std::integral_constant<int, KM>) for the smallest bound KM of k
template <typename F>
hipError_t with_bound(int k, F&& f) {
  if (k <= 2) return f(std::integral_constant<int, 2>{});
  if (k <= 4) return f(std::integral_constant<int, 4>{});
  if (k <= 8) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, kMaxTopK>{});
}
template <typename F>
hipError_t with_type(int dtype, F&& f) {
  if (dtype == MOE_F32) return f(std::integral_constant<int, MOE_F32>{});
  if (dtype == MOE_F16) return f(std::integral_constant<int, MOE_F16>{});
  return f(std::integral_constant<int, MOE_BF16>{});
}

}  // namespace

hipError_t launch_dispatch_rows(const moe_shape& s, int dtype, const void* x, const int32_t* row_of_slot,
                                const float* weights, int num_rows, void* out, hipStream_t st) {
  const int granules = s.hidden / granule(dtype), items = s.num_tokens * granules;  // (T * H fits an int)
  return with_type(dtype, [&](auto dt) {
    return with_bound(s.top_k, [&](auto km) {
      const dim3 grid((items + 255) / 256), block(256);
      if (weights)
        hipLaunchKernelGGL((k_dispatch_rows<dt.value, km.value, true>), grid, block, 0, st, items, granules, s.hidden,
                           s.top_k, x, row_of_slot, weights, num_rows, out);
      else
        hipLaunchKernelGGL((k_dispatch_rows<dt.value, km.value, false>), grid, block, 0, st, items, granules, s.hidden,
                           s.top_k, x, row_of_slot, weights, num_rows, out);
      return hipGetLastError();
    });
  });
}

hipError_t launch_dispatch_rows_fp8(const moe_shape& s, int dtype, const void* x, const int32_t* row_of_slot,
                                    int num_rows, void* codes, float* scales, hipStream_t st) {
  const int items = s.num_tokens * (s.hidden / 16);
  return with_type(dtype, [&](auto dt) {
    return with_bound(s.top_k, [&](auto km) {
      hipLaunchKernelGGL((k_dispatch_rows_fp8<dt.value, km.value>), dim3((items + 255) / 256), dim3(256), 0, st, items,
                         s.hidden, s.top_k, x, row_of_slot, num_rows, static_cast<uint8_t*>(codes), scales);
      return hipGetLastError();
    });
  });
}

hipError_t launch_quant_fp8(int src_dtype, const void* src, int rows, int cols, const int32_t* rows_dev, void* codes,
                            float* scales, hipStream_t st, uint32_t* h_flags) {
  const long long items = (long long)rows * (cols / 16), blocks = (items + 255) / 256;
  if (items <= 0) return hipSuccess;
  return with_type(src_dtype, [&](auto dt) {
    hipLaunchKernelGGL(k_quant_fp8<dt.value>, dim3((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20)), dim3(256), 0, st,
                       items, cols / 16, rows_dev, src, static_cast<uint8_t*>(codes), scales, h_flags);
    return hipGetLastError();
  });
}

hipError_t launch_quant_fp8_weights(int src_dtype, const void* src, int experts, int n, int k, void* codes,
                                    float* scales, hipStream_t st) {
  const dim3 grid(k / kFp8Block, (n + kFp8Block - 1) / kFp8Block, experts);
  return with_type(src_dtype, [&](auto dt) {
    hipLaunchKernelGGL(k_quant_fp8_weights<dt.value>, grid, dim3(256), 0, st, n, k, src, static_cast<uint8_t*>(codes),
                       scales);
    return hipGetLastError();
  });
}

hipError_t launch_dispatch_rows_backward(const moe_shape& s, int dtype, const void* d_perm, const int32_t* row_of_slot,
                                         int num_rows, const float* weights, const void* x, void* d_x,
                                         float* d_weights, hipStream_t st) {
  return with_type(dtype, [&](auto dt) {
    return with_bound(s.top_k, [&](auto km) {
      constexpr int D = dt.value, KM = km.value;
      if (!weights)
        return launch_slots_nt<D, D, KM, true, false, false>(s.num_tokens, s.hidden, s.top_k, d_perm, row_of_slot,
                                                             num_rows, nullptr, nullptr, d_x, nullptr, st);
      if (!d_weights)
        return launch_slots_nt<D, D, KM, true, false, true>(s.num_tokens, s.hidden, s.top_k, d_perm, row_of_slot,
                                                            num_rows, weights, nullptr, d_x, nullptr, st);
      return launch_slots_nt<D, D, KM, true, true, true>(s.num_tokens, s.hidden, s.top_k, d_perm, row_of_slot,
                                                         num_rows, weights, x, d_x, d_weights, st);
    });
  });
}

hipError_t launch_combine_backward(const moe_shape& s, int out_dtype, const void* d_out, int y_dtype, const void* y,
                                   const int32_t* row_of_slot, const float* gates, int num_rows, void* d_y,
                                   float* d_gates, hipStream_t st) {
  return with_type(y_dtype, [&](auto dr) {
    return with_type(out_dtype, [&](auto dt) {
      return with_bound(s.top_k, [&](auto km) {
        constexpr int DR = dr.value, DT = dt.value, KM = km.value;
        if (d_gates)
          return launch_slots_nt<DR, DT, KM, false, true, true>(s.num_tokens, s.hidden, s.top_k, y, row_of_slot,
                                                                num_rows, gates, d_out, d_y, d_gates, st);
        return launch_slots_nt<DR, DT, KM, false, false, true>(s.num_tokens, s.hidden, s.top_k, y, row_of_slot,
                                                               num_rows, gates, d_out, d_y, nullptr, st);
      });
    });
  });
}

}  // namespace moe
