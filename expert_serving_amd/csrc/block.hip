// The row operators around the layer: the RMS norm in front of it (with the
// int8 quantisation of its rows), the quantisation alone, and the end of the
// block -- the gate-weighted combine with the norm behind the layer, the gate
// and the scaled residual.
//
// All are bound by memory: every value is read once and kept in registers
// between the pass that reduces over its row and the pass that writes it.  One
// block takes one row; a thread owns granules of 16 loaded bytes (8 values of 2
// bytes, 4 of 4), granule g of the row in thread g % NT, V of them per thread.
// Rows too long for that (V = 0) are read a second time.
// Measured: norm of 8192 x 7168 fp32 to bf16 71.5 us (352 MB, 4.9 TB/s, a device copy
// 4.7), to bf16 and codes 82.5 us (411 MB, 5.0 TB/s), of bf16 to both 64 us (294 MB,
// 4.6 TB/s); 65536 x 1024 fp16 to codes 41 us (4.9 TB/s); combine of 8192 x 7168, eight
// slots and a shared expert, with norm, gate and residual 282 us (1.39 GB, 4.9
// TB/s); 64 rows of 4096 in 4.9 us, of which the launch takes 4.7.
#include "moe_internal.h"
#include "quant_int8.h"
#include "swiglu.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t f32_to_bf16_rne(float f) {
  const uint32_t b = __float_as_uint(f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return (b >> 16) | 0x40u;  // NaN stays NaN
  return (b + (((b >> 16) & 1u) + 0x7FFFu)) >> 16;
}

// values of one 16-byte granule of a type
constexpr int granule(int dt) { return dt == MOE_F32 ? 4 : 8; }

template <int DT>
__device__ __forceinline__ u32x4 load_raw(const void* p, size_t i) {
  return *reinterpret_cast<const u32x4*>(static_cast<const char*>(p) + i * (DT == MOE_F32 ? 4 : 2));
}

template <int DT>
__device__ __forceinline__ void widen(const u32x4 w, float* f) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t x = w[q];
    if constexpr (DT == MOE_F32) {
      f[q] = __uint_as_float(x);
    } else {
      if constexpr (DT == MOE_BF16) {
        f[2 * q] = __uint_as_float(x << 16);
        f[2 * q + 1] = __uint_as_float(x & 0xFFFF0000u);
      } else {
        const f16x2 h = __builtin_bit_cast(f16x2, x);
        f[2 * q] = (float)h[0];
        f[2 * q + 1] = (float)h[1];
      }
    }
  }
}

template <int DT>
__device__ __forceinline__ void load_granule(const void* p, size_t i, float* f) {
  widen<DT>(load_raw<DT>(p, i), f);
}

// N consecutive fp32 or bf16 values at element i (i a multiple of N, N 4 or 8)
template <int N>
__device__ __forceinline__ void load_stream(const void* p, bool bf16, size_t i, float* f) {
  if (bf16) {
    const uint16_t* s = static_cast<const uint16_t*>(p) + i;
#pragma unroll
    for (int q = 0; q < N; q += 4) {
      const u32x2 w = *reinterpret_cast<const u32x2*>(s + q);
      f[q] = __uint_as_float(w[0] << 16), f[q + 1] = __uint_as_float(w[0] & 0xFFFF0000u);
      f[q + 2] = __uint_as_float(w[1] << 16), f[q + 3] = __uint_as_float(w[1] & 0xFFFF0000u);
    }
  } else {
    const float* s = static_cast<const float*>(p) + i;
#pragma unroll
    for (int q = 0; q < N; q += 4) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(s + q);
      f[q] = v[0], f[q + 1] = v[1], f[q + 2] = v[2], f[q + 3] = v[3];
    }
  }
}

template <int N>
__device__ __forceinline__ void store_stream(void* p, bool bf16, size_t i, const float* f) {
  if (bf16) {
    uint32_t w[N / 2];
#pragma unroll
    for (int q = 0; q < N / 2; ++q) w[q] = f32_to_bf16_rne(f[2 * q]) | (f32_to_bf16_rne(f[2 * q + 1]) << 16);
    uint16_t* d = static_cast<uint16_t*>(p) + i;
    if constexpr (N == 8) *reinterpret_cast<u32x4*>(d) = u32x4{w[0], w[1], w[2], w[3]};
    else *reinterpret_cast<u32x2*>(d) = u32x2{w[0], w[1]};
  } else {
    float* d = static_cast<float*>(p) + i;
#pragma unroll
    for (int q = 0; q < N; q += 4) *reinterpret_cast<f32x4*>(d + q) = f32x4{f[q], f[q + 1], f[q + 2], f[q + 3]};
  }
}

// Blocks of one row each in a grid whose first axis stays below 2^32 threads.
constexpr int kGridRows = 1 << 21;
inline dim3 row_grid(int rows) {
  return dim3(rows < kGridRows ? rows : kGridRows, (unsigned)(((long long)rows + kGridRows - 1) / kGridRows));
}
// this block's row, from kGridRows * blockIdx.y; at or past the last in the rest of a grid's last line
__device__ __forceinline__ int grid_row() {
  const uint32_t r = blockIdx.y * (uint32_t)kGridRows + blockIdx.x;
  return r < 0x7FFFFFFFu ? (int)r : 0x7FFFFFFF;
}

// Sum, in a fixed order, and maximum over the block, on every thread.
template <int NT>
__device__ __forceinline__ void block_sum_max(float& sum, uint32_t& top) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    sum += __shfl_xor(sum, off, 64);
    top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
  }
  if constexpr (NT > 64) {
    __shared__ float s_sum[NT / 64];
    __shared__ uint32_t s_top[NT / 64];
    if ((threadIdx.x & 63) == 0) {
      s_sum[threadIdx.x >> 6] = sum;
      s_top[threadIdx.x >> 6] = top;
    }
    __syncthreads();
    sum = s_sum[0];
    top = s_top[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) {
      sum += s_sum[w];
      top = max(top, s_top[w]);
    }
  }
}

// Norm of a row and / or its int8 codes.  With t = x * weight (the norm's
// factor 1 / sqrt(mean x^2 + eps) is common to the row and cancels in the
// codes), one reduction gives both the sum of squares and the row's maximum.
// NORM false: quantisation of x itself.  The maximum is taken over the magnitudes
// as words, which keeps a NaN.
template <int DT, int V, int NT, bool NORM>
__global__ __launch_bounds__(NT) void k_rows(int rows, int cols, const void* x, const float* __restrict__ weight, float eps,
                                             int out_bf16, void* out, uint8_t* __restrict__ codes,
                                             float* __restrict__ scales, const int32_t* __restrict__ rows_dev,
                                             uint32_t* __restrict__ h_flags) {
  constexpr int G = granule(DT);
  const int r = grid_row();
  if (r >= (rows_dev ? min(rows, *rows_dev) : rows)) return;  // uniform over the block
  const int granules = cols / G;
  const size_t base = (size_t)r * cols;
  float t[V > 0 ? V : 1][G];
  float sum = 0.f;
  uint32_t top = 0u;
  bool range = false;
  auto take = [&](int g, float* f) {  // t of granule g, its squares and maximum
    load_granule<DT>(x, base + (size_t)g * G, f);
    if constexpr (DT == MOE_F16) {
      if (h_flags) {
#pragma unroll
        for (int q = 0; q < G; ++q) {
          if (!(fabsf(f[q]) <= 65504.f)) range = true;
          f[q] = clamp_half(f[q]);
        }
      }
    }
    if constexpr (NORM) {
      float w[G];
      if (weight) load_stream<G>(weight, false, (size_t)g * G, w);
#pragma unroll
      for (int q = 0; q < G; ++q) {
        sum = fmaf(f[q], f[q], sum);
        if (weight) f[q] *= w[q];
      }
    }
#pragma unroll
    for (int q = 0; q < G; ++q) top = max(top, i8_magnitude(f[q]));
  };
  if constexpr (V > 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int g = threadIdx.x + j * NT;
      if (g < granules) take(g, t[j]);
    }
  } else {
    for (int g = threadIdx.x; g < granules; g += NT) take(g, t[0]);
  }
  block_sum_max<NT>(sum, top);
  const float rstd = NORM ? 1.0f / sqrtf(sum / (float)cols + eps) : 1.0f;
  const float amax = __uint_as_float(top);
  const I8Row q8 = i8_row(amax);
  auto put = [&](int g, const float* f) {
    const size_t i = base + (size_t)g * G;
    if (NORM && out) {
      float o[G];
#pragma unroll
      for (int q = 0; q < G; ++q) o[q] = f[q] * rstd;
      store_stream<G>(out, out_bf16 != 0, i, o);
    }
    if (!NORM || codes) {
      uint32_t w[G / 4];
#pragma unroll
      for (int q = 0; q < G / 4; ++q)
        w[q] = i8_pack4(i8_code(f[4 * q], q8), i8_code(f[4 * q + 1], q8), i8_code(f[4 * q + 2], q8),
                        i8_code(f[4 * q + 3], q8));
      if constexpr (G == 8) *reinterpret_cast<u32x2*>(codes + i) = u32x2{w[0], w[1]};
      else *reinterpret_cast<uint32_t*>(codes + i) = w[0];
    }
  };
  if constexpr (V > 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int g = threadIdx.x + j * NT;
      if (g < granules) put(g, t[j]);
    }
  } else {
    for (int g = threadIdx.x; g < granules; g += NT) {
      take(g, t[0]);  // (adds to sum and top again: not used from here on)
      put(g, t[0]);
    }
  }
  if (DT == MOE_F16 && range) atomicOr(h_flags, (uint32_t)MOE_FLAG_H_RANGE);
  if (scales && threadIdx.x == 0) scales[r] = NORM ? amax * rstd / 127.0f : amax / 127.0f;
}

template <int DT, bool NORM>
hipError_t launch_rows(int rows, int cols, const void* x, const float* weight, float eps, int out_dtype, void* out,
                       void* codes, float* scales, const int32_t* rows_dev, uint32_t* h_flags, hipStream_t st) {
  if (rows <= 0) return hipSuccess;
  const int granules = cols / granule(DT);
#define MOE_ROWS(V, NT)                                                                                      \
  hipLaunchKernelGGL((k_rows<DT, V, NT, NORM>), row_grid(rows), dim3(NT), 0, st, rows, cols, x, weight, eps, \
                     out_dtype == MOE_BF16 ? 1 : 0, out, static_cast<uint8_t*>(codes), scales, rows_dev, h_flags)
  // many short rows to quantise: a wavefront each, without the block's barrier
  // (65536 rows of 1024 fp16 41 against 60 us, of 2048 73 against 83; 16384 rows 11.1
  // against 14.7 and 21.5 against 21.7); fewer or longer ones, and the norm with its
  // weight: a block each (norm of 8192 rows of 2048 fp32 17.1 us either way; of 1024
  // a wavefront each would be 9.6 against 11.0)
  const bool waves = !NORM && rows >= 16384;
  if (granules <= 64) MOE_ROWS(1, 64);
  else if (waves && granules <= 128) MOE_ROWS(2, 64);
  else if (waves && granules <= 256) MOE_ROWS(4, 64);
  else if (granules <= 256) MOE_ROWS(1, 256);
  else if (granules <= 512) MOE_ROWS(2, 256);
  else if (granules <= 1024) MOE_ROWS(4, 256);
  else if (granules <= 2048) MOE_ROWS(8, 256);
  else if (granules <= 8192) MOE_ROWS(8, 1024);
  else MOE_ROWS(0, 1024);
#undef MOE_ROWS
  return hipGetLastError();
}

// ---- the end of the block -----------------------------------------------------

struct BlockEnd {
  const float* weight;  // post norm, nullable
  const void* gate;
  const void* residual;
  void* out;
  long long gate_stride;
  float eps, residual_scale;
  int gate_mode;  // 0: none, 1: one value per token, 2: aligned rows, 3: rows at any alignment
  int gate_bf16, stream_bf16;
};

__device__ __forceinline__ float gate_at(const BlockEnd& e, size_t i) {
  return e.gate_bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(e.gate)[i] << 16)
                     : static_cast<const float*>(e.gate)[i];
}

// One token per block.  Pass 1: y of a granule as k_combine forms it (slots
// ascending, then the shared expert), kept in registers, and its squares; pass
// 2: norm, gate, residual, one rounding.  KM bounds top_k, so that all rows'
// loads of a granule are in flight together.  y in `parts` partial sums
// (fp32 only) as k_combine takes them.
template <int DT, int KM, int V, int NT>
__global__ __launch_bounds__(NT) void k_combine_norm(const void* __restrict__ y, int parts, long long part_stride,
                                                     const int32_t* __restrict__ row_of_slot,
                                                     const float* __restrict__ gates,
                                                     const void* __restrict__ shared, int T, int H, int k_max,
                                                     const BlockEnd e) {
  constexpr int G = granule(DT);
  const int t = grid_row();
  if (t >= T) return;
  // the token's slots, uniform over the block (scalar registers).  A slot
  // without a row loads the row of a slot that has one (from the cache) and
  // masks it to zeros, so that no load waits behind a branch
  int row[KM], any = 0;
  uint32_t live[KM];
  float weight[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    const int r = j < k_max ? row_of_slot[(size_t)t * k_max + j] : -1;
    live[j] = r >= 0 ? 0xFFFFFFFFu : 0u;
    weight[j] = r >= 0 ? gates[(size_t)t * k_max + j] : 0.f;
    row[j] = r;
    if (r >= 0) any = r;
  }
#pragma unroll
  for (int j = 0; j < KM; ++j) row[j] = live[j] ? row[j] : any;
  const int granules = H / G;
  float acc[V > 0 ? V : 1][G];
  float sum = 0.f;
  const void* last = shared ? shared : y;
  const size_t last_row = shared ? (size_t)t : (size_t)any;
  const uint32_t last_live = shared ? 0xFFFFFFFFu : 0u;
  auto take = [&](int g, float* a) {
    u32x4 raw[KM + 1];
#pragma unroll
    for (int j = 0; j < KM; ++j) raw[j] = load_raw<DT>(y, (size_t)row[j] * H + (size_t)g * G);
    raw[KM] = load_raw<DT>(last, last_row * H + (size_t)g * G);
#pragma unroll
    for (int q = 0; q < G; ++q) a[q] = 0.f;
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      float v[G];
      widen<DT>(raw[j] & live[j], v);
      if constexpr (DT == MOE_F32) {
        if (live[j]) {
          for (int p = 1; p < parts; ++p) {
            float w[G];
            load_granule<DT>(static_cast<const float*>(y) + p * part_stride, (size_t)row[j] * H + (size_t)g * G, w);
#pragma unroll
            for (int q = 0; q < G; ++q) v[q] += w[q];
          }
        }
      }
#pragma unroll
      for (int q = 0; q < G; ++q) a[q] = fmaf(weight[j], v[q], a[q]);
    }
    float v[G];
    widen<DT>(raw[KM] & last_live, v);
#pragma unroll
    for (int q = 0; q < G; ++q) a[q] += v[q];
#pragma unroll
    for (int q = 0; q < G; ++q) sum = fmaf(a[q], a[q], sum);
  };
  if constexpr (V > 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int g = threadIdx.x + j * NT;
      if (g < granules) take(g, acc[j]);
    }
  } else if (e.weight) {
    for (int g = threadIdx.x; g < granules; g += NT) take(g, acc[0]);
  }
  float rstd = 1.0f;
  if (e.weight) {
    uint32_t none = 0u;
    block_sum_max<NT>(sum, none);
    rstd = 1.0f / sqrtf(sum / (float)H + e.eps);
  }
  const float token_gate = e.gate_mode == 1 ? gate_at(e, (size_t)(t * e.gate_stride)) : 1.0f;
  auto put = [&](int g, float* a) {
    const size_t c = (size_t)g * G, i = (size_t)t * H + c;
    if (e.weight) {
      float w[G];
      load_stream<G>(e.weight, false, c, w);
#pragma unroll
      for (int q = 0; q < G; ++q) a[q] = a[q] * rstd * w[q];
    }
    if (e.gate_mode == 1) {
#pragma unroll
      for (int q = 0; q < G; ++q) a[q] *= token_gate;
    } else if (e.gate_mode == 2) {
      float w[G];
      load_stream<G>(e.gate, e.gate_bf16 != 0, (size_t)(t * e.gate_stride) + c, w);
#pragma unroll
      for (int q = 0; q < G; ++q) a[q] *= w[q];
    } else if (e.gate_mode == 3) {
#pragma unroll
      for (int q = 0; q < G; ++q) a[q] *= gate_at(e, (size_t)(t * e.gate_stride) + c + q);
    }
    if (e.residual_scale != 0.f) {
      float w[G];
      load_stream<G>(e.residual, e.stream_bf16 != 0, i, w);
#pragma unroll
      for (int q = 0; q < G; ++q) a[q] = fmaf(e.residual_scale, w[q], a[q]);
    }
    store_stream<G>(e.out, e.stream_bf16 != 0, i, a);
  };
  if constexpr (V > 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int g = threadIdx.x + j * NT;
      if (g < granules) put(g, acc[j]);
    }
  } else {
    for (int g = threadIdx.x; g < granules; g += NT) {
      take(g, acc[0]);
      put(g, acc[0]);
    }
  }
}

template <int DT, int KM>
hipError_t launch_end(const moe_shape& s, const void* y, const int32_t* row_of_slot, const float* gates,
                      const void* shared, const BlockEnd& e, hipStream_t st, int parts, long long part_stride) {
  const int granules = s.hidden / granule(DT);
#define MOE_END(V, NT)                                                                                       \
  hipLaunchKernelGGL((k_combine_norm<DT, KM, V, NT>), row_grid(s.num_tokens), dim3(NT), 0, st, y, parts,     \
                     part_stride, row_of_slot, gates, shared, s.num_tokens, s.hidden, s.top_k, e)
  if (granules <= 256) MOE_END(1, 256);
  else if (granules <= 512) MOE_END(2, 256);
  else if (granules <= 1024) MOE_END(4, 256);
  else if (granules <= 4096) MOE_END(4, 1024);
  else MOE_END(0, 1024);
#undef MOE_END
  return hipGetLastError();
}

template <int DT>
hipError_t launch_end_k(const moe_shape& s, const void* y, const int32_t* row_of_slot, const float* gates,
                        const void* shared, const BlockEnd& e, hipStream_t st, int parts, long long part_stride) {
  if (s.top_k <= 2) return launch_end<DT, 2>(s, y, row_of_slot, gates, shared, e, st, parts, part_stride);
  if (s.top_k <= 4) return launch_end<DT, 4>(s, y, row_of_slot, gates, shared, e, st, parts, part_stride);
  if (s.top_k <= 8) return launch_end<DT, 8>(s, y, row_of_slot, gates, shared, e, st, parts, part_stride);
  return launch_end<DT, kMaxTopK>(s, y, row_of_slot, gates, shared, e, st, parts, part_stride);
}

}  // namespace

hipError_t launch_norm(int rows, int cols, int src_dtype, const void* x, const float* weight, float eps,
                       int out_dtype, void* out, void* codes, float* scales, hipStream_t st) {
  if (src_dtype == MOE_BF16)
    return launch_rows<MOE_BF16, true>(rows, cols, x, weight, eps, out_dtype, out, codes, scales, nullptr, nullptr, st);
  return launch_rows<MOE_F32, true>(rows, cols, x, weight, eps, out_dtype, out, codes, scales, nullptr, nullptr, st);
}

hipError_t launch_quant_int8(int src_dtype, const void* src, int rows, int cols, const int32_t* rows_dev, void* codes,
                             float* scales, hipStream_t st, uint32_t* h_flags) {
  if (src_dtype == MOE_BF16)
    return launch_rows<MOE_BF16, false>(rows, cols, src, nullptr, 0.f, 0, nullptr, codes, scales, rows_dev, nullptr,
                                        st);
  if (src_dtype == MOE_F16)
    return launch_rows<MOE_F16, false>(rows, cols, src, nullptr, 0.f, 0, nullptr, codes, scales, rows_dev, h_flags,
                                       st);
  return launch_rows<MOE_F32, false>(rows, cols, src, nullptr, 0.f, 0, nullptr, codes, scales, rows_dev, nullptr, st);
}

hipError_t launch_combine_norm(const moe_shape& s, const moe_block& b, int y_dtype, const void* y,
                               const int32_t* row_of_slot, const float* gates, const void* y_shared,
                               const void* residual, void* out, hipStream_t st, int parts, long long part_stride) {
  if (parts > 1 && y_dtype != MOE_F32) return hipErrorInvalidValue;
  BlockEnd e{};
  e.weight = b.post_norm;
  e.gate = b.gate;
  e.residual = residual;
  e.out = out;
  e.gate_stride = b.gate_row_stride;
  e.eps = b.eps;
  e.residual_scale = b.residual_scale;
  e.gate_bf16 = b.gate_dtype == MOE_BF16;
  e.stream_bf16 = b.stream_dtype == MOE_BF16;
  if (b.gate) {
    const int gb = e.gate_bf16 ? 2 : 4;
    const bool aligned = (reinterpret_cast<uintptr_t>(b.gate) & 15u) == 0 && (b.gate_row_stride * gb) % 16 == 0;
    e.gate_mode = b.gate_col_stride == 0 ? 1 : (aligned ? 2 : 3);
  }
  if (y_dtype == MOE_F32)
    return launch_end_k<MOE_F32>(s, y, row_of_slot, gates, y_shared, e, st, parts, part_stride);
  if (y_dtype == MOE_F16)
    return launch_end_k<MOE_F16>(s, y, row_of_slot, gates, y_shared, e, st, 1, 0);
  return launch_end_k<MOE_BF16>(s, y, row_of_slot, gates, y_shared, e, st, 1, 0);
}

}  // namespace moe
