// Routing with a balance bias: scores plus a per-expert bias choose groups and
// experts, the scores alone give the gates.
//
// The choice is discrete, so it has to be that of the fp64 keys: fp32 sigmoids
// saturate (17 and 18 become the same score) and their last bit differs from
// one implementation to the next, while two fp64 keys that differ at all
// differ by far more than fp64 rounding for any logits and biases given in
// fp32.  fp64 exponentials and compares of every expert would bound the kernel
// (8192 tokens of 256 experts: 26 us against 9 now), so a token is first routed
// on fp32 keys with a bound on their error; where any decision -- the next expert
// of a slot, the last group kept -- falls within the bound, which random logits
// do for a few tokens in ten thousand, the wavefront routes that token again in
// fp64.  Gates are fp64 either way, of the chosen experts only.
//
// One 64-lane wavefront per token; lane l holds EPL consecutive experts (l * EPL
// ..), so lower lanes hold lower experts and ties go to the lower lane.
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kWavesPerBlock = 4;
constexpr int kMaxGroupTopn = 8;

__device__ __forceinline__ double neg_inf() { return -__builtin_inf(); }

// An order-preserving map of a key, rounded to fp32, to the integers above 0;
// 0 stands for no key.
__device__ __forceinline__ uint32_t rank_word(double key, bool valid) {
  const uint32_t b = __float_as_uint((float)key);
  const uint32_t u = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return valid ? u : 0u;
}

// Largest word over the wavefront, in a scalar: row shifts, then broadcasts of
// the rows' last lanes (lane 63 ends with the maximum of all).
template <int CTRL>
__device__ __forceinline__ uint32_t max_step(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
  return v > o ? v : o;
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max_step<0x111>(v);
  v = max_step<0x112>(v);
  v = max_step<0x114>(v);
  v = max_step<0x118>(v);
  v = max_step<0x142>(v);
  v = max_step<0x143>(v);
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ double read_lane(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Lane with the largest key among the lanes whose `valid` holds, lower lanes
// first among equals; -1 if none.  fp32 rounding is monotone, so the largest
// key is among the lanes with the largest rounded key, nearly always one.
__device__ __forceinline__ int wave_best(double key, bool valid) {
  const uint32_t u = rank_word(key, valid);
  const uint32_t top = wave_max_u32(u);
  if (top == 0u) return -1;
  uint64_t mask = __ballot(u == top);
  int best = __builtin_ctzll(mask);
  mask &= mask - 1;
  while (mask) {  // keys that round to the same fp32 value
    const int other = __builtin_ctzll(mask);
    mask &= mask - 1;
    if (read_lane(key, other) > read_lane(key, best)) best = other;
  }
  return best;
}

// A token's inputs in a wavefront, and where its outputs go.
template <int EPL>
struct Token {
  float v[EPL], bias[EPL];  // logits (finite), selection bias
  bool avail[EPL];
  int32_t* ids;
  float* gates;
};

struct RouteArgs {
  int E, k_max, score, renorm, G, topk_groups, topn;
  float scale;
};

// Lists of the n largest rank words, largest first.
template <int N>
__device__ __forceinline__ void list_insert(uint32_t (&top)[N], uint32_t x) {
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const uint32_t hi = max(top[q], x);
    x = min(top[q], x);
    top[q] = hi;
  }
}

__device__ __forceinline__ float rank_value(uint32_t w) {
  return __uint_as_float((w & 0x80000000u) ? w ^ 0x80000000u : ~w);
}
__device__ __forceinline__ uint32_t rank_word32(float f) {
  const uint32_t b = __float_as_uint(f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// Groups of the token kept on fp32 keys: false where the last one kept and the
// best one left are closer than `tol`.
template <int EPL, int N>
__device__ __forceinline__ bool keep_groups(uint32_t (&w)[EPL], const RouteArgs& a, uint32_t* lds, int lane,
                                            float tol) {
  const int gs = a.E / a.G;
  uint32_t top[N];
#pragma unroll
  for (int q = 0; q < N; ++q) top[q] = 0u;
  int lpg = gs / EPL;  // lanes of a group
  if (gs % EPL == 0 && (lpg & (lpg - 1)) == 0) {
    // groups on whole, aligned runs of lanes: a lane's own experts
#pragma unroll
    for (int i = 0; i < EPL; ++i) list_insert(top, w[i]);
  } else {
    // other group shapes: through LDS, the largest power of two of lanes per group
    lpg = 64 >> (32 - __builtin_clz(a.G - 1));
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane * EPL + i < a.E) lds[lane * EPL + i] = w[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the lanes read each other's words
    __builtin_amdgcn_wave_barrier();
    const int g = lane / lpg;
    if (g < a.G)
      for (int i = lane % lpg; i < gs; i += lpg) list_insert(top, lds[g * gs + i]);
  }
  for (int m = 1; m < lpg; m <<= 1) {
    uint32_t other[N];
#pragma unroll
    for (int q = 0; q < N; ++q) other[q] = (uint32_t)__shfl_xor((int)top[q], m, 64);
#pragma unroll
    for (int q = 0; q < N; ++q) list_insert(top, other[q]);
  }
  float total = rank_value(top[0]), size = fabsf(total);
#pragma unroll
  for (int q = 1; q < N; ++q) {
    if (q < a.topn && top[q] != 0u) {
      total += rank_value(top[q]);
      size += fabsf(rank_value(top[q]));  // keys of opposite sign: the sum's rounding follows their size
    }
  }
  const int from = (lane < a.G ? lane : 0) * lpg;
  uint32_t gw = (uint32_t)__shfl((int)(top[0] != 0u ? rank_word32(total) : 0u), from, 64);
  if (lane >= a.G) gw = 0u;
  uint64_t kept = 0;
  uint32_t last = 0u;
  for (int n = 0; n < a.topk_groups;) {
    const uint32_t best = wave_max_u32(gw);
    if (best == 0u) break;
    last = best;
    const uint64_t mask = __ballot(gw == best);
    kept |= mask;
    n += __builtin_popcountll(mask);
    if (n > a.topk_groups) return false;
    if (gw == best) gw = 0u;
  }
  const uint32_t left = wave_max_u32(gw);
  if (last != 0u && left != 0u) {
    const float most = rank_value(wave_max_u32(top[0] != 0u ? rank_word32(size) : 0u));
    if (!(rank_value(left) < rank_value(last) - a.topn * (tol + 2.4e-7f * most))) return false;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    if (e < a.E && !((kept >> (e / gs)) & 1ull)) w[i] = 0u;
  }
  return true;
}

// The token on fp32 keys; false (nothing written) where a decision is closer
// than the keys' error.  That error: a sigmoid's exponential is off by its
// argument's rounding, at most |x| 2^-24 log2 e relative, which the slope, s (1 - s)
// |x| <= 0.23, brings to 2e-8 absolute, and its own and the reciprocal's steps
// add 1.2e-7; a softmax's is off by as much of the largest score, and by the 20
// roundings of the sum (1.2e-6 of it).  `tol` is more than twice that.  The sum
// with the bias adds 6e-8 of the key, and so does the difference that the bound
// is compared through.
template <int EPL>
__device__ __forceinline__ bool route_fp32(const Token<EPL>& t, const RouteArgs& a, int kt, uint32_t* lds, int lane,
                                           const float* lt, int parts, long long part_stride) {
  float s[EPL], m = 0.f, tol = 1.0e-6f;
  if (a.score == MOE_SCORE_SOFTMAX) {
    uint32_t mw = 0u;
#pragma unroll
    for (int i = 0; i < EPL; ++i) mw = max(mw, t.avail[i] ? rank_word32(t.v[i]) : 0u);
    mw = wave_max_u32(mw);
    m = mw ? rank_value(mw) : 0.f;
    float d = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      s[i] = t.avail[i] ? __expf(t.v[i] - m) : 0.f;
      d += s[i];
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) d += __shfl_xor(d, off, 64);
    const float r = d > 0.f ? 1.0f / d : 0.f;
    tol = 3.0e-6f * r;  // the largest score is 1 / d
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] *= r;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-t.v[i]));
  }
  uint32_t w[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) w[i] = t.avail[i] ? rank_word32(s[i] + t.bias[i]) : 0u;
  if (a.G > 1) {
    const bool sure = a.topn == 1 ? keep_groups<EPL, 1>(w, a, lds, lane, tol)
                                  : (a.topn == 2 ? keep_groups<EPL, 2>(w, a, lds, lane, tol)
                                                 : keep_groups<EPL, kMaxGroupTopn>(w, a, lds, lane, tol));
    if (!sure) return false;
  }
  int my_id = -1;
  for (int j = 0; j < kt; ++j) {
    uint32_t best = w[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) best = max(best, w[i]);
    best = wave_max_u32(best);
    if (best == 0u) break;
    const float f = rank_value(best);
    const uint32_t near = rank_word32(f - (tol + 2.4e-7f * fabsf(f)));
    int n = 0, id = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const uint64_t mask = __ballot(w[i] >= near);
      n += __builtin_popcountll(mask);
      if (mask) id = __builtin_ctzll(mask) * EPL + i;
      if (w[i] >= near) w[i] = 0u;
    }
    if (n != 1) return false;  // (for an infinite key, `near` is above every word: 0)
    if (lane == j) my_id = id;
  }
  // gates, fp64: lane j of slot j
  double g = 0.0, d = 0.0;
  if (my_id >= 0) {
    float x = lt[my_id];
    for (int p = 1; p < parts; ++p) x += lt[p * part_stride + my_id];
    x = fminf(fmaxf(x, -3.402823466e38f), 3.402823466e38f);
    g = a.score == MOE_SCORE_SOFTMAX ? exp((double)x - (double)m) : 1.0 / (1.0 + exp(-(double)x));
  }
  if (a.renorm) {
    d = g;
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) d += __shfl_xor(d, off, 64);  // the slots' lanes: the first 16
    g = d > 0.0 ? g / d : 0.0;
  } else if (a.score == MOE_SCORE_SOFTMAX) {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (t.avail[i]) d += exp((double)t.v[i] - (double)m);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) d += __shfl_xor(d, off, 64);
    g /= d;
  }
  if (lane < a.k_max) {
    t.ids[lane] = my_id;
    t.gates[lane] = my_id >= 0 ? (float)(g * (double)a.scale) : 0.0f;
  }
  return true;
}

// The token on fp64 keys.
template <int EPL>
__device__ __forceinline__ void route_fp64(Token<EPL>& t, const RouteArgs& a, int kt, double* lds, int lane) {
  auto& v = t.v;
  auto& avail = t.avail;
  const int E = a.E;
  // scores and keys
  double s[EPL], key[EPL];
  if (a.score == MOE_SCORE_SOFTMAX) {
    float m = -3.402823466e38f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (avail[i]) m = fmaxf(m, v[i]);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      s[i] = avail[i] ? exp((double)v[i] - (double)m) : 0.0;
      d += s[i];
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) d += __shfl_xor(d, off, 64);
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] /= d;  // d >= 1, or no expert is available
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] = 1.0 / (1.0 + exp(-(double)v[i]));
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) key[i] = avail[i] ? s[i] + (double)t.bias[i] : neg_inf();

  // group limit: the lanes of a group share its experts, each keeps the topn
  // largest keys of its own, and a butterfly over them merges the lists
  if (a.G > 1) {
    const int G = a.G, topn = a.topn;
    const int gs = E / G;
    double top[kMaxGroupTopn];
#pragma unroll
    for (int q = 0; q < kMaxGroupTopn; ++q) top[q] = neg_inf();
    auto insert = [&](double x) {
#pragma unroll
      for (int q = 0; q < kMaxGroupTopn; ++q) {
        if (q < topn && x > top[q]) {
          const double y = top[q];
          top[q] = x;
          x = y;
        }
      }
    };
    int lpg = gs / EPL;  // lanes of a group
    if (gs % EPL == 0 && (lpg & (lpg - 1)) == 0) {
      // groups on whole, aligned runs of lanes: a lane's own experts
#pragma unroll
      for (int i = 0; i < EPL; ++i) insert(key[i]);
    } else {
      // other group shapes: through LDS, the largest power of two of lanes per group
      lpg = 64 >> (32 - __builtin_clz(G - 1));
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (lane * EPL + i < E) lds[lane * EPL + i] = key[i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the lanes read each other's keys
      __builtin_amdgcn_wave_barrier();
      const int g = lane / lpg;
      if (g < G)
        for (int i = lane % lpg; i < gs; i += lpg) insert(lds[g * gs + i]);
    }
    for (int m = 1; m < lpg; m <<= 1) {
      double other[kMaxGroupTopn];
#pragma unroll
      for (int q = 0; q < kMaxGroupTopn; ++q)
        if (q < topn) other[q] = __shfl_xor(top[q], m, 64);
#pragma unroll
      for (int q = 0; q < kMaxGroupTopn; ++q)
        if (q < topn) insert(other[q]);
    }
    const bool any = top[0] > neg_inf();
    double total = top[0];
#pragma unroll
    for (int q = 1; q < kMaxGroupTopn; ++q)
      if (q < topn && top[q] > neg_inf()) total += top[q];
    // lane g takes group g's score; the best groups
    total = __shfl(total, (lane < G ? lane : 0) * lpg, 64);
    bool open = __shfl((int)any, (lane < G ? lane : 0) * lpg, 64) && lane < G;
    uint64_t kept = 0;
    for (int q = 0; q < a.topk_groups; ++q) {
      const int b = wave_best(total, open);
      if (b < 0) break;
      kept |= 1ull << b;
      if (lane == b) open = false;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane * EPL + i;
      avail[i] = avail[i] && e < E && ((kept >> (e / gs)) & 1ull);
    }
  }

  // k_t rounds: every lane offers its best expert, the wavefront takes the best
  double my_s = 0.0, sum = 0.0;
  int my_id = -1;
  for (int j = 0; j < kt; ++j) {
    double bk = 0.0, bs = 0.0;
    int bi = -1;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if (avail[i] && (bi < 0 || key[i] > bk)) {
        bk = key[i];
        bs = s[i];
        bi = lane * EPL + i;
      }
    }
    const int win = wave_best(bk, bi >= 0);
    if (win < 0) break;
    const int id = __builtin_amdgcn_readlane(bi, win);
    const double sc = read_lane(bs, win);
    sum += sc;
    if (lane == j) {
      my_id = id;
      my_s = sc;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane * EPL + i == id) avail[i] = false;
  }
  double g = my_s;
  if (a.renorm) g = sum > 0.0 ? my_s / sum : 0.0;
  if (lane < a.k_max) {
    t.ids[lane] = my_id;
    t.gates[lane] = my_id >= 0 ? (float)(g * (double)a.scale) : 0.0f;
  }
}

// flag_word (nullable): with it, this launch alone sets the call's flag word --
// block 0 looks through every k_t -- and no launch has to clear it before.
template <int EPL>
__global__ __launch_bounds__(256) void k_route_biased(const float* __restrict__ logits,
                                                      const float* __restrict__ select_bias, int T,
                                                      const int32_t* __restrict__ kpt, const RouteArgs a,
                                                      int32_t* __restrict__ ids, float* __restrict__ gates,
                                                      uint32_t* __restrict__ flags, int own_flags, int vec, int parts,
                                                      long long part_stride, float* __restrict__ sum_out) {
  __shared__ double s_key[kWavesPerBlock][EPL * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * kWavesPerBlock + wave;
  if (own_flags && blockIdx.x == 0) {
    __shared__ int s_bad;
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    if (kpt) {
      bool bad = false;
      for (int i = threadIdx.x; i < T; i += 256) bad |= kpt[i] < 1 || kpt[i] > a.k_max;
      if (bad) s_bad = 1;
    }
    __syncthreads();
    if (threadIdx.x == 0) *flags = s_bad ? (uint32_t)MOE_FLAG_BAD_K : 0u;
  }
  if (t >= T) return;  // uniform over the wavefront; nothing below synchronises the block

  // logits (parts in order, as k_route_topk adds them) and availability
  Token<EPL> tk;
  tk.ids = ids + (size_t)t * a.k_max;
  tk.gates = gates + (size_t)t * a.k_max;
  const int E = a.E;
  const float* lt = logits + (size_t)t * E;
  const int kt = kpt ? __builtin_amdgcn_readfirstlane(kpt[t]) : a.k_max;
  if (vec) {  // a lane's experts are all real or none, and 16-byte aligned
    typedef float vf __attribute__((ext_vector_type(EPL >= 4 ? 4 : EPL)));
    const int e0 = lane * EPL < E ? lane * EPL : 0;
#pragma unroll
    for (int i = 0; i < EPL; i += (EPL >= 4 ? 4 : EPL)) {
      const vf x = *reinterpret_cast<const vf*>(lt + e0 + i), y = *reinterpret_cast<const vf*>(select_bias + e0 + i);
      if constexpr (EPL == 1) {
        tk.v[i] = x[0], tk.bias[i] = y[0];
      } else {
#pragma unroll
        for (int q = 0; q < (EPL >= 4 ? 4 : EPL); ++q) tk.v[i + q] = x[q], tk.bias[i + q] = y[q];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = min(lane * EPL + i, E - 1);
      tk.v[i] = lt[e];
      tk.bias[i] = select_bias[e];
    }
  }
  for (int p = 1; p < parts; ++p) {
    float w[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) w[i] = lt[p * part_stride + min(lane * EPL + i, E - 1)];
#pragma unroll
    for (int i = 0; i < EPL; ++i) tk.v[i] += w[i];
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const bool real = lane * EPL + i < E;
    if (parts > 1 && sum_out && real) sum_out[(size_t)t * E + lane * EPL + i] = tk.v[i];
    tk.avail[i] = real && tk.bias[i] > -__builtin_inff() && tk.v[i] == tk.v[i];  // (a NaN bias compares false)
    tk.v[i] = fminf(fmaxf(tk.v[i], -3.402823466e38f), 3.402823466e38f);
  }
  if (kt < 1 || kt > a.k_max) {
    if (lane < a.k_max) {
      tk.ids[lane] = -1;
      tk.gates[lane] = 0.0f;
    }
    if (!own_flags && lane == 0) atomicOr(flags, (uint32_t)MOE_FLAG_BAD_K);
    return;
  }
  if (!route_fp32<EPL>(tk, a, kt, reinterpret_cast<uint32_t*>(s_key[wave]), lane, lt, parts, part_stride))
    route_fp64<EPL>(tk, a, kt, s_key[wave], lane);
}

}  // namespace

hipError_t launch_route_biased(const moe_shape& s, const float* logits, const float* select_bias,
                               const int32_t* k_per_token, int32_t* ids, float* gates, uint32_t* flags,
                               bool own_flags, hipStream_t st, int parts, long long part_stride, float* sum_out) {
  const int T = s.num_tokens, E = s.num_experts;
  const int grid = (T + kWavesPerBlock - 1) / kWavesPerBlock;
  const RouteArgs a{E,           s.top_k,       s.score,
                    s.renormalize, s.num_groups > 1 ? s.num_groups : 1,
                    s.topk_groups, s.group_topn > 0 ? s.group_topn : 1, s.routed_scale};
  const auto aligned = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
#define MOE_ROUTE_LAUNCH(EPL)                                                                              \
  hipLaunchKernelGGL(k_route_biased<EPL>, dim3(grid), dim3(256), 0, st, logits, select_bias, T,            \
                     k_per_token, a, ids, gates, flags, own_flags ? 1 : 0,                                 \
                     E % (EPL < 4 ? 4 : EPL) == 0 && aligned(logits) && aligned(select_bias), parts,       \
                     part_stride, sum_out)
  if (E <= 64) MOE_ROUTE_LAUNCH(1);
  else if (E <= 128) MOE_ROUTE_LAUNCH(2);
  else if (E <= 256) MOE_ROUTE_LAUNCH(4);
  else MOE_ROUTE_LAUNCH(8);
#undef MOE_ROUTE_LAUNCH
  return hipGetLastError();
}

}  // namespace moe
