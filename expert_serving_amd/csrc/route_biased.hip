// Routing with a balance bias: scores plus a per-expert bias choose groups and
// experts, the scores alone give the gates.
//
// The choice is discrete, so its keys are held in fp64: fp32 sigmoids saturate
// (17 and 18 become the same score) and their last bit differs from one
// implementation to the next, while two fp64 keys that differ at all differ by
// far more than fp64 rounding for any logits and biases given in fp32.
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

template <int EPL>
__global__ __launch_bounds__(256) void k_route_biased(const float* __restrict__ logits,
                                                      const float* __restrict__ select_bias, int T, int E, int k_max,
                                                      const int32_t* __restrict__ kpt, int score, int renorm,
                                                      float scale, int G, int topk_groups, int topn,
                                                      int32_t* __restrict__ ids, float* __restrict__ gates,
                                                      uint32_t* __restrict__ flags, int parts, long long part_stride,
                                                      float* __restrict__ sum_out) {
  __shared__ double s_key[kWavesPerBlock][kMaxExperts];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * kWavesPerBlock + wave;
  if (t >= T) return;  // uniform over the wavefront; nothing below synchronises the block

  // logits (parts in order, as k_route_topk adds them) and availability
  float v[EPL], bias[EPL];
  bool avail[EPL];
  int ec[EPL];
  const float* lt = logits + (size_t)t * E;
  const int kt = kpt ? kpt[t] : k_max;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    ec[i] = e < E ? e : E - 1;
    v[i] = lt[ec[i]];
    bias[i] = select_bias[ec[i]];
  }
  for (int p = 1; p < parts; ++p) {
    float w[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) w[i] = lt[p * part_stride + ec[i]];
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] += w[i];
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const bool real = lane * EPL + i < E;
    if (parts > 1 && sum_out && real) sum_out[(size_t)t * E + ec[i]] = v[i];
    avail[i] = real && bias[i] > -__builtin_inff() && v[i] == v[i];  // (a NaN bias compares false)
    v[i] = fminf(fmaxf(v[i], -3.402823466e38f), 3.402823466e38f);
  }
  if (kt < 1 || kt > k_max) {
    if (lane < k_max) {
      ids[(size_t)t * k_max + lane] = -1;
      gates[(size_t)t * k_max + lane] = 0.0f;
    }
    if (lane == 0) atomicOr(flags, (uint32_t)MOE_FLAG_BAD_K);
    return;
  }

  // scores and keys
  double s[EPL], key[EPL];
  if (score == MOE_SCORE_SOFTMAX) {
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
  for (int i = 0; i < EPL; ++i) key[i] = avail[i] ? s[i] + (double)bias[i] : neg_inf();

  // group limit: the lanes of a group share its experts, each keeps the topn
  // largest keys of its own, and a butterfly over them merges the lists
  if (G > 1) {
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
      lpg = 64 >> (G > 1 ? 32 - __builtin_clz(G - 1) : 0);
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (lane * EPL + i < E) s_key[wave][lane * EPL + i] = key[i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the lanes read each other's keys
      __builtin_amdgcn_wave_barrier();
      const int g = lane / lpg;
      if (g < G)
        for (int i = lane % lpg; i < gs; i += lpg) insert(s_key[wave][g * gs + i]);
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
    for (int q = 0; q < topk_groups; ++q) {
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
  if (renorm) g = sum > 0.0 ? my_s / sum : 0.0;
  if (lane < k_max) {
    ids[(size_t)t * k_max + lane] = my_id;
    gates[(size_t)t * k_max + lane] = my_id >= 0 ? (float)(g * (double)scale) : 0.0f;
  }
}

}  // namespace

hipError_t launch_route_biased(const moe_shape& s, const float* logits, const float* select_bias,
                               const int32_t* k_per_token, int32_t* ids, float* gates, uint32_t* flags,
                               hipStream_t st, int parts, long long part_stride, float* sum_out) {
  const int T = s.num_tokens, E = s.num_experts;
  const int grid = (T + kWavesPerBlock - 1) / kWavesPerBlock;
  const int G = s.num_groups > 1 ? s.num_groups : 1;
  const int topn = s.group_topn > 0 ? s.group_topn : 1;
#define MOE_ROUTE_LAUNCH(EPL)                                                                             \
  hipLaunchKernelGGL(k_route_biased<EPL>, dim3(grid), dim3(256), 0, st, logits, select_bias, T, E,        \
                     s.top_k, k_per_token, s.score, s.renormalize, s.routed_scale, G, s.topk_groups,      \
                     topn, ids, gates, flags, parts, part_stride, sum_out)
  if (E <= 64) MOE_ROUTE_LAUNCH(1);
  else if (E <= 128) MOE_ROUTE_LAUNCH(2);
  else if (E <= 256) MOE_ROUTE_LAUNCH(4);
  else MOE_ROUTE_LAUNCH(8);
#undef MOE_ROUTE_LAUNCH
  return hipGetLastError();
}

}  // namespace moe
