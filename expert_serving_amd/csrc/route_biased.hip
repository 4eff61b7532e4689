// Routing with a balance bias: scores plus a per-expert bias choose groups and
// experts, the scores alone give the gates.
//
// The choice is discrete, so it has to be that of the fp64 keys: fp32 sigmoids
// saturate (17 and 18 become the same score) and their last bit differs from
// one implementation to the next, while the fp64 keys of different fp32 logits
// in the range that routers give differ by far more than fp64 rounding.  fp64 has
// limits of its own -- sigmoids of logits above 36.8 are all 1, and a bias of
// magnitude m leaves the scores beside it a resolution of m * 1e-16 -- and keys
// that are equal there go to the lower expert.  fp64 exponentials and compares of every expert would bound the kernel
// (8192 tokens of 256 experts: 26 us), so a token is first routed
// on fp32 keys with a bound on their error; where any decision -- the next expert
// of a slot, the last group kept -- falls within the bound, which random logits
// do for a few tokens in ten thousand, the wavefront routes that token again in
// fp64.  Gates are fp64 either way, of the chosen experts only.
//
// fp32 keys: a row of 16 lanes per token (the 16 lanes data-parallel primitives
// exchange among), so that the instructions of a round serve four tokens; for
// batches that leave compute units idle anyway a whole wavefront per token,
// whose rounds are shorter (256 experts in 8 groups, one token: 5.0 against 6.2
// us; 2048 tokens: 7.8 against 7.0).  fp64 keys: a wavefront per token.  Each
// gives a lane consecutive experts.  What bounds it: the issue of the vector
// units, about 300 instructions per token, and below some thousand tokens the
// launch and the chain of rounds; 8192 tokens of 256 experts 8.7 us, 16381 of
// 128 with a budget each 9.0 us, where their logits alone take 2 us.
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

struct RouteArgs {
  const float* logits;
  const float* select_bias;
  int T, E, k_max, score, renorm, G, topk_groups, topn;
  float scale;
  int parts;
  long long part_stride;
  int32_t* ids;
  float* gates;
  // a group: its experts, and the power of two of a token's lanes that score
  // it; whole: the group's experts are those lanes' own (else they go through
  // LDS); rows: the fp32 keys can take this grouping (at most 16 groups)
  int gs, lpg, whole, rows;
  float inv_gs;
  int vec;  // four consecutive experts are all real or none, and 16-byte aligned
};

constexpr float kMaxFinite = 3.402823466e38f;
__device__ __forceinline__ float finite(float x) { return fminf(fmaxf(x, -kMaxFinite), kMaxFinite); }

// Group of expert e < 512 (the quotient's distance from a whole number is at
// least 1 / (2 * 512), far more than its rounding).
__device__ __forceinline__ int group_of(int e, const RouteArgs& a) { return (int)(((float)e + 0.5f) * a.inv_gs); }

// N consecutive experts' logits (parts in order, as k_route_topk adds them) and
// biases, from expert e0 on; places past the last expert repeat it.
template <int N>
__device__ __forceinline__ void load_experts(const RouteArgs& a, int t, int e0, float (&v)[N], float (&bias)[N]) {
  const float* lt = a.logits + (size_t)t * a.E;
  if (N % 4 == 0 && a.vec) {
    typedef float f32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int i = 0; i + 3 < N; i += 4) {
      const int e = e0 + i < a.E ? e0 + i : 0;
      const f32x4 x = *reinterpret_cast<const f32x4*>(lt + e), y = *reinterpret_cast<const f32x4*>(a.select_bias + e);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[i + q] = x[q], bias[i + q] = y[q];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = min(e0 + i, a.E - 1);
      v[i] = lt[e];
      bias[i] = a.select_bias[e];
    }
  }
  for (int p = 1; p < a.parts; ++p) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += lt[p * a.part_stride + min(e0 + i, a.E - 1)];
  }
}

// ---- rows of 16 lanes -----------------------------------------------------------

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) { return __uint_as_float(dpp<CTRL>(__float_as_uint(v))); }
template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, ((uint64_t)dpp<CTRL>((uint32_t)(b >> 32)) << 32) | dpp<CTRL>((uint32_t)b));
}
// over the row, on each of its lanes (rotations by 8, 4, 2, 1)
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, dpp<0x128>(v));
  v = max(v, dpp<0x124>(v));
  v = max(v, dpp<0x122>(v));
  return max(v, dpp<0x121>(v));
}
__device__ __forceinline__ uint32_t row_sum(uint32_t v) {
  v += dpp<0x128>(v);
  v += dpp<0x124>(v);
  v += dpp<0x122>(v);
  return v + dpp<0x121>(v);
}
__device__ __forceinline__ float row_sum(float v) {
  v += dpp_f<0x128>(v);
  v += dpp_f<0x124>(v);
  v += dpp_f<0x122>(v);
  return v + dpp_f<0x121>(v);
}
__device__ __forceinline__ double row_sum(double v) {
  v += dpp_d<0x128>(v);
  v += dpp_d<0x124>(v);
  v += dpp_d<0x122>(v);
  return v + dpp_d<0x121>(v);
}

// Over the 16 or 64 lanes of a token, on each of them.
template <int TEAM>
__device__ __forceinline__ uint32_t team_max(uint32_t v) {
  v = row_max(v);
  if constexpr (TEAM == 64) {
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(a[0], a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max(b[0], b[1]);
  }
  return v;
}
template <int TEAM, typename T>
__device__ __forceinline__ T team_sum(T v) {
  v = row_sum(v);
  if constexpr (TEAM == 64) {
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
  }
  return v;
}

__device__ __forceinline__ float rank_value(uint32_t w) {
  return __uint_as_float((w & 0x80000000u) ? w ^ 0x80000000u : ~w);
}
__device__ __forceinline__ uint32_t rank_word32(float f) {
  const uint32_t b = __float_as_uint(f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

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

// Zeroes the words outside the groups kept on fp32 keys; false (on all lanes of
// the token) where a kept group and one left out are closer than the keys' error.
template <int EPL, int TEAM, int N>
__device__ __forceinline__ bool keep_groups(uint32_t (&w)[EPL], const RouteArgs& a, uint32_t* lds, int rl, float tol) {
  uint32_t top[N];
#pragma unroll
  for (int q = 0; q < N; ++q) top[q] = 0u;
  if (a.whole) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) list_insert(top, w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) lds[rl * EPL + i] = w[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the lanes read each other's words
    __builtin_amdgcn_wave_barrier();
    const int g = rl / a.lpg;
    if (g < a.G)
      for (int i = rl % a.lpg; i < a.gs; i += a.lpg) list_insert(top, lds[g * a.gs + i]);
  }
  // merge over the group's lanes: after each step 2, 4, .. lanes hold one list,
  // so a mirrored order is as good an exchange as a butterfly's
  auto merge = [&](auto&& other_of) {
    uint32_t other[N];
#pragma unroll
    for (int q = 0; q < N; ++q) other[q] = other_of(top[q]);
    if constexpr (N == 2) {
      const uint32_t lo = min(top[0], other[0]);
      top[0] = max(top[0], other[0]);
      top[1] = max(lo, max(top[1], other[1]));
    } else {
#pragma unroll
      for (int q = 0; q < N; ++q) list_insert(top, other[q]);
    }
  };
  if (a.lpg > 1) merge([](uint32_t v) { return dpp<0xB1>(v); });   // quads: lane ^ 1
  if (a.lpg > 2) merge([](uint32_t v) { return dpp<0x4E>(v); });   // quads: lane ^ 2
  if (a.lpg > 4) merge([](uint32_t v) { return dpp<0x141>(v); });  // eights mirrored
  if (a.lpg > 8) merge([](uint32_t v) { return dpp<0x140>(v); });  // sixteens mirrored
  if constexpr (TEAM == 64) {
    // (two groups: at most 32 lanes each)
    if (a.lpg > 16) merge([](uint32_t v) { return (uint32_t)__shfl_xor((int)v, 16, 64); });
  }
  float total = rank_value(top[0]), size = fabsf(total);
#pragma unroll
  for (int q = 1; q < N; ++q) {
    if (q < a.topn && top[q] != 0u) {
      total += rank_value(top[q]);
      size += fabsf(rank_value(top[q]));  // keys of opposite sign: the sum's rounding follows their size
    }
  }
  const float most = rank_value(team_max<TEAM>(top[0] != 0u ? rank_word32(size) : 0u));
  // lane g of each row takes group g's word (0: a group without an expert)
  const int lane = threadIdx.x & 63, g16 = lane & 15;
  uint32_t word = top[0] != 0u ? rank_word32(total) : 0u;
  word = (uint32_t)__shfl((int)word, (TEAM == 64 ? 0 : lane & 48) + min(g16 * a.lpg, TEAM - 1), 64);
  if (g16 >= a.G) word = 0u;
  uint32_t ahead = 0;
  auto look = [&](uint32_t o) { ahead += o > word ? 1u : 0u; };
  look(dpp<0x121>(word)), look(dpp<0x122>(word)), look(dpp<0x123>(word)), look(dpp<0x124>(word));
  look(dpp<0x125>(word)), look(dpp<0x126>(word)), look(dpp<0x127>(word)), look(dpp<0x128>(word));
  look(dpp<0x129>(word)), look(dpp<0x12A>(word)), look(dpp<0x12B>(word)), look(dpp<0x12C>(word));
  look(dpp<0x12D>(word)), look(dpp<0x12E>(word)), look(dpp<0x12F>(word));
  const bool keep = word != 0u && ahead < (uint32_t)a.topk_groups;
  uint32_t kept = keep ? 1u << g16 : 0u;
  kept |= dpp<0x128>(kept);
  kept |= dpp<0x124>(kept);
  kept |= dpp<0x122>(kept);
  kept |= dpp<0x121>(kept);
  const uint32_t lowest = ~row_max(keep ? ~word : 0u), left = row_max(keep ? 0u : word);
  // (more than topk_groups stay only among equals)
  const bool sure = __builtin_popcount(kept) <= a.topk_groups &&
                    (left == 0u || rank_value(left) < rank_value(lowest) - a.topn * (tol + 2.4e-7f * most));
  if (a.whole) {
    const bool mine = (kept >> ((rl / a.lpg) & 31)) & 1u;
#pragma unroll
    for (int i = 0; i < EPL; ++i) w[i] = mine ? w[i] : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (!((kept >> (group_of(rl * EPL + i, a) & 31)) & 1u)) w[i] = 0u;  // (places without an expert hold 0 already)
  }
  return sure;
}

// Tokens on fp32 keys, one per TEAM lanes; false (nothing written) on the lanes of
// those that have to be routed again.  Slots whose fp32 keys are closer than their
// error are put in order by the fp64 keys of the chosen experts and of the first
// one left out; what is left to fp64 altogether are groups that close, a third
// expert as close to the last slot, or equal words in one lane.
//
// The keys' error: a sigmoid's exponential is off by its argument's rounding,
// at most |x| 2^-24 log2 e relative, which the slope, s (1 - s) |x| <= 0.23, brings
// to 2e-8, and by one unit in the last place, 3e-8 after the slope; the sum and
// the reciprocal add 1.8e-7 s: 2.3e-7 in all, `tol` covers two.  A softmax's is off
// by as much of the largest score, and by the 40 roundings of its sum (2.4e-6
// of a score).  The sum with the bias adds 6e-8 of the key, and so does the difference
// that the bound is compared through.
template <int EPL, int TEAM>
__device__ __forceinline__ bool route_fp32(const RouteArgs& a, int t, int kt, uint32_t* lds, int rl,
                                           float* __restrict__ sum_out) {
  float v[EPL], bias[EPL], s[EPL];
  const int e0 = rl * EPL;
  load_experts<EPL>(a, t, e0, v, bias);
  if (a.parts > 1 && sum_out) {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (e0 + i < a.E) sum_out[(size_t)t * a.E + e0 + i] = v[i];
  }
  uint32_t w[EPL];
  float m = 0.f, tol = 5.0e-7f;
  auto avail = [&](int i) {  // (a NaN bias compares false)
    return e0 + i < a.E && bias[i] > -__builtin_inff() && v[i] == v[i];
  };
  if (a.score == MOE_SCORE_SOFTMAX) {
    uint32_t mw = 0u;
#pragma unroll
    for (int i = 0; i < EPL; ++i) mw = max(mw, avail(i) ? rank_word32(finite(v[i])) : 0u);
    mw = team_max<TEAM>(mw);
    m = mw ? rank_value(mw) : 0.f;
    float d = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      s[i] = avail(i) ? __expf(finite(v[i]) - m) : 0.f;
      d += s[i];
    }
    d = team_sum<TEAM>(d);
    const float r = d > 0.f ? 1.0f / d : 0.f;
    // the largest score is r; the sum's error is common to all scores, so it moves
    // two close keys apart by no more than it moves their biases' difference
    float b = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) b = fmaxf(b, avail(i) && bias[i] < __builtin_inff() ? fabsf(bias[i]) : 0.f);
    b = __uint_as_float(team_max<TEAM>(__float_as_uint(b)));
    tol = 5.0e-7f * r + 5.0e-6f * fminf(r, b);
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] *= r;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-v[i]));
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) w[i] = avail(i) ? rank_word32(s[i] + bias[i]) : 0u;
  bool sure = true;
  if (a.G > 1)
    sure = a.topn == 1 ? keep_groups<EPL, TEAM, 1>(w, a, lds, rl, tol)
                       : (a.topn == 2 ? keep_groups<EPL, TEAM, 2>(w, a, lds, rl, tol)
                                      : keep_groups<EPL, TEAM, kMaxGroupTopn>(w, a, lds, rl, tol));
  uint32_t left = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) left += w[i] != 0u ? 1u : 0u;
  // rounds of the wavefront's tokens together, as many as the longest needs; lane
  // j < 16 of a token keeps the j-th best expert and its word, one more than the
  // slots where there is a lane for it, and `after` the word that follows those
  const int cands = min(kt + 1, 16);
  int most = cands;
  if constexpr (TEAM == 16) {
    most = max(most, __shfl_xor(most, 16, 64));
    most = max(most, __shfl_xor(most, 32, 64));
  }
  most = __builtin_amdgcn_readfirstlane(most);
  int my_id = -1;
  uint32_t mine = 0u, after = 0u, rounds = 0;
  for (int j = 0; j <= most; ++j) {
    uint32_t best = w[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) best = max(best, w[i]);
    best = team_max<TEAM>(best);
    if (j == cands) after = best;
    if (j == most) break;
    uint32_t id = 0;
    const uint32_t match = best != 0u ? best : 0xFFFFFFFFu;  // (no word is all ones)
    bool hit[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      hit[i] = w[i] == match;
      id = hit[i] ? (uint32_t)(e0 + i) : id;
    }
    id = team_max<TEAM>(id);
    const bool owner = id - (uint32_t)e0 < (uint32_t)EPL;  // of equal words one lane's go
#pragma unroll
    for (int i = 0; i < EPL; ++i) w[i] = hit[i] && owner ? 0u : w[i];
    rounds += best != 0u ? 1u : 0u;
    if (rl == j && j < cands && best != 0u) {
      my_id = (int)id;
      mine = best;
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) left -= w[i] != 0u ? 1u : 0u;
  sure = sure && team_sum<TEAM>(left) == rounds;  // (else a lane lost equal words)
  auto below = [&](uint32_t word, float f) { return rank_value(word) < f - (tol + 2.4e-7f * fabsf(f)); };
  const float f = rank_value(mine);
  if (rl == kt - 1 && mine != 0u && after != 0u && !below(after, f)) sure = false;
  uint32_t next = dpp<0x101>(mine);  // of lane + 1 (0 behind the row)
  if (cands == 16 && rl == 15) next = 0u;
  const bool close = rl < kt && mine != 0u && next != 0u && !below(next, f);
  // scores of the candidates in fp64 (a softmax's up to their common factor)
  double g = 0.0, d = 0.0;
  if (my_id >= 0) {
    const float* lt = a.logits + (size_t)t * a.E;
    float x = lt[my_id];
    for (int p = 1; p < a.parts; ++p) x += lt[p * a.part_stride + my_id];
    x = finite(x);
    g = a.score == MOE_SCORE_SOFTMAX ? exp((double)x - (double)m) : 1.0 / (1.0 + exp(-(double)x));
  }
  const bool any_close = __ballot(close) != 0;
  if (a.score == MOE_SCORE_SOFTMAX && (any_close || !a.renorm)) {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (avail(i)) d += exp((double)finite(v[i]) - (double)m);
    d = team_sum<TEAM>(d);
  }
  if (any_close) {  // neighbours change places where fp64 says so: even and odd pairs, then a look at all
    double key = neg_inf();
    if (my_id >= 0) key = (a.score == MOE_SCORE_SOFTMAX ? g / d : g) + (double)a.select_bias[my_id];
    auto first = [](double ka, int ia, double kb, int ib) { return ib < 0 || (ia >= 0 && (ka > kb || (ka == kb && ia < ib))); };
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      const bool lower = ((rl ^ pass) & 1) == 0;  // this lane is the pair's first
      const double kn = dpp_d<0x101>(key), kp = dpp_d<0x111>(key), gn = dpp_d<0x101>(g), gp = dpp_d<0x111>(g);
      const int in = (int)dpp<0x101>((uint32_t)my_id), ip = (int)dpp<0x111>((uint32_t)my_id);
      if (lower ? rl < 15 : rl > 0) {
        const double ko = lower ? kn : kp, go = lower ? gn : gp;
        const int io = lower ? in : ip;
        const bool keep = my_id < 0 || io < 0 || (lower ? first(key, my_id, ko, io) : first(ko, io, key, my_id));
        if (!keep) {
          key = ko;
          g = go;
          my_id = io;
        }
      }
    }
    const double kn = dpp_d<0x101>(key);
    const int in = (int)dpp<0x101>((uint32_t)my_id);
    if (rl < 15 && my_id >= 0 && in >= 0 && !first(key, my_id, kn, in)) sure = false;
  }
  sure = team_max<TEAM>(sure ? 0u : 1u) == 0u;
  if (rl >= kt) {  // the candidate left out
    my_id = -1;
    g = 0.0;
  }
  if (a.renorm) {
    d = row_sum(g);  // (the slots' lanes are one row)
    g = d > 0.0 ? g / d : 0.0;
  } else if (a.score == MOE_SCORE_SOFTMAX) {
    g /= d;
  }
  if (sure && rl < a.k_max) {
    a.ids[(size_t)t * a.k_max + rl] = my_id;
    a.gates[(size_t)t * a.k_max + rl] = my_id >= 0 ? (float)(g * (double)a.scale) : 0.0f;
  }
  return sure;
}

// ---- a wavefront -------------------------------------------------------------------

// One token on fp64 keys.
template <int EPL>
__device__ __forceinline__ void route_fp64(const RouteArgs& a, int t, int kt, double* lds, int lane,
                                           float* __restrict__ sum_out) {
  const int E = a.E;
  float v[EPL], bias[EPL];
  bool avail[EPL];
  load_experts<EPL>(a, t, lane * EPL, v, bias);
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    avail[i] = lane * EPL + i < E && bias[i] > -__builtin_inff() && v[i] == v[i];
    if (!a.rows && a.parts > 1 && sum_out && lane * EPL + i < E) sum_out[(size_t)t * E + lane * EPL + i] = v[i];
    v[i] = finite(v[i]);
  }

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
  for (int i = 0; i < EPL; ++i) key[i] = avail[i] ? s[i] + (double)bias[i] : neg_inf();

  // group limit: the lanes of a group share its experts, each keeps the topn
  // largest keys of its own, and a butterfly over them merges the lists
  if (a.G > 1) {
    const int G = a.G, topn = a.topn;
    const int gs = a.gs;
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
    a.ids[(size_t)t * a.k_max + lane] = my_id;
    a.gates[(size_t)t * a.k_max + lane] = my_id >= 0 ? (float)(g * (double)a.scale) : 0.0f;
  }
}

// TEAM lanes per token, EPL experts per lane.  own_flags: this launch alone sets the call's
// flag word -- one more block looks through every k_t -- and no launch has to
// clear it before.
template <int EPL, int TEAM>
__global__ __launch_bounds__(256) void k_route_biased(const RouteArgs a, const int32_t* __restrict__ kpt,
                                                      uint32_t* __restrict__ flags, int own_flags,
                                                      float* __restrict__ sum_out) {
  constexpr int WPL = (EPL * TEAM + 63) / 64;  // experts per lane of a wavefront
  constexpr int TPW = 64 / TEAM;               // tokens of a wavefront
  // fp64 keys of a token, or the words of the wavefront's tokens
  __shared__ double s_key[kWavesPerBlock][WPL * 64 > EPL * 32 ? WPL * 64 : EPL * 32];
  const int lane = threadIdx.x & 63, rl = lane % TEAM;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (own_flags && blockIdx.x == gridDim.x - 1) {
    __shared__ int s_bad;
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    if (kpt) {
      bool bad = false;
      for (int i0 = threadIdx.x; i0 < a.T; i0 += 16 * 256) {
        int k[16];  // sixteen loads in flight
#pragma unroll
        for (int q = 0; q < 16; ++q) k[q] = kpt[min(i0 + q * 256, a.T - 1)];
#pragma unroll
        for (int q = 0; q < 16; ++q) bad |= k[q] < 1 || k[q] > a.k_max;
      }
      if (bad) s_bad = 1;
    }
    __syncthreads();
    if (threadIdx.x == 0) *flags = s_bad ? (uint32_t)MOE_FLAG_BAD_K : 0u;
    return;
  }
  const int t0 = (blockIdx.x * kWavesPerBlock + wave) * TPW;
  if (t0 >= a.T) return;  // uniform over the wavefront; nothing below synchronises the block

  // lanes past the last token repeat it (the same values, written twice)
  const int t = min(t0 + lane / TEAM, a.T - 1);
  int kt = kpt ? kpt[t] : a.k_max;
  const bool bad_k = kt < 1 || kt > a.k_max;
  if (bad_k) kt = 0;
  if (bad_k && !own_flags && rl == 0) atomicOr(flags, (uint32_t)MOE_FLAG_BAD_K);
  bool sure = false;
  if (a.rows)
    sure = route_fp32<EPL, TEAM>(a, t, kt, reinterpret_cast<uint32_t*>(s_key[wave]) + (lane / TEAM) * (TEAM * EPL), rl,
                                 sum_out);
  uint64_t again = __ballot(!sure);
  while (again) {  // tokens that fp64 has to decide
    const int from = __builtin_ctzll(again) / TEAM * TEAM;
    again &= TEAM == 64 ? 0ull : ~(0xFFFFull << from);
    route_fp64<WPL>(a, __builtin_amdgcn_readlane(t, from), __builtin_amdgcn_readlane(kt, from), s_key[wave], lane,
                    sum_out);
  }
}

// tokens up to which each takes a whole wavefront (both sides: head of the file)
constexpr int kWideTokens = 1024;

}  // namespace

hipError_t launch_route_biased(const moe_shape& s, const float* logits, const float* select_bias,
                               const int32_t* k_per_token, int32_t* ids, float* gates, uint32_t* flags,
                               bool own_flags, hipStream_t st, int parts, long long part_stride, float* sum_out) {
  const int E = s.num_experts;
  const int team = s.num_tokens <= kWideTokens ? 64 : 16;
  const int per_block = 64 / team * kWavesPerBlock;
  const int grid = (s.num_tokens + per_block - 1) / per_block;
  int epl = 1;  // experts per lane of a token
  while (team * epl < E) epl *= 2;
  RouteArgs a{};
  a.logits = logits;
  a.select_bias = select_bias;
  a.T = s.num_tokens;
  a.E = E;
  a.k_max = s.top_k;
  a.score = s.score;
  a.renorm = s.renormalize;
  a.G = s.num_groups > 1 ? s.num_groups : 1;
  a.topk_groups = s.topk_groups;
  a.topn = s.group_topn > 0 ? s.group_topn : 1;
  a.scale = s.routed_scale;
  a.parts = parts;
  a.part_stride = part_stride;
  a.ids = ids;
  a.gates = gates;
  a.gs = E / a.G;
  a.inv_gs = 1.0f / (float)a.gs;
  const int own = a.gs / epl;
  a.whole = a.gs % epl == 0 && (own & (own - 1)) == 0;
  a.lpg = team;
  while (a.lpg * a.G > team && a.lpg > 1) a.lpg >>= 1;
  if (a.whole) a.lpg = own;
  a.rows = a.G <= 16;
  const auto aligned = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  a.vec = E % 4 == 0 && aligned(logits) && aligned(select_bias);
#define MOE_ROUTE_LAUNCH(EPL, TEAM)                                                                              \
  hipLaunchKernelGGL((k_route_biased<EPL, TEAM>), dim3(grid + (own_flags ? 1 : 0)), dim3(256), 0, st, a,          \
                     k_per_token, flags, own_flags ? 1 : 0, sum_out)
  if (team == 64) {
    switch (epl) {
      case 1: MOE_ROUTE_LAUNCH(1, 64); break;
      case 2: MOE_ROUTE_LAUNCH(2, 64); break;
      case 4: MOE_ROUTE_LAUNCH(4, 64); break;
      default: MOE_ROUTE_LAUNCH(8, 64); break;
    }
  } else {
    switch (epl) {
      case 1: MOE_ROUTE_LAUNCH(1, 16); break;
      case 2: MOE_ROUTE_LAUNCH(2, 16); break;
      case 4: MOE_ROUTE_LAUNCH(4, 16); break;
      case 8: MOE_ROUTE_LAUNCH(8, 16); break;
      case 16: MOE_ROUTE_LAUNCH(16, 16); break;
      default: MOE_ROUTE_LAUNCH(32, 16); break;
    }
  }
#undef MOE_ROUTE_LAUNCH
  return hipGetLastError();
}

}  // namespace moe
