// Internal declarations of the gfx950 MoE-layer library (not part of the C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "moe_mi355x.h"

namespace moe {

constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 16;
constexpr int kDispatchTileSlots = 1024;  // slots per dispatch tile (one block)

// One row-tile of the grouped GEMM: `rows` (1..BM) consecutive permuted rows
// starting at row0, all belonging to `expert`.  group: for big tiles, the tile's
// place among up to kTileGroup neighbours of its expert, and their number
// (tile_group), which a launch may take column by column.
struct MTile {
  int expert;
  int row0;
  int rows;
  int group;
};
constexpr int kTileGroup = 8;
__host__ __device__ constexpr int tile_group(int place, int size) { return (size << 8) | place; }

// compute units of one MI355X (8 XCDs x 32)
constexpr int kUnits = 256;

// Byte offsets of every region inside the caller's workspace.
// MXFP8 layers add the quantised x (xq, scales xsc with stride T, and the
// same scales in dispatch-row order, xscp with stride T*top_k) and the scales
// of h (hsc, stride T*top_k) and of the shared expert's h (hssc, stride T);
// h and hs then hold one-byte codes.  Int8 layers keep h and hs in fp16 and
// add their codes (hq, hsq: the hq region serves both) and the fp32 row scales
// of x (xsc), h (hsc) and hs (hssc).  Block calls with a norm in front add the
// normed x (xn).
struct WsLayout {
  size_t xn, hq, flags, logits, logits_parts, ids, gates, counts, offsets, tile_counts, row_of_slot, row_token,
      num_dropped, sched_big, sched_small, sched_count, h, y, hs, ys, xq, xsc, xscp, hsc, hssc, gu_parts,
      ep_tile_counts, total;
  int n_dispatch_tiles;
  // K-split of the layer's down projection (decode-sized layers, and layers
  // with few 256-row tiles): y holds ksplit partial sums,
  // part p at y + p * slots * H floats (1: no split)
  int ksplit;
  // K-split of the gate/up projection for a token or two (routed experts,
  // ks_gu) and of the shared expert's for a few tokens (ks_gus): fp32
  // partial gate and up sums in gu_parts, reduced by launch_swiglu_parts
  int ks_gu, ks_gus;
  int max_tiles_big, max_tiles_small;
  // int8 layers: the routed and the shared expert's products run as streams
  // of the weights (launch_stream_i8; then ksplit, ks_gu and ks_gus are 1)
  bool stream, stream_shared;
};

// K from which the 32-row bf16 down tiles are 8-wave 32 x 256 blocks (else
// 4-wave 32 x 128)
constexpr int kDown8MinK = 2048;

// Row-tile height of the weight-streaming class in the interleaved
// (big + small) launches: an expert of up to 64 rows (or a big expert's tail
// of up to 64 rows) streams each weight tile once, where 32-row tiles would
// stream it once per 32 rows; the extra MFMA work stays hidden behind the
// weight stream.
constexpr int kMergedSmallRows = 64;

// K-split parts of the MFMA router (E > 32 and more tokens than the sliced
// vector router takes): 2 when its tiles keep fewer blocks than compute
// units busy, else 1
int router_parts(const moe_shape& s);

// GEMM tile configuration chosen by the host for a shape.
// Row tiling of the grouped GEMMs.  Experts with at least split_rows kept rows
// are cut into tiles of bm_big rows, the others into tiles of bm_small rows;
// each class gets its own tile list and launch (split_rows = 0: all big,
// INT_MAX: all small).
struct GemmPlan {
  int bm_big, bm_small, split_rows;
  int tail_rows = 0;  // remainder rows of a big expert placed on small tiles (0: none)
  bool has_big() const { return split_rows != 0x7fffffff; }
  bool has_small() const { return split_rows != 0; }
};

GemmPlan choose_gemm_plan(const moe_shape& s);
// number format of the experts
enum ExpertFormat { kExpertsAct = 0, kExpertsMX = 1, kExpertsI8 = 2 };
// normed: the call also keeps a normed copy of x
WsLayout plan_workspace(const moe_shape& s, int format = kExpertsAct, bool normed = false);

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Raises a kernel's dynamic LDS limit once per device when it exceeds the
// default 64 KiB (setting it again is harmless, so concurrent first calls may
// both set it).
inline hipError_t allow_lds(const void* kernel, int lds, std::atomic<uint64_t>& set_on) {
  if (lds <= 65536) return hipSuccess;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (set_on.load(std::memory_order_acquire) & bit) return hipSuccess;
  e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  set_on.fetch_or(bit, std::memory_order_release);
  return hipSuccess;
}

// ---- launchers (each returns the launch status) ----------------------------
hipError_t launch_clear_flags(uint32_t* flags, hipStream_t st);

// logits may come in `parts` partial sums part_stride floats apart (a
// K-split router); their sums are then also written to sum_out (nullable)
hipError_t launch_route_topk(const moe_shape& s, const float* logits, const int32_t* k_per_token,
                             int32_t* ids, float* gates, uint32_t* flags, hipStream_t st, int parts = 1,
                             long long part_stride = 0, float* sum_out = nullptr);

hipError_t launch_logistic(const float* x, float* y, long long n, hipStream_t st);

// S1 without MFMA for bf16 layers with at most kRouterSkinnyMaxExperts experts
constexpr int kRouterSkinnyMaxExperts = 32;
// ... and for more experts up to this many tokens (slices of 8 experts; the
// 128-row MFMA router keeps only a few compute units busy below it)
constexpr int kRouterSlicedMaxTokens = 1024;
bool router_skinny_supported(const moe_shape& s);
// (flags, nullable: cleared to 0 by the launch)
hipError_t launch_router_skinny(const moe_shape& s, const void* x, const void* w_router,
                                const float* bias, float* logits, uint32_t* flags, hipStream_t st);

hipError_t launch_dispatch(const moe_shape& s, const int32_t* ids, int32_t* counts,
                           int32_t* offsets, int32_t* row_of_slot, int32_t* row_token,
                           int32_t* num_dropped, int32_t* tile_counts, int n_tiles,
                           uint32_t* flags, hipStream_t st);

// phys[s] = replica of slot s's expert (rank in the uncapped dispatch mod n_e)
hipError_t launch_map_replicas(const moe_shape& s, const int32_t* ids, const int32_t* row_of_slot,
                               const int32_t* offsets, const int32_t* rep_off,
                               const int32_t* rep_exp, int num_physical, int32_t* phys,
                               uint32_t* flags, hipStream_t st);

hipError_t launch_gather(const moe_shape& s, const void* x, const int32_t* row_token,
                         const int32_t* offsets, void* x_perm, hipStream_t st);

// Both tile lists (see GemmPlan); count[0] = big tiles, count[1] = small tiles.
// flags (nullable) is cleared.  fill_cols > 0 (kernels that take tiles of any
// height): the column tiles of the launch; the row tiles of a sparse last
// round are cut in kFillSplit (some parts without rows; the list needs room
// for kUnits more).
constexpr int kFillSplit = 4;
hipError_t launch_build_schedule(const int32_t* offsets, int E, const GemmPlan& plan,
                                 MTile* sched_big, int max_big, MTile* sched_small, int max_small,
                                 int32_t* count, hipStream_t st, uint32_t* flags = nullptr, int fill_cols = 0);

// Grouped GEMMs.  `sched`/`count` give the row tiles; when sched == nullptr
// the rows [0, static_rows) form one group (expert 0) tiled statically.
// gate/up + SwiGLU: h[r][n] = silu(A[r].Bg[e][n]) * (A[r].Bu[e][n]); for bf16
// layers h is fp16 and values outside fp16's range set MOE_FLAG_H_RANGE
// a_rows (nullable): A row r is A[a_rows[r]] (the dispatch gather fused into
// the tile loads); else A is contiguous.
hipError_t launch_gemm_gateup(int dtype, int bm, const void* A, const int32_t* a_rows, int lda,
                              const void* Bg, const void* Bu, int N, int K, void* h, int ldh,
                              const MTile* sched, const int32_t* count, int max_tiles,
                              int static_rows, uint32_t* flags, hipStream_t st);
// gate/up on 32-row tiles with K split into ksplit ranges, no SwiGLU: range
// p's fp32 sums A.Bg^T at parts + p * part_elems and A.Bu^T at parts +
// (ksplit + p) * part_elems (rows of N floats); bf16 layers.
hipError_t launch_gemm_gateup_parts(const void* A, const int32_t* a_rows, int lda, const void* Bg,
                                    const void* Bu, int N, int K, float* parts, const MTile* sched,
                                    const int32_t* count, int max_tiles, int static_rows, int ksplit,
                                    long long part_elems, hipStream_t st);
// h[r] = fp16(silu(sum of gate parts) * sum of up parts) for r below *rows_dev
// (or static_rows when rows_dev is null); max_rows bounds the grid.
hipError_t launch_swiglu_parts(const float* parts, int nparts, long long part_elems, int N,
                               const int32_t* rows_dev, int static_rows, int max_rows, void* h, int ldh,
                               uint32_t* flags, hipStream_t st);
// The same two steps on MXFP8 operands; the reduction re-quantises h (codes
// [rows][N], scales as the MXFP8 gate/up epilogue writes them).
hipError_t launch_gemm_gateup_mx_parts(const void* A, const int32_t* a_rows, const uint8_t* sa,
                                       int sa_stride, const void* Bg, const uint8_t* sbg, const void* Bu,
                                       const uint8_t* sbu, int sb_stride, int N, int K, float* parts,
                                       const MTile* sched, const int32_t* count, int max_tiles,
                                       int static_rows, int ksplit, long long part_elems, hipStream_t st,
                                       bool sa_direct);
hipError_t launch_swiglu_parts_mx(const float* parts, int nparts, long long part_elems, int N,
                                  const int32_t* rows_dev, int static_rows, int max_rows, void* h,
                                  uint8_t* hsc, int hs_stride, uint32_t* flags, hipStream_t st);
// plain: Y[r][n] = A[r].B[e][n] (+ bias[n]), fp32 out.  a_is_h: A is the
// fp16 h of a bf16 layer (down projection), B is converted to fp16 on load.
// ksplit > 1 (32-row down tiles): K in ksplit ranges of whole 64-element
// stages, range p's partial sums at Y + p * part_elems.
// y_half (down projections of a bf16 layer, ksplit 1): Y is fp16 instead of
// fp32; values outside fp16's range set MOE_FLAG_Y_RANGE in flags.
hipError_t launch_gemm_plain(int dtype, int bm, bool a_is_h, const void* A, int lda,
                             const void* B, int N, int K, const float* bias, void* Y, int ldy,
                             const MTile* sched, const int32_t* count, int max_tiles,
                             int static_rows, hipStream_t st,
                             int ksplit = 1, long long part_elems = 0, bool y_half = false,
                             uint32_t* flags = nullptr, bool w16 = false);
// w16 (down projections, a_is_h): B holds fp16 weights (moe_convert_bf16_to_f16)
hipError_t launch_bf16_to_f16(const void* src, void* dst, long long n, hipStream_t st);

// MXFP8 path (codes + E8M0 scales; scale words group-major, see mxfp8.hip).
// Quantises rows x cols (cols a multiple of 128) of bf16 / fp32 src; inf/NaN
// inputs set MOE_FLAG_H_RANGE when flags is given.
// row_of_slot (nullable, [rows][k]): also write each scale byte at the
// dispatch rows of the row's kept slots in perm_scales (stride perm_stride).
hipError_t launch_quant_mxfp8(int src_dtype, const void* src, int rows, int cols, int stride,
                              uint8_t* codes, uint8_t* scales, uint32_t* flags, hipStream_t st,
                              const int32_t* row_of_slot = nullptr, int k = 0,
                              uint8_t* perm_scales = nullptr, int perm_stride = 0);
// gate/up + SwiGLU with h re-quantised to MXFP8; bm 256 / 128 / 32
hipError_t launch_gemm_gateup_mx(int bm, const void* A, const int32_t* a_rows, const uint8_t* sa,
                                 int sa_stride, const void* Bg, const uint8_t* sbg, const void* Bu,
                                 const uint8_t* sbu, int sb_stride, int N, int K, void* h,
                                 uint8_t* hsc, int hs_stride, const MTile* sched,
                                 const int32_t* count, int max_tiles, int static_rows,
                                 uint32_t* flags, hipStream_t st, bool sa_direct = false);
hipError_t launch_gemm_down_mx(int bm, const void* A, const uint8_t* hsc, int hs_stride,
                               const void* B, const uint8_t* sb, int sb_stride, int N, int K,
                               void* Y, int ldy, const MTile* sched, const int32_t* count,
                               int max_tiles, int static_rows, hipStream_t st,
                               int ksplit = 1, long long part_elems = 0, bool y_half = false,
                               uint32_t* flags = nullptr);

// Both row-tile classes (256-row and 32-row tiles of the big and small
// schedules) in one interleaved launch.
hipError_t launch_gemm_gateup2(const void* A, const int32_t* a_rows, int lda, const void* Bg,
                               const void* Bu, int N, int K, void* h, int ldh, const MTile* sb,
                               const int32_t* cb, int mb, const MTile* ss, const int32_t* cs, int ms,
                               uint32_t* flags, hipStream_t st);
hipError_t launch_gemm_down2(const void* A, int lda, const void* B, int N, int K, void* Y, int ldy,
                             const MTile* sb, const int32_t* cb, int mb, const MTile* ss,
                             const int32_t* cs, int ms, hipStream_t st, int ksplit = 1,
                             long long part_elems = 0, bool y_half = false, uint32_t* flags = nullptr,
                             bool w16 = false);
hipError_t launch_gemm_gateup_mx2(const void* A, const int32_t* a_rows, const uint8_t* sa, int sa_stride,
                                  const void* Bg, const uint8_t* sbg, const void* Bu, const uint8_t* sbu,
                                  int sb_stride, int N, int K, void* h, uint8_t* hsc, int hs_stride,
                                  const MTile* sb, const int32_t* cb, int mb, const MTile* ss,
                                  const int32_t* cs, int ms, uint32_t* flags, hipStream_t st,
                                  bool sa_direct = false);
hipError_t launch_gemm_down_mx2(const void* A, const uint8_t* hsc, int hs_stride, const void* B,
                                const uint8_t* sb_w, int sb_stride, int N, int K, void* Y, int ldy,
                                const MTile* sb, const int32_t* cb, int mb, const MTile* ss,
                                const int32_t* cs, int ms, hipStream_t st, int ksplit = 1,
                                long long part_elems = 0, bool y_half = false, uint32_t* flags = nullptr);

// Row-tile height the GEMM launchers use for a dtype and a requested height.
int gemm_tile_rows(int dtype, int bm_hint);

// ---- int8 operands (gemm.hip, int8.hip) ----------------------------------------
// Token codes A with one fp32 scale per row (sa; gathered through a_rows with
// the rows), weight codes with one per output channel (sb*, expert e's start at
// e * N), int32 sums.  K a multiple of 128, N of 16, bm 256, 128 or 32.
hipError_t launch_gemm_gateup_i8(int bm, const void* A, const int32_t* a_rows, const float* sa, const void* Bg,
                                 const float* sbg, const void* Bu, const float* sbu, int N, int K, void* h,
                                 const MTile* sched, const int32_t* count, int max_tiles, int static_rows,
                                 uint32_t* flags, hipStream_t st);
// the int32 gate and up sums of ksplit ranges of K (32-row tiles): range p's at
// parts + p * part_elems and parts + (ksplit + p) * part_elems
hipError_t launch_gemm_gateup_i8_parts(const void* A, const int32_t* a_rows, const void* Bg, const void* Bu, int N,
                                       int K, int32_t* parts, const MTile* sched, const int32_t* count,
                                       int max_tiles, int static_rows, int ksplit, long long part_elems,
                                       hipStream_t st);
// y = sa sb A.B^T in y_dtype; ksplit > 1 (fp32): K in ksplit ranges, range p's
// share at Y + p * part_elems
hipError_t launch_gemm_down_i8(int bm, const void* A, const float* sa, const void* B, const float* sb, int N, int K,
                               int y_dtype, void* Y, const MTile* sched, const int32_t* count, int max_tiles,
                               int static_rows, uint32_t* flags, hipStream_t st, int ksplit = 1,
                               long long part_elems = 0);
// row tiles of up to 256 rows, each at the height its rows need; halves: as two
// of up to 128, on tiles of 128 columns instead of 256
hipError_t launch_gemm_gateup_i8_rows(const void* A, const int32_t* a_rows, const float* sa, const void* Bg,
                                      const float* sbg, const void* Bu, const float* sbu, int N, int K, void* h,
                                      const MTile* sched, const int32_t* count, int max_tiles, uint32_t* flags,
                                      hipStream_t st);
hipError_t launch_gemm_down_i8_rows(const void* A, const float* sa, const void* B, const float* sb, int N, int K,
                                    int y_dtype, void* Y, const MTile* sched, const int32_t* count, int max_tiles,
                                    bool halves, uint32_t* flags, hipStream_t st, int ksplit = 1,
                                    long long part_elems = 0);
// The products of few rows (stream_i8.hip).  offsets [E + 1] (null: rows [0,
// static_rows) of one expert); max_tiles bounds the 32-row tiles, max_rows the
// rows of an expert.  clear_flags: the launch first clears the flag word (it
// adds to it only for an fp16 y, so then another launch has to clear it).
// Gate/up with SwiGLU to fp16 h; values out of fp16's range become infinite.
hipError_t launch_stream_gateup_i8(const void* A, const int32_t* a_rows, const float* sa, const moe_int8_ffn& w,
                                   int N, int K, void* h, const int32_t* offsets, int E, int max_tiles,
                                   int max_rows, int static_rows, uint32_t* flags, bool clear_flags, hipStream_t st);
// y = sa sb A.B^T in y_dtype.  sa null (max_rows <= 16): A holds fp16 rows,
// quantised on the way (infinite values: as launch_quant_int8).
hipError_t launch_stream_i8(const void* A, const float* sa, const void* B, const float* sb, int N, int K, int y_dtype,
                            void* y, const int32_t* offsets, int E, int max_tiles, int max_rows, int static_rows,
                            uint32_t* flags, bool clear_flags, hipStream_t st);
// rows of src (bf16, fp32 or fp16) to int8 codes and a scale per row; rows at
// and beyond *rows_dev (nullable) are left alone.  h_flags (nullable, fp16): an
// infinite value counts as the largest finite one and sets MOE_FLAG_H_RANGE.
hipError_t launch_quant_int8(int src_dtype, const void* src, int rows, int cols, const int32_t* rows_dev, void* codes,
                             float* scales, hipStream_t st, uint32_t* h_flags = nullptr);
// h = fp16(silu(g) u) from int32 partial sums (see launch_gemm_gateup_i8_parts)
hipError_t launch_swiglu_parts_i8(const int32_t* parts, int nparts, long long part_elems, int N,
                                  const int32_t* a_rows, const float* sa, const float* sbg, const float* sbu,
                                  const MTile* sched, const int32_t* count, int max_tiles, int static_rows,
                                  void* h, uint32_t* flags, hipStream_t st);
// y = the sum of nparts partial sums in order, in y_dtype
hipError_t launch_sum_parts(const float* parts, int nparts, long long part_elems, int N, const int32_t* rows_dev,
                            int max_rows, int y_dtype, void* y, uint32_t* flags, hipStream_t st);

// ---- 8-bit floating-point operands with a scale per block of 128 (gemm_fp8.hip) ------
// Row codes A [rows][K] with fp32 scales (row r, group g at sa[r * sa_row + g *
// sa_group]), weight codes B0 (and B1 for gate/up) [E][N][K] with one scale per 128 x
// 128 block ([E][N / 128 up][K / 128]).  K a multiple of 128, N of 16.
struct Fp8Args {
  const uint8_t* A;
  const float* sa;
  long long sa_row, sa_group;
  const uint8_t* B0;
  const uint8_t* B1;
  const float* sb0;
  const float* sb1;
  int N, K;
  void* out;
  int y_dtype;            // MOE_F16 or MOE_BF16 (one matrix)
  const MTile* sched;     // row tiles, their number and the queues (launch_schedule_fp8)
  int32_t* count;
  int static_rows;        // streams without offsets
  uint32_t* flags;
  float* out_scales;      // gate/up: scale of h row r, group g at g * out_group + r
  long long out_group;
  const int32_t* offsets; // streams: [E + 1]; null: rows [0, static_rows) of expert 0
};
// one matrix: y; dual (gate/up): h as codes and scales.  Row tiles of up to 256 rows;
// halves (one matrix): as two of up to 128, on 128 columns instead of 256, of at most
// row_tiles uncut ones (the large tiles' blocks draw theirs from the schedule alone).  A
// schedule serves one launch of either kind.
hipError_t launch_gemm_fp8(const Fp8Args& a, bool dual, bool halves, int row_tiles, hipStream_t st);
// count: all tiles, those before the quarter tiles, and a queue for each kind of launch
constexpr int kFp8QueueUp = 4, kFp8QueueDown = 16, kFp8CountWords = 32;
hipError_t launch_schedule_fp8(const int32_t* offsets, int E, int static_rows, MTile* sched, int max_tiles,
                               int32_t* count, uint32_t* flags, int fill_cols, hipStream_t st);
// The products of few rows (stream_fp8.hip), 32-row tiles; max_tiles bounds them,
// max_rows the rows of an expert.  dual: fp32 h.  quantise (one matrix, max_rows <= 16):
// A holds fp32 h, quantised on the way (an h that is not finite sets MOE_FLAG_H_RANGE).
// clear_flags: the launch first clears the flag word (it adds to it only for an fp16 y or
// where it quantises, so then another launch has to clear it).
hipError_t launch_stream_fp8(const Fp8Args& a, bool dual, bool quantise, int E, int max_tiles, int max_rows,
                             bool clear_flags, hipStream_t st);

// rows [rows][cols] (cols a multiple of 128) to codes and scales [rows][cols / 128];
// rows at and beyond *rows_dev (nullable) are left alone.  h_flags (nullable): a value
// that is not finite sets MOE_FLAG_H_RANGE
hipError_t launch_quant_fp8(int src_dtype, const void* src, int rows, int cols, const int32_t* rows_dev, void* codes,
                            float* scales, hipStream_t st, uint32_t* h_flags = nullptr);
hipError_t launch_quant_fp8_weights(int src_dtype, const void* src, int experts, int n, int k, void* codes,
                                    float* scales, hipStream_t st);

// ---- rows to expert order and back (rows.hip) ---------------------------------------
// rows named outside [0, num_rows) count as none; weights nullable
hipError_t launch_dispatch_rows(const moe_shape& s, int dtype, const void* x, const int32_t* row_of_slot,
                                const float* weights, int num_rows, void* out, hipStream_t st);
hipError_t launch_dispatch_rows_fp8(const moe_shape& s, int dtype, const void* x, const int32_t* row_of_slot,
                                    int num_rows, void* codes, float* scales, hipStream_t st);
// d_weights (nullable) only with weights and x; d_x nullable with d_weights
hipError_t launch_dispatch_rows_backward(const moe_shape& s, int dtype, const void* d_perm, const int32_t* row_of_slot,
                                         int num_rows, const float* weights, const void* x, void* d_x,
                                         float* d_weights, hipStream_t st);
// d_y or d_gates may be null, y only without d_gates
hipError_t launch_combine_backward(const moe_shape& s, int out_dtype, const void* d_out, int y_dtype, const void* y,
                                   const int32_t* row_of_slot, const float* gates, int num_rows, void* d_y,
                                   float* d_gates, hipStream_t st);

// ---- norms around the layer (block.hip) ------------------------------------------
hipError_t launch_norm(int rows, int cols, int src_dtype, const void* x, const float* weight, float eps,
                       int out_dtype, void* out, void* codes, float* scales, hipStream_t st);
hipError_t launch_combine_norm(const moe_shape& s, const moe_block& b, int y_dtype, const void* y,
                               const int32_t* row_of_slot, const float* gates, const void* y_shared,
                               const void* residual, void* out, hipStream_t st, int parts = 1,
                               long long part_stride = 0);

// ---- routing with a balance bias (route_biased.hip) --------------------------------
// own_flags: the launch writes the flag word itself (else it adds to it);
// for at most kRouteOwnFlagsTokens tokens, or without k_per_token
constexpr int kRouteOwnFlagsTokens = 32768;
hipError_t launch_route_biased(const moe_shape& s, const float* logits, const float* select_bias,
                               const int32_t* k_per_token, int32_t* ids, float* gates, uint32_t* flags,
                               bool own_flags, hipStream_t st, int parts = 1, long long part_stride = 0,
                               float* sum_out = nullptr);

// ---- expert-parallel exchange over G virtual ranks (ep.hip) -----------------
constexpr int kMaxRanks = 64;
// 64-token tiles of the send-layout kernels (tile_counts: tiles x G ints)
int ep_tiles(int num_tokens);
hipError_t launch_ep_layout(const moe_shape& s, int G, const int32_t* ids, const float* gates,
                            int32_t* rank_counts, int32_t* rank_offsets, int32_t* send_token,
                            int32_t* send_ids, float* send_gates, int32_t* slot_send_pos,
                            int32_t* tile_counts, uint32_t* flags, hipStream_t st);
hipError_t launch_ep_combine(const moe_shape& s, int G, const float* partial, const int32_t* slot_send_pos,
                             const float* y_shared, void* out, hipStream_t st);

// y_half: y_perm and y_shared hold fp16 values (then parts must be 1)
hipError_t launch_combine(const moe_shape& s, const void* y_perm, const int32_t* row_of_slot,
                          const float* gates, const void* y_shared, void* out, hipStream_t st,
                          int parts = 1, long long part_stride = 0, bool y_half = false);

}  // namespace moe
