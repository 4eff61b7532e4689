/*
 * moe_mi355x.h -- C ABI of the MI355X (gfx950) MoE-layer forward library.
 *
 * One GPU's share of an expert-parallel Mixture-of-Experts layer forward:
 * router scoring and top-k selection, dispatch of token rows into per-expert
 * contiguous groups, the per-expert SwiGLU FFN as a grouped GEMM, and the
 * gate-weighted combine back to token order.  On one GPU the dispatch and
 * combine all-to-alls of expert parallelism become an on-device permutation
 * and its inverse.
 *
 * Problem statement the arguments follow:
 *   - tokens x hidden in, a router choosing the top-k of E experts per token
 *     ("Expert parallelism for MoE serving", overview and deep dive;
 *     "Expert Parallelism: MoE model parallel split", §1);
 *   - router weights weight the sum of the k expert outputs (same page, §1 and
 *     §12 Q2);
 *   - a per-expert capacity with tokens beyond it dropped ("Expert parallelism
 *     for MoE serving", technical notes and FAQ);
 *   - k as a per-request runtime control (MoE-Prism summary, §1 and §5);
 *   - a shared expert ("LLM MoE Expert Parallel production practice", launch
 *     checklist; "Expert Parallelism: MoE model parallel split", §4);
 *   - node-limited (group-limited) routing ("Expert parallelism for MoE
 *     serving", deployment examples).
 *
 * Conventions for every call:
 *   - Tensor pointers are DEVICE pointers, row-major, owned by the caller and
 *     aligned to 16 bytes.  The library allocates no memory and keeps no state
 *     between calls; scratch space is the caller's workspace `ws` of at least
 *     moe_workspace_size() bytes.  Calls on different streams need distinct
 *     workspaces.  (The one exception, moe_layer_forward_noalloc, takes its
 *     workspace from an array in the library's own device memory.)
 *   - Weights are output-major with K contiguous: router [E][H]; gate and up
 *     [E][I][H]; down [E][H][I]; shared gate/up [Is][H], shared down [H][Is].
 *   - `stream` is a hipStream_t (NULL = the null stream).  Every call only
 *     enqueues work; none synchronises with the host (except
 *     moe_read_device_flags), so calls can be captured in a graph.
 *   - Host-checkable errors return before anything is enqueued.
 *   - Every call that takes a workspace and enqueues work clears its flag word at the
 *     start; the word reports that call only.  A failed
 *     launch returns MOE_ERR_HIP (the HIP error code is kept per thread, see
 *     moe_last_hip_error).  Errors found in data on the device (a k_t outside
 *     [1, k_max], an expert id outside [-1, E)) mark the affected slot unused
 *     and set bits in a flag word at the head of the workspace.
 *   - Routing, counts, offsets and the permutation are bitwise deterministic;
 *     all other outputs are run-to-run deterministic (no atomics in sums).
 *   - num_tokens == 0 is valid and enqueues nothing, and so is rows == 0 where a call
 *     takes its rows' number: outputs and the flag word stay as they were.
 */
#ifndef MOE_MI355X_H
#define MOE_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = -1,  /* null/misaligned pointer, inconsistent shape       */
  MOE_ERR_UNSUPPORTED = -2,  /* valid but outside what the kernels handle         */
  MOE_ERR_WORKSPACE = -3,    /* ws smaller than moe_workspace_size()              */
  MOE_ERR_HIP = -4           /* a HIP call or kernel launch failed                */
} moe_status;

typedef enum { MOE_F32 = 0, MOE_BF16 = 1, MOE_F16 = 2 } moe_dtype;
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;

/* device flag bits (moe_read_device_flags) */
#define MOE_FLAG_BAD_K 1u       /* some k_per_token[t] outside [1, top_k]: token routed nowhere */
#define MOE_FLAG_BAD_EXPERT 2u  /* some topk_ids entry outside [-1, E): slot treated as unused  */
#define MOE_FLAG_H_RANGE 4u     /* some SwiGLU activation h exceeded fp16 range (bf16 and int8
                                   experts) or was not finite (MXFP8 and fp8 experts; int8: or
                                   NaN)                                                        */
#define MOE_FLAG_BAD_REPLICA 8u /* a routed expert without a replica, or a replica id out of range */
#define MOE_FLAG_Y_RANGE 16u    /* some expert output exceeded fp16 range inside a layer call
                                   (moe_layer_forward, moe_layer_forward_mxfp8), a block call or
                                   an fp16 y of the int8 and fp8 calls                         */

typedef struct {
  int32_t num_tokens;          /* T >= 0                                                  */
  int32_t hidden;              /* H; bf16: multiple of 64; fp32: multiple of 4            */
  int32_t num_experts;         /* E in [1, 512]                                            */
  int32_t intermediate;        /* I; same rule as H                                        */
  int32_t top_k;               /* k, or k_max when k_per_token is given; 1..min(E, 16)    */
  int32_t score;               /* moe_score                                                */
  int32_t renormalize;         /* 1: gates divided by their sum over the token's slots     */
  float routed_scale;          /* multiplies routed gates after renormalising (usually 1) */
  int32_t num_groups;          /* G >= 1 consecutive expert groups; 1 = no group limit     */
  int32_t topk_groups;         /* groups kept per token, 1..G (ignored when G == 1)        */
  int32_t group_topn;          /* group score = sum of the group's n best sigmoid scores;
                                  0 means 1; at most E/G                                   */
  float capacity_factor;       /* C = ceil(cf * A / E), A = routed slots; <= 0: no limit   */
  int32_t shared_intermediate; /* Is; 0 = no shared expert; same rule as H                 */
  int32_t act_dtype;           /* moe_dtype of x and of every weight (MOE_F32 or MOE_BF16)  */
  int32_t out_dtype;           /* moe_dtype of the layer output (MOE_F32 or MOE_BF16)       */
  int32_t down_dtype;          /* 0 or act_dtype: the down weights (routed and shared) have
                                  act_dtype; MOE_F16 (bf16 layers only): they were converted
                                  once by moe_convert_bf16_to_f16 -- the same products, without
                                  the conversion inside every call                           */
} moe_shape;
/* Element offsets are int32 inside the kernels: T*top_k <= 2^30 and each of
 * T*H, E*H, I*H and Is*H <= 2^31-1, else MOE_ERR_UNSUPPORTED. */

/* Stages of moe_layer_forward, for the timing events of moe_debug. */
typedef enum {
  MOE_STAGE_ROUTER = 0,   /* S1 router logits                         */
  MOE_STAGE_ROUTE = 1,    /* S2 scoring, top-k, gates                 */
  MOE_STAGE_DISPATCH = 2, /* S3-S5 histogram, capacity, permutation   */
  MOE_STAGE_GATHER = 3,   /* S6 x_perm gather (fused into S7: empty)  */
  MOE_STAGE_GATE_UP = 4,  /* S7 grouped gate/up GEMM + SwiGLU         */
  MOE_STAGE_DOWN = 5,     /* S8 grouped down GEMM                     */
  MOE_STAGE_SHARED = 6,   /* S9 shared expert (both GEMMs)            */
  MOE_STAGE_COMBINE = 7,  /* S10 combine                              */
  MOE_NUM_STAGES = 8
} moe_stage;

/* Optional outputs of moe_layer_forward for inspection and timing.  Each
 * member may be NULL.  Device buffer sizes: logits T*E, topk_ids/topk_gates/
 * row_of_slot/row_token T*top_k, expert_counts E, expert_offsets E+1,
 * num_dropped 1 (row_token as moe_dispatch writes it: entries at and beyond
 * expert_offsets[E] are left untouched).
 * stage_start[i]/stage_stop[i] are hipEvent_t handles recorded on the call's
 * stream immediately before the first and after the last launch of stage i
 * (a stage that does not run records both at the same point). */
typedef struct {
  float* logits;
  int32_t* topk_ids;
  float* topk_gates;
  int32_t* expert_counts;
  int32_t* expert_offsets;
  int32_t* row_of_slot;
  int32_t* num_dropped;
  void* stage_start[MOE_NUM_STAGES];
  void* stage_stop[MOE_NUM_STAGES];
  int32_t* row_token;
} moe_debug;

/* Bytes of workspace every call below needs for this shape (host only, no HIP
 * call).  The same workspace serves all calls. */
moe_status moe_workspace_size(const moe_shape* shape, size_t* bytes);

/* S1 + S2: router logits and top-k selection.  A router picks the top-k
 * experts of each token ("Expert parallelism for MoE serving", deep dive;
 * "Expert Parallelism: MoE model parallel split", §1: router -> top-k experts
 * -> weighted sum), optionally limited to a few groups of experts (node-
 * limited routing, "Expert parallelism for MoE serving", deployment
 * examples), with k chosen per request (MoE-Prism summary, §1 and §5).
 * logits[t][e] = sum_h x[t][h] * w_router[e][h] + router_bias[e], fp32 accumulate.
 * If logits_in is non-NULL it is used instead and x/w_router/router_bias are
 * ignored (may be NULL).  logits_out (nullable) receives the computed logits.
 * Per token t with k_t = k_per_token ? k_per_token[t] : top_k:
 *   eligible experts: all, or with num_groups > 1 those in the topk_groups
 *   groups of E/G consecutive experts with the largest group score;
 *   selection: the k_t eligible experts with the largest logits, equal logits
 *   going to the lower expert index, written to slots 0..k_t-1 in that order;
 *   gates: softmax over all E logits (or sigmoid of the logit), divided by
 *   their sum over the k_t slots when renormalize, times routed_scale.
 * Outputs topk_ids [T][top_k] int32 (-1 in unused slots) and topk_gates
 * [T][top_k] fp32 (0 in unused slots).  Clears the workspace flag word. */
moe_status moe_route_topk(const moe_shape* shape, const void* x, const void* w_router,
                          const float* router_bias, const float* logits_in, float* logits_out,
                          const int32_t* k_per_token, int32_t* topk_ids, float* topk_gates,
                          void* ws, size_t ws_bytes, void* stream);

/* S3-S6: dispatch ("Expert Parallelism: MoE model parallel split" §3 and §12
 * Q2; token sorting §7; capacity from "Expert parallelism for MoE serving").
 * Slots s = t*top_k + j are visited in token-major order.
 *   expert_counts[e]  = routed slots with id e                         [E]
 *   C                 = ceil(capacity_factor * A / E) in fp64 (A = sum of counts),
 *                       unlimited when capacity_factor <= 0
 *   expert_offsets    = exclusive prefix sum of min(count, C)          [E+1]
 *   row_of_slot[s]    = expert_offsets[e] + (rank of s among slots of e), or -1
 *                       when the slot is unused or its rank >= C       [T][top_k]
 *   row_token[row]    = t for every kept row (rows >= R left untouched) [T*top_k]
 *   num_dropped       = A - R, R = expert_offsets[E]                   [1]
 *   x_perm[row]       = x[row_token[row]] (skipped when x or x_perm is NULL)
 * Clears the workspace flag word, then sets MOE_FLAG_BAD_EXPERT in it for ids
 * outside [-1, E).  expert_offsets[E] <= T*top_k always holds on return. */
moe_status moe_dispatch(const moe_shape* shape, const void* x, const int32_t* topk_ids,
                        int32_t* expert_counts, int32_t* expert_offsets, int32_t* row_of_slot,
                        int32_t* row_token, int32_t* num_dropped, void* x_perm, void* ws,
                        size_t ws_bytes, void* stream);

/* S7-S8: grouped SwiGLU FFN over permuted rows ("LLM MoE Expert Parallel
 * production practice", four-step layer: local expert compute).
 * For every expert e and row r in [expert_offsets[e], expert_offsets[e+1]):
 *   h = silu(x_perm[r] . w_gate[e]^T) * (x_perm[r] . w_up[e]^T),
 *       silu(z) = z / (1 + exp(-z)); fp32 accumulation; h is kept in fp32
 *       for fp32 layers and rounded to fp16 (11-bit significand) for bf16
 *       layers, whose down projection then runs on fp16 inputs (w_down
 *       converted from bf16, exact for |w| >= 2^-14, or already fp16 when
 *       shape->down_dtype is MOE_F16); |h| > 65504 sets MOE_FLAG_H_RANGE
 *   y_perm[r] = h . w_down[e]^T                                    (fp32)
 * Rows at or beyond expert_offsets[E] are not written.  x_perm [T*top_k][H],
 * y_perm [T*top_k][H] fp32.  expert_offsets must be non-decreasing with
 * expert_offsets[0] = 0 and expert_offsets[E] <= T*top_k (as moe_dispatch
 * writes them); the kernels trust them. */
moe_status moe_grouped_ffn(const moe_shape* shape, const void* x_perm,
                           const int32_t* expert_offsets, const void* w_gate, const void* w_up,
                           const void* w_down, float* y_perm, void* ws, size_t ws_bytes,
                           void* stream);

/* Redundant experts: the replica each routed slot goes to.  A hot expert may
 * have identical copies ("LLM MoE Expert Parallel production practice", step
 * 3: selective replicas, the router picks the copy with the lower load;
 * "Expert Parallelism: MoE model parallel split" §6.2: static replicas, the
 * router splits by load).  Logical expert e (of shape->num_experts) has the
 * replicas replica_experts[replica_offsets[e] .. replica_offsets[e+1]),
 * physical expert ids in [0, num_physical).  Slots are visited in token-major
 * order; each goes to the replica of its expert with the fewest slots of this
 * batch assigned so far, ties to the lower replica index -- so the r-th slot
 * of e (token-major) takes replica r mod n_e.
 *   phys_ids[s] = physical expert of slot s, -1 when topk_ids[s] is unused,
 *                 outside [0, E), or e has no valid replica       [T][top_k]
 * topk_ids as moe_route_topk writes them; replica_offsets [E+1] and
 * replica_experts are device arrays (contents checked on the device: an
 * empty replica list or an id outside [0, num_physical) sets
 * MOE_FLAG_BAD_REPLICA and leaves the slot at -1).  The physical ids then go
 * through moe_dispatch / moe_grouped_ffn / moe_combine with num_experts =
 * num_physical and weights [num_physical][..] in which every replica holds its
 * expert's weights; no capacity applies here.  Uses the workspace of
 * `shape`; clears its flag word. */
moe_status moe_map_replicas(const moe_shape* shape, const int32_t* topk_ids,
                            const int32_t* replica_offsets, const int32_t* replica_experts,
                            int32_t num_physical, int32_t* phys_ids, void* ws, size_t ws_bytes,
                            void* stream);

/* S10: combine ("Expert Parallelism: MoE model parallel split" §1 weighted
 * sum, §12 Q2 combine).  out[t] = sum over j ascending with
 * row_of_slot[t][j] >= 0 of topk_gates[t][j] * y_perm[row_of_slot[t][j]],
 * plus y_shared[t] when y_shared is non-NULL; fp32 arithmetic, out in
 * out_dtype. */
moe_status moe_combine(const moe_shape* shape, const float* y_perm, const int32_t* row_of_slot,
                       const float* topk_gates, const float* y_shared, void* out, void* stream);

/* The whole layer: S1-S10 in one call (may fuse steps internally).  The four
 * steps of an MoE layer of "LLM MoE Expert Parallel production practice"
 * (route each token to its top-K experts, send its activations to them, run
 * the expert FFNs, send the outputs back and merge them), with the sends of
 * expert parallelism replaced by an on-device permutation and its inverse
 * ("Expert Parallelism: MoE model parallel split", §1 weighted sum, §3 the
 * dispatch and combine exchanges, §12 Q2 k target positions per token;
 * "Expert parallelism for MoE serving", deep dive and technical notes).
 * out[t] = sum over kept slots of gate * FFN_e(x[t]) + FFN_shared(x[t]):
 * the routing, dispatch, FFN and combine of moe_route_topk, moe_dispatch,
 * moe_grouped_ffn and moe_combine, with the same argument rules.
 * The shared expert runs when shape->shared_intermediate > 0 (then ws_gate,
 * ws_up and ws_down are required; "LLM MoE Expert Parallel production
 * practice", launch checklist; "Expert Parallelism…" §4).  dbg (nullable)
 * receives intermediates.  Clears the workspace flag word. */
moe_status moe_layer_forward(const moe_shape* shape, const void* x, const void* w_router,
                             const float* router_bias, const int32_t* k_per_token,
                             const void* w_gate, const void* w_up, const void* w_down,
                             const void* ws_gate, const void* ws_up, const void* ws_down,
                             void* out, const moe_debug* dbg, void* ws, size_t ws_bytes,
                             void* stream);

/* ---- the expert-parallel exchange over G ranks, on one GPU -------------
 * With expert parallelism over G GPUs ("Expert Parallelism: MoE model
 * parallel split", §8: each GPU holds one contiguous block of E/G experts)
 * every MoE layer exchanges twice (§3, §12 Q2): dispatch sends each token's
 * hidden state to the ranks holding its experts, combine returns their
 * outputs to the token's own rank.  Rows bound for one rank are grouped into
 * one send (§7 and §12, token sorting), and a token travels once to each
 * rank holding any of its experts -- with node-limited routing ("Expert
 * parallelism for MoE serving", deployment examples; group-limited routing
 * with num_groups = G here) at most topk_groups ranks rather than k copies.
 * The two calls below are the source side of both exchanges, run with G
 * virtual ranks on one GPU: the send layout, and the sum of the rows the
 * ranks return.  A rank's own work on the rows it receives is the step
 * chain moe_dispatch / moe_grouped_ffn / moe_combine with its local expert
 * ids, its E/G experts' weights and the received gates (num_tokens = its
 * row count): one pre-reduced row per received row.  Capacity, if any, is
 * the receiving rank's: the layout sends every routed slot. */

/* Send layout of the dispatch exchange.  Rank d holds experts d*E/G ..
 * (d+1)*E/G - 1 (1 <= G <= 64, E % G == 0).  Rows are destination-major,
 * tokens ascending within a rank, no padding:
 *   rank_counts[d]      rows for rank d                                  [G]
 *   rank_offsets        exclusive prefix sum of rank_counts              [G+1]
 *   send_token[p]       token of row p                                   [n_rows]
 *   send_ids[p][j]      topk_ids[t][j] - d*E/G for the slots j of token t
 *                       on rank d, -1 for its other slots                [n_rows][k]
 *   send_gates[p][j]    topk_gates[t][j] where send_ids[p][j] >= 0, else 0
 *   slot_send_pos[t][j] row p of token t's row for the rank of slot j,
 *                       -1 for an unused slot                            [T][k]
 *   send_x[p]           x[send_token[p]] for p < rank_offsets[G]  [n_rows][H]
 *                       (skipped when x and send_x are NULL)
 * n_rows = T * min(top_k, G).  Rows from rank_offsets[G] to n_rows - 1 get
 * send_token -1, send_ids -1 and send_gates 0 (send_x is not written there).
 * topk_ids / topk_gates as moe_route_topk writes them; ids outside [-1, E)
 * count as unused and set MOE_FLAG_BAD_EXPERT.  Uses the workspace of
 * `shape`; clears its flag word.  Positions are bitwise deterministic. */
moe_status moe_ep_dispatch_layout(const moe_shape* shape, int32_t num_ranks, const int32_t* topk_ids,
                                  const float* topk_gates, const void* x, int32_t* rank_counts,
                                  int32_t* rank_offsets, int32_t* send_token, int32_t* send_ids,
                                  float* send_gates, int32_t* slot_send_pos, void* send_x, void* ws,
                                  size_t ws_bytes, void* stream);

/* The combine exchange's last step at the source: partial [n_rows][H] fp32
 * holds, at each row p of the send layout, the gate-weighted sum of the
 * outputs of the experts of rank d for token send_token[p] (what rank d
 * returns).  out[t] = sum of the token's distinct rows (the non-negative
 * slot_send_pos[t][*]) in ascending order -- ascending rank -- plus
 * y_shared[t] when non-NULL; fp32 arithmetic; out in out_dtype.  A token
 * with no routed slot gets y_shared[t] or 0.  No workspace. */
moe_status moe_ep_combine(const moe_shape* shape, int32_t num_ranks, const float* partial,
                          const int32_t* slot_send_pos, const float* y_shared, void* out, void* stream);

/* ---- the layer without a caller workspace ------------------------------
 * For callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc.  Computes
 * exactly what moe_layer_forward computes (same kernels, bit-identical
 * results) with its workspace taken from an array the library keeps in its
 * own device memory: MOE_NOALLOC_SCRATCH_BYTES per GPU, placed when the
 * library's code is loaded on that GPU and held until the process ends.  The
 * call allocates nothing (no hipMalloc, hipFree or allocating library call);
 * its first call on a GPU looks up that GPU's array (the current device's;
 * `stream` must belong to it).  Shapes whose moe_workspace_size() exceeds
 * MOE_NOALLOC_SCRATCH_BYTES return MOE_ERR_WORKSPACE before anything is
 * enqueued (e.g. decode-sized layers fit: 64 tokens of a Mixtral-8x7B-shaped
 * layer need 7.5 MiB, of a DeepSeek-V3-shaped layer 34 MiB).  Every call on a
 * GPU shares that GPU's array and leaves its contents behind; each call
 * clears what it needs cleared (the flag word) itself.  Calls that overlap in
 * time on one GPU (different streams or threads, or a graph replay beside an
 * eager call) race on the array: serialise them.  The flag word of the array
 * is not readable through moe_read_device_flags. */
#define MOE_NOALLOC_SCRATCH_BYTES (64u << 20)
moe_status moe_layer_forward_noalloc(const moe_shape* shape, const void* x, const void* w_router,
                                     const float* router_bias, const int32_t* k_per_token,
                                     const void* w_gate, const void* w_up, const void* w_down,
                                     const void* ws_gate, const void* ws_up, const void* ws_down,
                                     void* out, const moe_debug* dbg, void* stream);

/* ---- 8-bit experts (MXFP8) ---------------------------------------------
 * The pages serve the experts with FP8 quantisation and keep the router in
 * higher precision ("LLM MoE Expert Parallel production practice", deployment
 * examples; "Expert parallelism for MoE serving", FAQ on router precision);
 * they fix no scaling granularity.  The format is MXFP8 of the OCP
 * Microscaling Formats specification v1.0, whose 32-element block scales
 * CDNA4's scaled MFMA applies in hardware:
 *   - each run of 32 consecutive elements of a row (the reduction axis of the
 *     GEMM that reads it) shares one E8M0 scale byte, value 2^(byte - 127);
 *   - each element is an E4M3 byte (OCP FP8: exponent bias 7, largest finite
 *     448, no infinities, 0x7F / 0xFF NaN);
 *   - quantisation: s = floor(log2 amax) - 8, at least -127 (byte 0 for an
 *     all-zero block); element = v / 2^s rounded to the nearest E4M3 value,
 *     ties to even, saturated to +-448, sign kept (a negative value that
 *     rounds to zero is 0x80).
 * Codes are [rows][cols] bytes.  Scales "with stride S" (S >= rows): the
 * four scales of columns [128 g, 128 g + 128) of row r form 32-bit word
 * g * S + r, the block of columns [128 g + 32 i, +32) in byte i.  cols must
 * be a multiple of 128.  The MXFP8 layer keeps x and the router in bf16 for
 * routing, quantises x per token, and re-quantises h per token along I
 * inside the gate/up GEMM.  H, I and Is must be multiples of 128, act_dtype
 * MOE_BF16. */
typedef struct {
  const void* gate;            /* [E][I][H] codes                      */
  const uint8_t* gate_scales;  /* MX scales, stride E*I                */
  const void* up;              /* [E][I][H] codes                      */
  const uint8_t* up_scales;    /* stride E*I                           */
  const void* down;            /* [E][H][I] codes                      */
  const uint8_t* down_scales;  /* stride E*H                           */
} moe_mxfp8_ffn;
/* The shared expert uses the same struct with E = 1: gate/up [Is][H] (scale
 * stride Is), down [H][Is] (scale stride H). */

/* Quantises src [rows][cols] (src_dtype MOE_BF16 or MOE_F32) to MXFP8 codes
 * [rows][cols] and scales with stride scale_stride >= rows.  Inputs are
 * assumed finite (inf / NaN give unspecified codes).  Expert weights are
 * quantised once with this call (rows = E*I or E*H). */
moe_status moe_quantize_mxfp8(int32_t rows, int32_t cols, int32_t src_dtype, const void* src,
                              int32_t scale_stride, void* codes, uint8_t* scales, void* stream);

/* Weight preparation for bf16 layers: dst[i] = src[i] (bf16) as fp16, for
 * i < n (device arrays, 16-byte aligned), with the conversion the down
 * projection applies to bf16 weights inside every layer call (fp16 is the
 * down projection's operand type; exact for |w| in [2^-14, 65504]); layer
 * calls whose shape has down_dtype = MOE_F16 take the converted down weights
 * and skip that conversion, with identical results.  Down weights are
 * converted once with this call (n = E*H*I, and H*Is for the shared expert). */
moe_status moe_convert_bf16_to_f16(int64_t n, const void* src, void* dst, void* stream);

/* Workspace of the two MXFP8 calls below (host only). */
moe_status moe_workspace_size_mxfp8(const moe_shape* shape, size_t* bytes);

/* S7-S8 with MXFP8 operands: as moe_grouped_ffn, with x_perm given as MXFP8
 * codes [T*top_k][H] and scales with stride x_scale_stride >= T*top_k; the
 * dot products accumulate the decoded products in fp32; h = silu(a) * u is
 * rounded from fp32 to MXFP8 along I (blocks of 32 per row) before the down
 * projection; y_perm fp32.  A non-finite h sets
 * MOE_FLAG_H_RANGE.  Clears the workspace flag word. */
moe_status moe_grouped_ffn_mxfp8(const moe_shape* shape, const void* x_codes,
                                 const uint8_t* x_scales, int32_t x_scale_stride,
                                 const int32_t* expert_offsets, const moe_mxfp8_ffn* experts,
                                 float* y_perm, void* ws, size_t ws_bytes, void* stream);

/* The whole layer with MXFP8 experts: S1-S5 as moe_layer_forward on the bf16
 * x and router; x quantised to MXFP8 per token (timed as the gather stage:
 * it is the dispatch payload); S7-S8 as moe_grouped_ffn_mxfp8 on the
 * gathered rows; the shared expert (shape->shared_intermediate > 0, `shared`
 * then required) on the quantised x; S10 as moe_combine. */
moe_status moe_layer_forward_mxfp8(const moe_shape* shape, const void* x, const void* w_router,
                                   const float* router_bias, const int32_t* k_per_token,
                                   const moe_mxfp8_ffn* experts, const moe_mxfp8_ffn* shared,
                                   void* out, const moe_debug* dbg, void* ws, size_t ws_bytes,
                                   void* stream);

/* ---- routing with a balance bias ---------------------------------------
 * A bias per expert that evens the experts' load without touching the model's
 * mixture: it decides which experts a token takes, not how they are weighted
 * (router_bias of moe_route_topk, a part of the logits, does both).  The
 * server raises the bias of an idle expert and lowers that of a busy one
 * between batches; -inf takes an expert out of service.
 * Per token t with logits l (as moe_route_topk computes or takes them):
 *   expert e is available when select_bias[e] > -inf and l[e] is not NaN;
 *   infinite logits count as the largest finite ones;
 *   score s[e]: sigmoid(l[e]), or the softmax of l over the available experts;
 *   key = s[e] + select_bias[e];
 *   with num_groups > 1 the eligible experts are those of the topk_groups
 *   groups with the largest group score, the sum of the group's group_topn
 *   (0: 1) largest keys (of all its available experts when it has fewer);
 *   equal scores go to the lower group, a group without one is never kept;
 *   selection: the k_t available eligible experts with the largest keys,
 *   equal keys to the lower expert, in slots 0.. in that order; slots without
 *   an expert get id -1 and gate 0;
 *   gates: s of the selected experts, divided by their sum when renormalize
 *   (for a sum of 0, gates of 0), times routed_scale.
 * Keys, group scores and gates are computed in fp64; gates are rounded once.
 * Keys that are equal in fp64 are equal: the sigmoids of all logits above 36.8
 * are 1, and beside a bias of magnitude m scores less than about m * 1e-16
 * apart make one key.  select_bias [E] fp32; the other arguments as for
 * moe_route_topk.  Clears the workspace flag word. */
moe_status moe_route_biased(const moe_shape* shape, const void* x, const void* w_router,
                            const float* router_bias, const float* select_bias, const float* logits_in,
                            float* logits_out, const int32_t* k_per_token, int32_t* topk_ids,
                            float* topk_gates, void* ws, size_t ws_bytes, void* stream);

/* ---- int8 experts ------------------------------------------------------
 * Symmetric 8-bit integers with one fp32 scale per token row and one per
 * output channel of a weight (per weight row, as weights are output-major):
 *   scale = amax / 127, code = 127 v / amax rounded to nearest, ties to even
 *   (a row of zeros has scale 0 and codes 0);
 *   y[r][n] = scale_a[r] * scale_b[n] * sum_k code_a[r][k] * code_b[n][k],
 *   the sum exact in int32.
 * K is a multiple of 128 and at most 131072, N a multiple of 16 (the calls
 * with a shape: H, I and Is multiples of 128), act_dtype MOE_BF16. */

/* Quantises src [rows][cols] (MOE_BF16, MOE_F32 or MOE_F16; cols a multiple
 * of 128) to codes [rows][cols] and scales [rows].  Weights are quantised once
 * with this call (rows = E*I or E*H).  A row with an infinity or NaN gets
 * unspecified codes and a scale that is infinite or NaN (NaN for a NaN), so that
 * products of it are not finite either. */
moe_status moe_quantize_int8(int32_t rows, int32_t cols, int32_t src_dtype, const void* src, int8_t* codes,
                             float* scales, void* stream);

/* Grouped product: for every expert e and row r in [expert_offsets[e],
 * expert_offsets[e+1]), y[r] = a[r] . b[e]^T as above, in y_dtype (MOE_F32,
 * MOE_F16 or MOE_BF16).  a [rows][k] codes, b [num_experts][n][k] codes with
 * scales [num_experts][n], y [rows][n].  expert_offsets [num_experts + 1] as
 * moe_dispatch writes them, expert_offsets[num_experts] <= rows; NULL with
 * num_experts == 1 for all rows.  Rows at or beyond
 * expert_offsets[num_experts] are neither read nor written.  An fp16 y out of
 * range sets MOE_FLAG_Y_RANGE in the workspace flag word (and is infinite).
 * Fewer rows can need the larger workspace (a split of k over partial sums):
 * a caller of several sizes takes the largest of their workspaces, here as for
 * the calls with a shape. */
moe_status moe_workspace_size_gemm_int8(int32_t rows, int32_t n, int32_t k, int32_t num_experts, size_t* bytes);
moe_status moe_grouped_gemm_int8(int32_t rows, int32_t n, int32_t k, int32_t num_experts, const int8_t* a,
                                 const float* a_scales, const int32_t* expert_offsets, const int8_t* b,
                                 const float* b_scales, int32_t y_dtype, void* y, void* ws, size_t ws_bytes,
                                 void* stream);

typedef struct {
  const int8_t* gate;        /* [E][I][H] codes  */
  const float* gate_scales;  /* [E][I]           */
  const int8_t* up;          /* [E][I][H] codes  */
  const float* up_scales;    /* [E][I]           */
  const int8_t* down;        /* [E][H][I] codes  */
  const float* down_scales;  /* [E][H]           */
} moe_int8_ffn;
/* The shared expert uses the same struct with E = 1. */

/* Workspace of moe_grouped_ffn_int8 and moe_block_forward_int8. */
moe_status moe_workspace_size_int8(const moe_shape* shape, size_t* bytes);

/* S7-S8 with int8 operands: as moe_grouped_ffn, with x_perm given as codes
 * [T*top_k][H] and scales [T*top_k]; h = silu(a) * u (fp32) is rounded to fp16
 * -- values outside its range are clamped to it and set MOE_FLAG_H_RANGE -- and
 * quantised per row before the down projection; a NaN in a row of h, as a NaN
 * scale leaves it, sets the flag and makes the y row NaN.  y_perm in y_dtype
 * (MOE_F32, or MOE_F16 or MOE_BF16; an fp16 value out of range sets
 * MOE_FLAG_Y_RANGE).  Clears the workspace flag word. */
moe_status moe_grouped_ffn_int8(const moe_shape* shape, const int8_t* x_codes, const float* x_scales,
                                const int32_t* expert_offsets, const moe_int8_ffn* experts, int32_t y_dtype,
                                void* y_perm, void* ws, size_t ws_bytes, void* stream);

/* ---- experts on 8-bit floating-point blocks of 128 ------------------------
 * E4M3 codes (OCP FP8: largest finite 448, no infinities, 0x7F / 0xFF NaN) with
 * one fp32 scale per block: 128 consecutive elements of a row along the axis the
 * product sums over, 128 x 128 elements of a weight (N x K; the last block of N
 * may be short):
 *   scale = amax / 448, code = 448 v / amax rounded to the nearest E4M3 value,
 *   ties to even (a block of zeros has scale 0 and codes 0);
 *   y[r][n] = sum over blocks b of scale_a[r][b] * scale_b[n / 128][b] *
 *             sum over k in b of code_a[r][k] * code_b[n][k].
 * Row codes [rows][K], scales [rows][K / 128]; weight codes [E][N][K], scales
 * [E][ceil(N / 128)][K / 128].  K is a multiple of 128 and at most 2^20, N a multiple
 * of 16 (the calls with a shape: H and I multiples of 128, act_dtype MOE_BF16).
 * The matrix units add the products of a group of codes after aligning them to
 * the largest one, dropping what lies below about 2^-13 of it; the groups' sums
 * go on in fp32.  Sums of codes of rounded normal values are off by 1.4e-5 of
 * their norm for that (measured), far below half a step of the 16-bit types
 * (fp16 2^-11, bf16 2^-8), so the products are written in those: y_dtype is
 * MOE_F16 or MOE_BF16, MOE_F32 is MOE_ERR_UNSUPPORTED.
 * Scales are not negative (the sign of one is unspecified in a product).
 * The rows' buffers of a call with no rows may be NULL.
 * A block with an infinity or NaN gets unspecified codes and a scale that is not
 * finite (NaN for a NaN); a row of a product with such a scale, or with a NaN
 * code, is NaN, as is a column of such a weight block.  A scale
 * below fp32's normal range (2^-126; 0 among them) may count as any number up to
 * that. */

/* Quantises rows src [rows][cols] (MOE_BF16, MOE_F32 or MOE_F16; cols a multiple
 * of 128). */
moe_status moe_quantize_fp8(int32_t rows, int32_t cols, int32_t src_dtype, const void* src, void* codes,
                            float* scales, void* stream);

/* Quantises weights src [num_experts][n][k] by 128 x 128 blocks, once.  The
 * gradient with respect to a product's rows is a product with the transposed
 * weights: where n is a multiple of 128, their codes and scales are these,
 * transposed. */
moe_status moe_quantize_fp8_weights(int32_t num_experts, int32_t n, int32_t k, int32_t src_dtype, const void* src,
                                    void* codes, float* scales, void* stream);

/* Grouped product: for every expert e and row r in [expert_offsets[e],
 * expert_offsets[e+1]), y[r] = a[r] . b[e]^T as above, rounded once to y_dtype.
 * y [rows][n].  expert_offsets [num_experts + 1] as moe_dispatch writes them,
 * expert_offsets[num_experts] <= rows; NULL with num_experts == 1 for all rows.
 * Rows at or beyond expert_offsets[num_experts] are neither read nor written.  An
 * fp16 y out of range sets MOE_FLAG_Y_RANGE in the workspace flag word (and is
 * infinite).  Fewer rows can need the larger workspace: a caller of several sizes
 * takes the largest of their workspaces, here as for the FFN. */
moe_status moe_workspace_size_gemm_fp8(int32_t rows, int32_t n, int32_t k, int32_t num_experts, size_t* bytes);
moe_status moe_grouped_gemm_fp8(int32_t rows, int32_t n, int32_t k, int32_t num_experts, const void* a,
                                const float* a_scales, const int32_t* expert_offsets, const void* b,
                                const float* b_scales, int32_t y_dtype, void* y, void* ws, size_t ws_bytes,
                                void* stream);

typedef struct {
  const void* gate;          /* [E][I][H] codes               */
  const float* gate_scales;  /* [E][I / 128][H / 128]         */
  const void* up;            /* [E][I][H] codes               */
  const float* up_scales;    /* [E][I / 128][H / 128]         */
  const void* down;          /* [E][H][I] codes               */
  const float* down_scales;  /* [E][H / 128][I / 128]         */
} moe_fp8_ffn;

/* S7-S8 on such operands: as moe_grouped_ffn, with x_perm given as codes
 * [T*top_k][H] and scales [T*top_k][H / 128]; h = silu(a) * u in fp32 is quantised
 * per row and block of 128 columns before the down projection (an h that is not
 * finite sets MOE_FLAG_H_RANGE, and its y row is NaN); y_perm in y_dtype (an fp16
 * value out of range sets MOE_FLAG_Y_RANGE).  Clears the workspace flag word.
 * silu of a gate below -87.3, less than 1.1e-36 in magnitude, counts as 0.
 * Few rows multiply the codes of gate and up as fp16 values and sum in fp32, more
 * rows take the 8-bit units, whose sums are off by some 1e-5 (above), and the
 * quotient 448 h / amax may be off by an fp32 rounding or two: an h that near to the
 * middle between two codes can take either.  So the codes of a row's h, each half a step
 * of its value from h either way, can differ with the number of rows of the call
 * (2-norm error of y against exact sums 1.7e-3 with few rows of normal data, bf16's own
 * rounding, and 1.9e-3 to 2.1e-3 with many); for the same call they are always
 * the same. */
moe_status moe_workspace_size_fp8(const moe_shape* shape, size_t* bytes);
moe_status moe_grouped_ffn_fp8(const moe_shape* shape, const void* x_codes, const float* x_scales,
                               const int32_t* expert_offsets, const moe_fp8_ffn* experts, int32_t y_dtype,
                               void* y_perm, void* ws, size_t ws_bytes, void* stream);

/* ---- rows to expert order, and the gradients of dispatch and combine --------
 * For rows of any type (MOE_F32, MOE_BF16 or MOE_F16; H a multiple of 8, of 4 when
 * every row of the call is fp32; num_tokens, hidden and top_k are all that these calls
 * take from their shape, whose other fields may be anything) given the permutation
 * that moe_dispatch leaves in row_of_slot [T][top_k]; entries outside [0,
 * num_rows) are slots without a row, the others are distinct.  num_rows is the
 * rows that the permuted buffers hold (0: they may be NULL; with no tokens every
 * buffer may).  Sums in fp32, in slot order, rounded once;
 * no workspace. */

/* x_perm[row_of_slot[t][j]] = weights[t][j] * x[t] (weights [T][top_k] fp32, NULL:
 * 1).  Rows that no slot names are left as they were. */
moe_status moe_dispatch_rows(const moe_shape* shape, int32_t dtype, const void* x, const int32_t* row_of_slot,
                             const float* weights, int32_t num_rows, void* x_perm, void* stream);

/* The same rows, unweighted, as the codes [num_rows][H] and scales [num_rows][H /
 * 128] that moe_quantize_fp8 makes of x[t]: the input of moe_grouped_ffn_fp8 and
 * moe_grouped_gemm_fp8.  H a multiple of 128; x in dtype. */
moe_status moe_dispatch_rows_fp8(const moe_shape* shape, int32_t dtype, const void* x, const int32_t* row_of_slot,
                                 int32_t num_rows, void* x_codes, float* x_scales, void* stream);

/* The gradient of moe_dispatch_rows (and, without weights, of moe_dispatch's
 * x_perm) from that of x_perm:
 *   d_x[t]          = sum over j with a row of weights[t][j] * d_perm[row]     [T][H]
 *   d_weights[t][j] = <d_perm[row], x[t]>, 0 for a slot without a row  [T][top_k] fp32
 * weights NULL: 1, and d_weights NULL.  d_x may be NULL when d_weights is not; x is
 * read only for d_weights (else it may be NULL). */
moe_status moe_dispatch_rows_backward(const moe_shape* shape, int32_t dtype, const void* d_perm,
                                      const int32_t* row_of_slot, int32_t num_rows, const float* weights,
                                      const void* x, void* d_x, float* d_weights, void* stream);

/* The gradient of moe_combine (and of the sum inside moe_combine_norm) from that
 * of its output, d_out [T][H] in out_dtype (which is also y_shared's gradient):
 *   d_y[row_of_slot[t][j]] = topk_gates[t][j] * d_out[t]        [num_rows][H] in y_dtype
 *   d_gates[t][j] = <d_out[t], y_perm[row]>, 0 for a slot without a row  [T][top_k] fp32
 * Rows of d_y that no slot names are left as they were.  d_y or d_gates may be NULL,
 * not both; y_perm [num_rows][H] in y_dtype is read only for d_gates (else it may be
 * NULL) and may be d_y itself. */
moe_status moe_combine_backward(const moe_shape* shape, int32_t out_dtype, const void* d_out, int32_t y_dtype,
                                const void* y_perm, const int32_t* row_of_slot, const float* topk_gates,
                                int32_t num_rows, void* d_y, float* d_gates, void* stream);

/* ---- the block around the layer ----------------------------------------
 * A transformer block's FFN half with the layer in it:
 *   n = norm(x; pre_norm),  y = layer(n),
 *   out = residual_scale * x + gate * norm(y; post_norm),
 *   norm(v; w) = v / sqrt(mean(v^2) + eps) * w   (over the H columns).
 * Sums and products in fp32, one rounding on each output. */
typedef struct {
  const float* select_bias;  /* [E]: routing as moe_route_biased; NULL: as moe_route_topk      */
  const float* pre_norm;     /* [H] fp32; NULL: the layer takes x itself                       */
  const float* post_norm;    /* [H] fp32; NULL: y is not normed                                */
  float eps;                 /* > 0, both norms                                                */
  float residual_scale;      /* finite; 0: x is not added                                      */
  const void* gate;          /* gate value of token t, column c at element
                                t * gate_row_stride + c * gate_col_stride; NULL: 1             */
  int64_t gate_row_stride;   /* >= 0; 0: the same for all tokens                               */
  int32_t gate_col_stride;   /* 0 (one value per token) or 1                                   */
  int32_t gate_dtype;        /* MOE_F32 or MOE_BF16                                            */
  int32_t stream_dtype;      /* MOE_F32 or MOE_BF16: x (the residual stream) and out           */
} moe_block;
/* The gate is 4-byte (fp32) or 2-byte (bf16) aligned; with column stride 1 its
 * rows may start anywhere at that alignment. */

/* The norm in front of the layer, with the quantisation the int8 experts want:
 * n = norm(x) of rows [rows][cols] (src_dtype MOE_F32 or MOE_BF16; cols a
 * multiple of 64, of 4 when src and out are fp32, of 128 with codes); out
 * (nullable) in out_dtype (MOE_F32 or MOE_BF16); codes and scales (both or
 * neither) quantise the unrounded n as moe_quantize_int8 does (a row of x with
 * an infinity or NaN gets the scale NaN).  weight [cols] fp32 or NULL (1).  out
 * may be x itself when the types are the same. */
moe_status moe_norm(int32_t rows, int32_t cols, int32_t src_dtype, const void* x, const float* weight, float eps,
                    int32_t out_dtype, void* out, int8_t* codes, float* scales, void* stream);

/* S10 with the end of the block: y = the sum moe_combine forms (y_perm and
 * y_shared in y_dtype: MOE_F32, MOE_F16 or MOE_BF16; a token without a kept
 * slot has y_shared[t] or 0), out = residual_scale * residual + gate *
 * norm(y; post_norm) in stream_dtype.  residual (stream_dtype) may be NULL only
 * when residual_scale is 0, and may be out itself.  Of `block`, select_bias and
 * pre_norm are not used.  H a multiple of 8 unless y_dtype and stream_dtype are
 * MOE_F32. */
moe_status moe_combine_norm(const moe_shape* shape, const moe_block* block, int32_t y_dtype, const void* y_perm,
                            const int32_t* row_of_slot, const float* topk_gates, const void* y_shared,
                            const void* residual, void* out, void* stream);

/* The block in one call: moe_norm, routing (moe_route_biased with a
 * select_bias, else moe_route_topk), moe_dispatch, moe_grouped_ffn,
 * moe_combine_norm.  x and out [T][H] in block->stream_dtype (which has to be
 * act_dtype when pre_norm is NULL); out may be x itself.  shape->out_dtype is
 * not used.  The other arguments as for moe_layer_forward; `dbg` stages: the
 * norm in front is outside every stage.  moe_workspace_size_block gives the
 * workspace. */
moe_status moe_workspace_size_block(const moe_shape* shape, size_t* bytes);
moe_status moe_block_forward(const moe_shape* shape, const moe_block* block, const void* x, const void* w_router,
                             const float* router_bias, const int32_t* k_per_token, const void* w_gate,
                             const void* w_up, const void* w_down, const void* ws_gate, const void* ws_up,
                             const void* ws_down, void* out, const moe_debug* dbg, void* ws, size_t ws_bytes,
                             void* stream);

/* The same with int8 experts and, when shape->shared_intermediate > 0, an int8
 * shared expert: the norm in front also quantises its rows (without one, x is
 * quantised: the gather stage). */
moe_status moe_block_forward_int8(const moe_shape* shape, const moe_block* block, const void* x,
                                  const void* w_router, const float* router_bias, const int32_t* k_per_token,
                                  const moe_int8_ffn* experts, const moe_int8_ffn* shared, void* out,
                                  const moe_debug* dbg, void* ws, size_t ws_bytes, void* stream);

/* The fp32 logistic function that group-limited routing sums into group
 * scores, evaluated elementwise: y[i] = sigma(x[i]) for i < n (device
 * arrays).  Node-limited routing ("Expert parallelism for MoE serving",
 * deployment examples) ranks groups by these sums, so the selected groups
 * depend on every bit of them; this entry point lets a checker compare those
 * bits with an independent implementation of the same operation sequence:
 * clamp to [-30, 30]; n = rint(-x * fp32(log2 e)); r = fma(-n, ln2_hi, -x),
 * r = fma(-n, ln2_lo, r) with ln2_hi = ln 2 to 17 significant bits and
 * ln2_lo = fp32(ln 2 - ln2_hi); p = degree-7 Taylor polynomial of e^r with
 * coefficients fp32(1/i!) in Horner form with fma; e = ldexp(p, n);
 * sigma = 1 / (1 + e); IEEE fp32 operations rounded to nearest even. */
moe_status moe_group_score_sigmoid(const float* x, float* y, int64_t n, void* stream);

/* Static text for a status code. */
const char* moe_status_string(moe_status status);

/* hipError_t of the last failed HIP call on this thread (0 if none). */
int32_t moe_last_hip_error(void);

/* Copies the workspace flag word to *flags and waits for it (synchronises the
 * stream).  For tests and diagnostics. */
moe_status moe_read_device_flags(const void* ws, void* stream, uint32_t* flags);

#ifdef __cplusplus
}
#endif
#endif /* MOE_MI355X_H */
