/*
 * gbmoe.h -- C ABI of the GB300 (sm_103a) fused Mixture-of-Experts layer.
 *
 * The layer (one sparse FFN of a MoE transformer) as the serving pages state
 * it (Xeon 6 / SGLang DeepSeek-R1 blog, section "MoE"; SGLang CPU backend
 * write-up, section "(3) FusedMoE"):
 *
 *   1. routing alignment: argsort the flat topk_ids so that the (token, slot)
 *      pairs of each expert are contiguous, pad every expert's group to a
 *      multiple of a block size and record the expert of every block;
 *   2. GEMM1 in the A x [B1, B2] = [C1, C2] form, W13 = [gate; up], with
 *      h = SiLU(C1) * C2 computed in the epilogue;
 *   3. GEMM2, the down projection y = h x W2^T;
 *   4. the weighted combine out[t] = sum_k topk_weights[t,k] * y[t,k].
 *
 * Weights are FP8 E4M3 with one fp32 scale per 128x128 block (DeepSeek-style
 * block quantisation), INT8 with one fp32 scale per output channel and
 * dynamic per-row INT8 activations (DA8W8), or INT4 with one fp32 scale per
 * row and 128 columns.  Weights stay in their stored format in HBM and are
 * expanded in registers or shared memory.
 *
 * Conventions shared by every entry point
 *  - All data pointers are DEVICE pointers owned by the caller.  The library
 *    allocates no memory and never synchronises the stream, except
 *    the readers of status words (moe_read_status, moe_read_tree_status,
 *    moe_read_static_scratch_status), which wait for the stream.
 *  - Every call is enqueued on `stream` (a cudaStream_t; NULL = the legacy
 *    default stream) and is ordered with the caller's other work on it.
 *  - Matrices are row-major and contiguous.
 *  - Host-checkable errors (bad sizes, NULL pointers, short workspace) are
 *    returned before anything is launched.  A failed launch returns
 *    MOE_ERR_CUDA.  Conditions only the GPU can see (expert ids outside
 *    [0, E)) are counted in a status word inside the workspace; read it with
 *    moe_read_status (tree attention: moe_read_tree_status).
 *  - A flat slot index is i = t * topk + k for token t and top-k column k.
 *  - Calls that share a workspace must not overlap on the GPU.
 */
#ifndef GBMOE_H
#define GBMOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* moe_stream_t; /* the same type as cudaStream_t */

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1, /* a size or pointer argument is invalid            */
  MOE_ERR_UNSUPPORTED = 2, /* valid, but outside what the kernels implement    */
  MOE_ERR_WORKSPACE = 3,   /* workspace NULL, misaligned or smaller than asked */
  MOE_ERR_CUDA = 4,        /* a CUDA runtime call or kernel launch failed      */
  MOE_ERR_TIMEOUT = 5,     /* a bounded device-side wait gave up               */
  MOE_ERR_BAD_IDS = 6      /* the device saw expert ids outside [0, E), or tree attention lengths,
                              offsets or cache pages out of range              */
} moe_status_t;

/* flags of fused_moe_fp8 / fused_moe_int8 / fused_moe_int4 / fused_moe_gated */
#define MOE_PATH_AUTO 0x0u    /* decode below MOE_AUTO_PREFILL_TOKENS tokens (INT4: up to
                                 MOE_MAX_DECODE_TOKENS), else prefill                 */
#define MOE_PATH_DECODE 0x1u  /* weight-streaming GEMV path (small token counts)    */
#define MOE_PATH_PREFILL 0x2u /* tcgen05 grouped-GEMM path (large token counts)     */
#define MOE_PATH_MASK 0x3u
/* fused_moe_fp8 only: FP8 x FP8 products.  x and the intermediate h are
 * quantised to E4M3 in groups of 1 x 128 (one fp32 scale per row and 128
 * columns, as moe_quant_act_fp8 does) before they enter the tensor cores.
 * Runs on the tcgen05 path at every M; MOE_PATH_DECODE with it is
 * MOE_ERR_UNSUPPORTED. */
#define MOE_ACT_FP8_1X128 0x10u

#define MOE_WEIGHT_FP8 0
#define MOE_WEIGHT_INT8 1
#define MOE_WEIGHT_INT4 2

/* Limits of this implementation (larger sizes return MOE_ERR_UNSUPPORTED). */
#define MOE_MAX_EXPERTS 1024
#define MOE_MAX_DECODE_TOKENS 128 /* MOE_PATH_DECODE handles M <= this */
#define MOE_AUTO_PREFILL_TOKENS 128 /* MOE_PATH_AUTO takes the tcgen05 path from this many tokens */

/*
 * Capacity (entries) of sorted_ids for the given routing problem:
 * M*topk + E*(block_size-1), rounded up to a multiple of block_size.  Every
 * expert may waste at most block_size-1 padding slots.  Returns 0 for
 * invalid arguments.
 */
size_t moe_align_max_padded(int M, int topk, int num_experts, int block_size);

/*
 * Routing alignment ("moe_align_index"): the argsort of topk_ids by expert,
 * blocked per expert (SGLang CPU backend write-up, section "(3) FusedMoE",
 * the moe_align_index and thread-offset paragraphs; Xeon 6 / SGLang blog,
 * section "MoE").
 *
 *   topk_ids        int32 [M, topk]   expert chosen by each (token, slot)
 *   sorted_ids      int32 [cap]       out: flat slot indices grouped by
 *                                     expert (ascending), ascending slot
 *                                     order inside an expert, each group
 *                                     padded to a multiple of block_size
 *                                     with the sentinel M*topk; the tail
 *                                     past the last group is sentinel too
 *   expert_ids      int32 [cap/block_size]  out: expert of each block, -1
 *                                     for blocks past the last group
 *   num_tokens_post_padded int32 [1]  out: sum of the padded group sizes
 *   expert_offsets  int32 [E+1]       out: start of each expert's group in
 *                                     sorted_ids (exclusive prefix sum)
 * cap = moe_align_max_padded(M, topk, E, block_size).  Slots whose id lies
 * outside [0, E) are left out (as a non-local expert would be).  Experts
 * with no slot get no block.  1 <= block_size <= 256, E <= MOE_MAX_EXPERTS.
 * The result is deterministic and equals a stable argsort bit for bit.
 */
moe_status_t moe_align_block_size(const int32_t* topk_ids, int M, int topk, int num_experts,
                                  int block_size, int32_t* sorted_ids, int32_t* expert_ids,
                                  int32_t* num_tokens_post_padded, int32_t* expert_offsets,
                                  moe_stream_t stream);

/*
 * Router gating: each token's experts and routing weights from its router
 * logits.  The pages take topk_ids / topk_weights as the router's given
 * output; the two gating functions here are those of the model
 * configurations the layer serves (softmax top-k as in Qwen3-MoE, and the
 * DeepSeek-V3/R1 sigmoid router with group-limited selection).  Equal scores
 * go to the lower expert index.
 *
 *  MOE_GATE_SOFTMAX: p = softmax(logits[t]); topk_ids[t] = the topk largest p
 *    in descending order; topk_weights[t,j] = p_j / (sum of the chosen p).
 *    Ranking p is ranking the logits, so only the chosen terms are formed:
 *    w_j = exp(l_j - l_max) / sum over chosen of exp(l_i - l_max).
 *  MOE_GATE_SIGMOID_GROUPED: s = sigmoid(logits[t]) and b = s + bias (the
 *    bias only ranks).  The E experts form n_group consecutive groups of
 *    E / n_group; a group's score is the sum of its two largest b (its only b
 *    in a group of one); the topk_group best groups are kept and
 *    topk_ids[t] = the topk largest b inside them, descending;
 *    topk_weights[t,j] = s_j / (sum of the chosen s) * routed_scaling.
 * Arithmetic is fp32 (expf, IEEE division); rankings compare fp32 scores, so
 * scores closer than a few fp32 ulps may rank either way.  Whatever the
 * logits (NaN included), every written id lies in [0, E).
 */
#define MOE_GATE_SOFTMAX 0
#define MOE_GATE_SIGMOID_GROUPED 1
typedef struct moe_gate_config {
  int scoring;          /* MOE_GATE_SOFTMAX or MOE_GATE_SIGMOID_GROUPED                      */
  int n_group;          /* SIGMOID_GROUPED: 1..32, divides E.  SOFTMAX: must be 1              */
  int topk_group;       /* SIGMOID_GROUPED: 1..n_group, topk <= topk_group * E / n_group.
                           SOFTMAX: must be 1                                                  */
  float routed_scaling; /* SIGMOID_GROUPED: > 0.  SOFTMAX: must be 1.0                         */
  const float* bias;    /* SIGMOID_GROUPED: fp32 [E] device pointer, or NULL for none.
                           SOFTMAX: must be NULL                                               */
  int shared_expert;    /* 0 or 1: also write column topk of every row as (id E, weight 1.0)   */
} moe_gate_config_t;

/*
 *   logits        fp32 [M, E]                     router logits
 *   topk_ids      int32 [M, topk + shared_expert] out
 *   topk_weights  fp32  [M, topk + shared_expert] out
 * 1 <= topk <= min(E, 32), E <= MOE_MAX_EXPERTS, M >= 0.  One warp ranks one
 * token.  Launched with programmatic dependent launch: the kernel waits for
 * the stream's previous kernel before it reads or writes anything, and the
 * next kernel of the library may be scheduled while it runs.
 */
moe_status_t moe_gate_topk(const float* logits, int M, int E, int topk, const moe_gate_config_t* gate,
                           int32_t* topk_ids, float* topk_weights, moe_stream_t stream);

/*
 * Dynamic per-row INT8 quantisation of bf16 activations (the DA8W8
 * activation side; SGLang CPU backend write-up, section "(3) FusedMoE", the
 * dynamic-quant fusion paragraph):
 *   scale[r] = max_c |x[r,c]| / 127 (fp32; 1 for an all-zero row)
 *   q[r,c]   = round-half-even(x[r,c] / scale[r]) (IEEE fp32 division),
 *              clamped to [-127, 127]
 *   x bf16 [M, H] -> q int8 [M, H], scale fp32 [M].  M >= 0, 1 <= H.
 * The fused INT8 layer applies exactly this function to its input rows.
 */
moe_status_t moe_quant_act_int8(const void* x_bf16, int M, int H, int8_t* q, float* scale,
                                moe_stream_t stream);

/*
 * Dynamic FP8 quantisation of bf16 activations in groups of 1 x 128 (the
 * activation side of MOE_ACT_FP8_1X128).  The pages keep FP8-weight
 * activations in BF16 (Xeon 6 / SGLang blog, section "FP8 inference"); this
 * is the FP8 x FP8 form of the grouped GEMMs named in the news rewrite of the
 * LMSYS large-scale-EP blog (section "DeepGEMM integration"), with the group
 * along H matching the weights' 128-wide scale blocks:
 *   scale[r,g] = max over c in [128g, 128g+128) of |x[r,c]| / 448 (fp32; 1 for
 *                an all-zero group)
 *   q[r,c]     = E4M3(x[r,c] / scale[r, c/128]), the division in IEEE fp32,
 *                rounded to nearest even, saturated to +-448
 *   x bf16 [M, H] -> q uint8 E4M3 codes [M, H], scale fp32 [M, H/128].
 * H must be a multiple of 128 (else MOE_ERR_UNSUPPORTED); M >= 0.  x 16-byte
 * aligned, q 4-byte aligned.  The fused layer applies exactly this function
 * to its input rows.
 */
moe_status_t moe_quant_act_fp8(const void* x_bf16, int M, int H, uint8_t* q, float* scale,
                               moe_stream_t stream);

/*
 * Bytes of scratch the fused layer needs for these sizes and flags
 * (weight_kind MOE_WEIGHT_FP8, MOE_WEIGHT_INT8 or MOE_WEIGHT_INT4).  The workspace must be
 * 256-byte aligned.  Returns 0 for invalid or unsupported arguments.
 */
size_t moe_workspace_size(int M, int H, int I, int E, int topk, int weight_kind,
                          unsigned flags);

/*
 * The whole MoE layer with FP8 E4M3 block-scaled weights; activations enter
 * the products at their bf16 values (weight-only FP8, as in the Xeon 6 /
 * SGLang blog, section "FP8 inference", and the SGLang CPU backend
 * write-up, section "(4) FP8 GEMM").
 *
 *   x_bf16        bf16 [M, H]
 *   topk_ids      int32 [M, topk]        ids outside [0, E) contribute 0
 *   topk_weights  fp32 [M, topk]
 *   w13_e4m3      uint8 [E, 2I, H]       rows 0..I-1 gate, I..2I-1 up
 *   w13_scale     fp32 [E, 2I/128, H/128]  W13 = decode(code) * scale of its block
 *   w2_e4m3       uint8 [E, H, I]
 *   w2_scale      fp32 [E, H/128, I/128]
 *   out_bf16      bf16 [M, H]            out[t] = sum_k w[t,k] * y[t,k]
 *   workspace     moe_workspace_size(M, H, I, E, topk, MOE_WEIGHT_FP8, flags)
 *                 bytes of device memory, 256-byte aligned
 * H and I must be multiples of 128; 1 <= topk <= 32; M >= 0 (M == 0 is a
 * no-op).  A shared expert is passed as one more expert with a top-k column
 * of weight 1.0.  The products run on tensor cores with fp16 operands and
 * fp32 accumulation; each 128x128 block scale is applied once per 128-deep
 * partial sum.  Operands keep the range of their source type: the E4M3 to
 * fp16 expansion is exact; each x row is stored as fp16 in a power-of-two
 * frame of its own (its max |x| scaled into [2^14, 2^15), so every bf16 value
 * within 2^-28 of the row's largest is exact); the intermediate h is stored
 * as fp16 in a power-of-two frame per row (values within 2^-21 of the row's
 * largest keep full fp16 precision); on the tcgen05 path the block scales
 * are folded into the fp16 weights relative to a power of two per 128-row
 * block.  The frames are taken back in fp32, so no finite input overflows an
 * fp16 operand.
 * With MOE_ACT_FP8_1X128 in flags, x is quantised as moe_quant_act_fp8 does,
 * and so is each intermediate row h (fp32, per 128 columns of I) of a
 * (token, expert) pair before the down projection; the products are E4M3 x
 * E4M3 on the tensor cores, and every 128-deep partial sum is scaled by its
 * weight block scale times its activation group scale in fp32.
 */
moe_status_t fused_moe_fp8(const void* x_bf16, const int32_t* topk_ids, const float* topk_weights,
                           const void* w13_e4m3, const float* w13_scale, const void* w2_e4m3,
                           const float* w2_scale, int M, int H, int I, int E, int topk,
                           unsigned flags, void* out_bf16, void* workspace,
                           size_t workspace_bytes, moe_stream_t stream);

/*
 * The whole MoE layer with INT8 per-output-channel weights and dynamic
 * per-row INT8 activations (DA8W8; SGLang CPU backend write-up, section
 * "(3) FusedMoE"): x rows are quantised as moe_quant_act_int8 does, and each
 * intermediate row h of a (token, expert) pair is quantised the same way
 * before the down projection.
 *
 *   w13        int8 [E, 2I, H],  w13_scale fp32 [E, 2I]
 *   w2         int8 [E, H, I],   w2_scale  fp32 [E, H]
 * other arguments as for fused_moe_fp8.  H and I must be multiples of 128.
 */
moe_status_t fused_moe_int8(const void* x_bf16, const int32_t* topk_ids, const float* topk_weights,
                            const int8_t* w13, const float* w13_scale, const int8_t* w2,
                            const float* w2_scale, int M, int H, int I, int E, int topk,
                            unsigned flags, void* out_bf16, void* workspace,
                            size_t workspace_bytes, moe_stream_t stream);

/*
 * The whole MoE layer with group-wise INT4 weights (W4A16).  The pages name
 * INT4 as the quantised alternative to native FP8 (SGLang CPU backend
 * write-up, closing section; OSDI'26 local-MoE summary, the INT4 decode
 * baseline of its evaluation) but fix no layout; this one is:
 *
 *   w13        uint8 [E, 2I, H/2]   two's-complement int4 codes in [-8, 7],
 *                                   column 2j in the low nibble of byte j,
 *                                   column 2j+1 in its high nibble
 *   w13_scale  fp32 [E, 2I, H/128]  W13[e,n,k] = q * w13_scale[e, n, k/128]
 *   w2         uint8 [E, H, I/2],   w2_scale fp32 [E, H, I/128]
 * other arguments as for fused_moe_fp8.  Activations enter the products at
 * their bf16 values (in fp16 power-of-two frames, as on the FP8 weight-only
 * path) and each 128-deep partial sum is scaled by its row's group scale in
 * fp32.
 * H and I must be multiples of 128.  Paths as for fused_moe_fp8 (the
 * weight-streaming kernels up to MOE_MAX_DECODE_TOKENS tokens, the tcgen05
 * grouped GEMMs above; MOE_PATH_DECODE is accepted at any M for INT4);
 * MOE_ACT_FP8_1X128 is MOE_ERR_INVALID_ARG.  Workspace:
 * moe_workspace_size(..., MOE_WEIGHT_INT4, flags).
 */
moe_status_t fused_moe_int4(const void* x_bf16, const int32_t* topk_ids, const float* topk_weights,
                            const uint8_t* w13, const float* w13_scale, const uint8_t* w2,
                            const float* w2_scale, int M, int H, int I, int E, int topk,
                            unsigned flags, void* out_bf16, void* workspace,
                            size_t workspace_bytes, moe_stream_t stream);

/*
 * The experts of the layer on the masked, fixed-capacity layout of
 * expert-parallel low-latency dispatch (the "masked" grouped GEMM of the
 * DeepGEMM integration in the news rewrite of the LMSYS large-scale-EP blog,
 * section "DeepGEMM集成"): tokens arrive already grouped by expert, each expert
 * holding up to `cap` rows, and only a device-side count says how many are real.
 * Nothing in the call depends on host knowledge of the counts, so it can be
 * captured in a CUDA graph and replayed with new counts.
 *
 *   x_bf16     bf16 [E, cap, H]   row (e, i) is the i-th token sent to expert e
 *   masked_m   int32 [E]          rows held by expert e (device memory, read by
 *                                 the kernels); values are clamped to [0, cap]
 *   w13, w2 (+ scales)            as for fused_moe_fp8 (weight_kind
 *                                 MOE_WEIGHT_FP8) or fused_moe_int4
 *                                 (MOE_WEIGHT_INT4); MOE_WEIGHT_INT8 is
 *                                 MOE_ERR_UNSUPPORTED
 *   out_bf16   bf16 [E, cap, H]   out[e, i] = W2_e (SiLU(W1_e x) * (W3_e x)) for
 *                                 i < masked_m[e]; rows past the count are left
 *                                 untouched.  No routing weight is applied (the
 *                                 combine of the dispatch applies it).
 *   workspace  moe_workspace_size_masked(E, cap, H, I, weight_kind) bytes,
 *              256-byte aligned
 * x, w13 and w2 16-byte aligned; out_bf16 2-byte aligned, 16-byte aligned
 * with MOE_PATH_PREFILL (else MOE_ERR_INVALID_ARG).  H and I multiples of 128, E <= MOE_MAX_EXPERTS, cap >= 1.  The products
 * use the arithmetic of the weight kind's layer entry point.  Since the counts
 * are on the device the caller picks the kernels: MOE_PATH_AUTO or
 * MOE_PATH_DECODE runs the weight-streaming kernels (best for a few rows per
 * expert); MOE_PATH_PREFILL runs the tcgen05 kernels (best for many rows per
 * expert).  Every kernel of the call is enqueued on `stream`.
 */
size_t moe_workspace_size_masked(int E, int cap, int H, int I, int weight_kind);
moe_status_t fused_moe_masked(int weight_kind, const void* x_bf16, const int32_t* masked_m, const void* w13,
                              const float* w13_scale, const void* w2, const float* w2_scale, int E, int cap,
                              int H, int I, unsigned flags, void* out_bf16, void* workspace,
                              size_t workspace_bytes, moe_stream_t stream);

/*
 * The whole layer from router logits: moe_gate_topk, then fused_moe_fp8
 * (weight_kind MOE_WEIGHT_FP8), fused_moe_int8 (MOE_WEIGHT_INT8) or
 * fused_moe_int4 (MOE_WEIGHT_INT4) on its result, with no host step between
 * them.
 *
 *   router_logits  fp32 [M, E]   E = routed experts
 *   gate           gating function and options, as for moe_gate_topk
 *   w13, w2 (+ scales)  hold E + gate->shared_expert experts; a shared
 *                  expert is the last one
 *   topk_ids, topk_weights  out, [M, topk + gate->shared_expert], as
 *                  moe_gate_topk writes them (the routing the layer used)
 *   workspace      moe_workspace_size(M, H, I, E + shared_expert,
 *                  topk + shared_expert, weight_kind, flags) bytes
 * other arguments as for fused_moe_fp8 / _int8 / _int4 (flags must suit the
 * weight kind).  When M <= MOE_GATE_INLINE_TOKENS and E <= 256 the ranking
 * runs inside the layer's first kernel, ahead of the routing alignment (one
 * launch fewer); otherwise it is one more launch, chained to the layer by
 * programmatic dependent launch.  Results are the same either way.
 */
#define MOE_GATE_INLINE_TOKENS 64
moe_status_t fused_moe_gated(int weight_kind, const void* x_bf16, const float* router_logits,
                             const moe_gate_config_t* gate, const void* w13, const float* w13_scale,
                             const void* w2, const float* w2_scale, int M, int H, int I, int E, int topk,
                             unsigned flags, int32_t* topk_ids, float* topk_weights, void* out_bf16,
                             void* workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * fused_moe_fp8 for callers that cannot allocate device memory.  The pages
 * have no counterpart of this entry point; it exists for callers that hold
 * only raw input and output pointers and may not call a device allocator (a
 * plugin whose host framework owns all device memory, a C caller without an
 * allocator, or a loop that must not pay for cudaMalloc / cudaFree).
 *
 * Same arguments, layouts and results as fused_moe_fp8, without the
 * workspace: the scratch is a static device buffer of
 * MOE_STATIC_SCRATCH_BYTES inside the library.  Each device on which it runs
 * holds that buffer from its first call until the process exits.
 *  - The first call on a device looks the buffer's address up
 *    (cudaGetSymbolAddress) with that device current; make that first call
 *    before any stream capture.  After a device reset the next call on that
 *    device looks it up again (a new CUDA context), so it too must come
 *    before any capture.
 *  - Invalid arguments return what fused_moe_fp8 returns for them.  Valid
 *    sizes whose moe_workspace_size(..., MOE_WEIGHT_FP8, flags) exceeds
 *    MOE_STATIC_SCRATCH_BYTES return MOE_ERR_UNSUPPORTED with a message that
 *    names the limit; nothing is launched.
 *  - Nothing is allocated or freed.  All calls share the buffer, which keeps
 *    the last call's contents; the kernels clear what must start at zero.
 *    Calls that overlap on the GPU race on it: serialise them.
 *  - Its device status words (ids out of range, a bounded wait that gave up)
 *    are read with moe_read_static_scratch_status.
 */
#define MOE_STATIC_SCRATCH_BYTES (16u << 20)
moe_status_t fused_moe_fp8_static_scratch(const void* x_bf16, const int32_t* topk_ids,
                                          const float* topk_weights, const void* w13_e4m3,
                                          const float* w13_scale, const void* w2_e4m3,
                                          const float* w2_scale, int M, int H, int I, int E, int topk,
                                          unsigned flags, void* out_bf16, moe_stream_t stream);

/*
 * moe_read_status for the static buffer of fused_moe_fp8_static_scratch on
 * the current device: waits for `stream`, then copies the status words of
 * the last call that ran there (see moe_read_status).  The pages have no
 * counterpart of this function either.
 */
moe_status_t moe_read_static_scratch_status(int32_t status_out[2], moe_stream_t stream);

/*
 * Waits for `stream`, then copies the workspace's status words to the host:
 *   status_out[0] = number of topk_ids entries outside [0, E) seen by the
 *                   last fused call on this workspace
 *   status_out[1] = bit set of device conditions (1 = a bounded wait gave up)
 * Returns MOE_ERR_BAD_IDS / MOE_ERR_TIMEOUT when they are non-zero.
 */
moe_status_t moe_read_status(const void* workspace, int32_t status_out[2], moe_stream_t stream);

/*
 * The routing alignment (step 1) that the last routed fused call on
 * `workspace` computed -- fused_moe_fp8, fused_moe_int8, fused_moe_int4 or
 * fused_moe_gated, called with these same M, H, I, E (all stored experts),
 * topk (all columns) and flags.  Outputs are as moe_align_block_size defines
 * them, for the block size the layer chose for its path (8 on the
 * weight-streaming kernels, 16 on the tcgen05 ones):
 *   block_size      HOST int out (may be NULL)
 *   sorted_ids      device int32 [moe_align_max_padded(M, topk, E, *block_size)]
 *   expert_ids      device int32 [that / *block_size]
 *   num_tokens_post_padded  device int32 [1]
 *   expert_offsets  device int32 [E + 1]
 * Any output pointer may be NULL (block_size alone answers the sizing
 * question).  The copies are stream-ordered device-to-device copies after
 * the layer's kernels; nothing synchronises.  The masked layout has no
 * alignment and is not covered.  Bad sizes give MOE_ERR_INVALID_ARG.
 */
moe_status_t moe_read_routing(const void* workspace, int M, int H, int I, int E, int topk, int weight_kind,
                              unsigned flags, int* block_size, int32_t* sorted_ids, int32_t* expert_ids,
                              int32_t* num_tokens_post_padded, int32_t* expert_offsets, moe_stream_t stream);

/*
 * Self-test of the failure path of the bounded device waits.  Launches one
 * small kernel whose waits can never complete: one gives up after
 * limit_cycles SM clocks (1000 <= limit_cycles <= 2^31, about a second at
 * most), sets bit 0 of the workspace's status words and the shared abort
 * flag; the other leaves through that flag, as every role of a GEMM kernel
 * does when one of them times out.  *gave_up (device int32) receives the
 * number of waits that gave up (2).  moe_read_status(workspace) then returns
 * MOE_ERR_TIMEOUT.  Only the status words (the first 8 bytes of any
 * workspace, at least 256 bytes, 256-byte aligned) and *gave_up are written;
 * nothing faults and the context stays usable.
 */
moe_status_t moe_selftest_wait_timeout(void* workspace, long long limit_cycles, int32_t* gave_up,
                                       moe_stream_t stream);

/*
 * Per-kernel timing of fused calls on the calling host thread (a profiling
 * aid; it changes nothing the layer computes).
 *
 * moe_profile_enable(max_calls): with max_calls > 0, creates CUDA timing
 * events on the current device for up to max_calls later fused calls and
 * starts recording: every such call records one event before its first
 * kernel and one after each kernel, on its own stream.  max_calls == 0 stops
 * recording and releases the events.  Calls past the limit are not recorded.
 *
 * moe_profile_read(stage_ms, stage_names, max_stages, n_stages, n_calls):
 * waits for the recorded events, writes per kernel ("stage") the summed
 * milliseconds over all recorded calls (stage order = launch order; all
 * recorded calls must have taken the same path) and the stage's name, then
 * forgets the recorded calls (recording continues).
 */
moe_status_t moe_profile_enable(int max_calls);
moe_status_t moe_profile_read(float* stage_ms, const char** stage_names, int max_stages, int* n_stages,
                              int* n_calls);

/*
 * Operators of a decode step around the layer: rotary positions with the append
 * to a paged cache, 4-bit linear layers, attention of drafted tokens over the
 * cache, and the verification of drafted tokens.  The pages have no counterpart
 * of these entry points; they follow the conventions above.  None of them
 * allocates or synchronises, and all can be captured in a CUDA graph.  Strides
 * are in elements; the last dimension of every tensor is contiguous.
 */
#define MOE_DTYPE_BF16 0
#define MOE_DTYPE_FP16 1
#define MOE_DTYPE_FP32 2
#define MOE_MAX_TREE_NODES 64 /* drafted tokens of one sequence */

/*
 * Rotary positions.  Pair i of a head at position p turns by p * inv_freq[i]
 * radians: with c, s = scale * cos, scale * sin of that angle,
 *   y0 = x0 c - x1 s,  y1 = x1 c + x0 s        (inverse != 0: -s for s)
 * interleaved == 0: pair i is (rot_offset + i, rot_offset + rot_dim / 2 + i);
 * interleaved != 0: (rot_offset + 2i, rot_offset + 2i + 1).  Elements outside
 * [rot_offset, rot_offset + rot_dim) are copied.  Angles are 64-bit fractions of
 * a turn, off by at most |p * inv_freq| * 2^-52 + |p| * 2^-62 radians at any
 * position; their sines and cosines are right to a few units of the last place of
 * fp32, products are fp32, rounded once to the tensors' type.
 *
 *   q, k         [tokens, heads, dim] by stride_t and stride_h
 *   q_out, k_out outputs; either may be its input (in place)
 *   positions    int32 [tokens], inv_freq fp64 [rot_dim / 2] (device)
 *   slots        NULL, or int32 [tokens]: the append.  Then k_out is a paged
 *                cache: the turned keys and the values v (k_heads heads) go to
 *                page slot / page_size, row slot % page_size of k_out
 *                (k_page_stride, k_out_stride_t, k_out_stride_h) and v_cache
 *                (v_page_stride, v_slot_stride, v_head_stride).  Slots outside
 *                [0, page_size * num_pages) are skipped; the others must differ.
 * rot_dim is even; dim <= 1024.  16-byte vectors are used where rows, strides and
 * the ends of the turning part allow, single elements (pairs) otherwise.
 */
typedef struct moe_rope_args {
  int dtype; /* MOE_DTYPE_BF16, _FP16 or _FP32 */
  int tokens, dim, rot_dim, rot_offset, interleaved, inverse;
  int q_heads, k_heads; /* either may be 0 */
  float scale;
  int page_size, num_pages;
  const int32_t* positions;
  const double* inv_freq;
  const int32_t* slots;
  const void *q, *k, *v;
  void *q_out, *k_out, *v_cache;
  int64_t q_stride_t, q_stride_h, k_stride_t, k_stride_h, v_stride_t, v_stride_h;
  int64_t q_out_stride_t, q_out_stride_h, k_page_stride, k_out_stride_t, k_out_stride_h;
  int64_t v_page_stride, v_slot_stride, v_head_stride;
} moe_rope_args_t;
moe_status_t moe_rope(const moe_rope_args_t* args, moe_stream_t stream);

/*
 * Linear layer with 4-bit weights in fused_moe_int4's code format:
 *   y[m, n] = sum_k x[m, k] * q[n, k] * w_scale[n, k / group]
 *   x        bf16 or fp16 [M, K] (dtype), row stride x_stride
 *   w        uint8 [N, K/2]: two's-complement codes, column 2j in the low nibble
 *            of byte j, column 2j+1 in its high nibble
 *   w_scale  fp32 [N, K/group], group 32, 64 or 128
 *   y        as x, [M, N], row stride y_stride
 * gated != 0: w and w_scale hold 2N rows, gate rows first, and
 *   y = SiLU(gate) * up.
 * K is a multiple of group; x rows and w start on 16 bytes.  x enters the products
 * as fp16 in a power-of-two frame per row and 128 columns (exact to 2^-35 of the
 * block's largest value), codes as q + 8, whose share of 8 sum x is taken off
 * again: a sum is off by a few units of 2^-24 of sum |x| (q + 16) w_scale, so
 * a code of 0 under a value that dwarfs its row is not free.  Sums are fp32, y is
 * rounded once.  Made for the few rows of a decode step (M up to 64 or so); any M
 * is accepted.
 *   workspace    moe_linear_int4_workspace_size(...) bytes, 256-byte aligned; 0
 *                bytes (NULL) for M <= 8 with K <= 12,000 and M <= 16 with K <= 5,500
 *                (M * K that fits into shared memory).  Where one is
 *                used, moe_read_status(workspace) tells whether a device wait gave up.
 */
size_t moe_linear_int4_workspace_size(int M, int N, int K, int group, int gated);
moe_status_t moe_linear_int4(int dtype, const void* x, int64_t x_stride, const uint8_t* w, const float* w_scale,
                             int M, int N, int K, int group, int gated, void* y, int64_t y_stride,
                             void* workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * Attention of drafted tokens over a paged cache.  Sequence b has
 * context_lens[b] committed slots and the nodes node_offsets[b] ..
 * node_offsets[b+1] - 1 (at most MOE_MAX_TREE_NODES), whose keys and values
 * stand in the slots right after the committed ones.  Node j (counted from the
 * sequence's first) sees every committed slot and slot context + i for each set
 * bit i of its tree_mask word:
 *   out[j, h] = sum_s softmax_s(scale * q[j, h] . K[s, h / g]) V[s, h / g],
 * g = q_heads / k_heads.  Zeros where it sees nothing.  Scores, the softmax's
 * sums and the output's are fp32; a weight is rounded to the caches' type before
 * it meets V (fp16: in full for weights down to about 2^-21 of the row's largest,
 * in steps of 2^-31 of it below).
 *   q, out       [nodes, q_heads, dim] by stride_t and stride_h, bf16 or fp16
 *   k_cache, v_cache  [num_pages, page_size, k_heads, dim] by their strides
 *                (any order of the dimensions), the type of q
 *   block_table  int32 [batch, table_width] (table_stride): slot s of sequence b
 *                is row s % page_size of page block_table[b, s / page_size];
 *                entries past the sequence's end are not read
 *   context_lens int32 [batch], node_offsets int32 [batch + 1] ascending
 *   tree_mask    uint64 [nodes], or NULL for chains (node j sees nodes <= j)
 * All lengths are read on the device, so a captured call serves any of them.
 * dim is 64 or 128; batch <= 1024; any page_size >= 1.  Strides are multiples of
 * 8 elements (out: 4), q and the caches 16-byte aligned.  Infinities and NaN in
 * slots that a node does not see do not reach it.
 * Checked on the device: pages outside [0, num_pages) are left out; lengths that
 * do not fit the table are shortened; sequences with bad offsets are left out
 * (their rows of out are not written).  moe_read_tree_status waits for the
 * stream and gives the number of sequences with bad lengths or offsets and the
 * number of bad page reads of the last call on this workspace
 * (MOE_ERR_BAD_IDS if any).
 */
typedef struct moe_tree_attention_args {
  int dtype; /* MOE_DTYPE_BF16 or _FP16 */
  int nodes, batch, q_heads, k_heads, dim;
  int page_size, num_pages, table_width;
  float scale;
  int64_t table_stride;
  const void *q, *k_cache, *v_cache;
  const int32_t *block_table, *context_lens, *node_offsets;
  const uint64_t* tree_mask;
  void* out;
  int64_t q_stride_t, q_stride_h, out_stride_t, out_stride_h;
  int64_t k_page_stride, k_slot_stride, k_head_stride, v_page_stride, v_slot_stride, v_head_stride;
} moe_tree_attention_args_t;
size_t moe_tree_attention_workspace_size(int nodes, int batch, int q_heads, int k_heads, int dim);
moe_status_t moe_tree_attention(const moe_tree_attention_args_t* args, void* workspace, size_t workspace_bytes,
                                moe_stream_t stream);
moe_status_t moe_read_tree_status(const void* workspace, int32_t status_out[2], moe_stream_t stream);

/*
 * Verification of drafted tokens from given random numbers.  Sequence b's nodes
 * are node_offsets[b] .. node_offsets[b+1] - 1 (n <= max_nodes); its target
 * rows start at node_offsets[b] + b: first the distribution after the committed
 * tokens, then the one after each node.  A node's coin is the one of its
 * parent's row.
 *  - draft_probs given (a chain; parents NULL): node j is kept if the ones before
 *    it are and coin * draft[j, token] < target[row of j-1, token] (exact).
 *    After a refusal the next token is a sample of max(target - draft, 0).
 *  - draft_probs NULL (parents, or NULL for a chain): a node's children share
 *    [0, 1) in index order, target[token] each; the child whose share holds the
 *    coin is kept (a repeat of an earlier sibling's token has no share).  If
 *    none does, the next token is a sample of the row without the children.
 * After the last kept node the next token is a sample of its row.  A sample of w
 * is the first x with w_0 + .. + w_x > last_coins[b] * sum(w), sums being exact
 * in units of 2^-60 (where a residual has no weight: of the target row).
 *   target_probs fp32 [nodes + batch, vocab], draft_probs fp32 [nodes, vocab], by
 *                row strides of at least vocab (no broadcast rows)
 *   tokens, parents int32 [nodes], parents[j] < j counted from the sequence's
 *                first node, -1 for the committed end
 *   coins fp32 [nodes + batch], last_coins fp32 [batch], in [0, 1)
 *   out_tokens   int32 [batch, max_nodes + 1] out: kept tokens, the next, then -1
 *   path         int32 [batch, max_nodes] out: kept nodes in order, then -1
 *   accepted     int32 [batch] out: number of kept nodes; -1 (and no tokens) for
 *                a sequence with bad offsets, tokens or parents, or where the row
 *                of the next token has no weight or a sum above 8
 * Probabilities above 1 count as 1, negative ones and NaN as 0, in the test of a
 * drafted token as in a sample.
 */
moe_status_t moe_verify_draft(const float* target_probs, int64_t target_stride, const float* draft_probs,
                              int64_t draft_stride, const int32_t* tokens, const int32_t* parents,
                              const int32_t* node_offsets, const float* coins, const float* last_coins, int batch,
                              int nodes, int vocab, int max_nodes, int32_t* out_tokens, int32_t* path,
                              int32_t* accepted, moe_stream_t stream);

/*
 * Paged caches of 8-bit keys and values: E4M3 codes with one fp32 scale for every
 * slot and KV head, value = code * scale.  A view of one (keys or values), by its
 * strides in elements; the dim codes of a head are contiguous.
 */
typedef struct moe_cache_view {
  void* data;   /* codes (uint8), or elements where a cache of 16 or 32 bits is allowed */
  float* scale; /* fp32, one a slot and head (codes only) */
  int64_t page_stride, slot_stride, head_stride;
  int64_t scale_page_stride, scale_slot_stride, scale_head_stride;
} moe_cache_view_t;

/*
 * Norms of queries and keys, each head by itself, with the rotary positions and the
 * append to a paged cache in the same pass:
 *   n = x * weight / sqrt(mean(x^2) + eps)      (mean over the dim elements of a head)
 * and the pairs of n turn as moe_rope turns them (same angles, scale, layouts).  A NULL
 * weight leaves its tensor without a norm.  Everything between is fp32, rounded once
 * to the output's type.
 *   cache        MOE_CACHE_NONE: keys go to k_out; v and slots are not used
 *                MOE_CACHE_SAME: keys and values go to slots of k_cache, v_cache,
 *                which hold elements of `dtype`, as in moe_rope
 *                MOE_CACHE_E4M3: as codes and scales.  Of a head y (keys after the
 *                turn, values as they are): scale = max|y| / 448, brought into
 *                [2^-64, 2^64], and 1 where all of y is zero; code = E4M3(y / scale),
 *                to nearest even, saturating.  A head that holds an infinity or NaN
 *                gets codes 0 and the scale NaN.
 *   slots        int32 [tokens]; outside [0, page_size * num_pages): not written.
 *                The others must differ.
 *   q_weight, k_weight  [dim] of `dtype`, or NULL
 *   q_out, k_out may be q, k (in place)
 * dim <= 1024, rot_dim even, or 0 (nothing turns).  16-byte vectors are used where rows,
 * strides, weights and the ends of the turning part allow, single elements (pairs)
 * otherwise.
 */
#define MOE_CACHE_NONE 0
#define MOE_CACHE_SAME 1
#define MOE_CACHE_E4M3 2
typedef struct moe_qk_norm_rope_args {
  int dtype; /* MOE_DTYPE_BF16, _FP16 or _FP32 */
  int tokens, dim, rot_dim, rot_offset, interleaved;
  int q_heads, k_heads; /* either may be 0 */
  int cache, page_size, num_pages;
  float scale, eps; /* scale of the rotation; eps >= 1e-20 */
  const int32_t* positions;
  const double* inv_freq;
  const int32_t* slots;
  const void *q, *k, *v, *q_weight, *k_weight;
  void *q_out, *k_out;
  int64_t q_stride_t, q_stride_h, k_stride_t, k_stride_h, v_stride_t, v_stride_h;
  int64_t q_out_stride_t, q_out_stride_h, k_out_stride_t, k_out_stride_h;
  moe_cache_view_t k_cache, v_cache;
} moe_qk_norm_rope_args_t;
moe_status_t moe_qk_norm_rope(const moe_qk_norm_rope_args_t* args, moe_stream_t stream);

/*
 * Reads slots of an E4M3 cache back: out[i, h] = code * scale of slot slots[i], the
 * product in fp32, rounded once to `dtype`.  Rows whose slot lies outside
 * [0, page_size * num_pages) are zeros.  A slot may be asked for more than once.
 *   k_out, v_out [n, heads, dim] by stride_t and stride_h; either pair (cache and
 *                output) may be NULL
 */
typedef struct moe_cache_read_args {
  int dtype; /* of the outputs: MOE_DTYPE_BF16, _FP16 or _FP32 */
  int n, heads, dim, page_size, num_pages;
  const int32_t* slots;
  void *k_out, *v_out;
  int64_t k_out_stride_t, k_out_stride_h, v_out_stride_t, v_out_stride_h;
  moe_cache_view_t k_cache, v_cache;
} moe_cache_read_args_t;
moe_status_t moe_cache_read(const moe_cache_read_args_t* args, moe_stream_t stream);

/*
 * moe_tree_attention over an E4M3 cache:
 *   out[j, h] = sum_s softmax_s(scale * q[j, h] . K[s, h / g]) V[s, h / g]
 * with K[s] = code * scale of the slot, V alike.  A sequence of one node is a plain decode
 * step.  Arguments, lengths, masks, device checks and moe_read_tree_status are those of
 * moe_tree_attention.  Codes enter the products exactly, as fp16; bf16 queries as fp16 in
 * a power-of-two frame per row (exact to 2^-38 of the row's largest); scores, the
 * softmax's sums and the output's are fp32.  A weight times its slot's value scale is
 * rounded to fp16 before it meets the codes (in full down to 2^-21 of the row's largest
 * such product, in steps of 2^-31 of it below).  Value scales count as brought into
 * [2^-64, 2^64], and those of a sequence's slots and head are taken to lie within a factor
 * of 2^100 of each other (slots far below that lose their share of the softmax's sum);
 * NaN stays NaN.  Slots of zero value codes with a scale of 1, as moe_qk_norm_rope writes
 * them, count with a scale of 2^-40 there and among the products that weights are rounded
 * by: they add nothing, and values far below 1 keep their bits beside them.  Infinities and NaN in slots that a node does not see do
 * not reach it; a drafted slot whose value codes hold a NaN (0x7f, 0xff) gives NaN in the
 * whole head to the nodes that see it.
 * Code rows start on 16 bytes and their strides are multiples of 16 elements; scales by
 * any strides.
 */
typedef struct moe_tree_attention_fp8_args {
  int dtype; /* of q and out: MOE_DTYPE_BF16 or _FP16 */
  int nodes, batch, q_heads, k_heads, dim;
  int page_size, num_pages, table_width;
  float scale;
  int64_t table_stride;
  const void* q;
  const int32_t *block_table, *context_lens, *node_offsets;
  const uint64_t* tree_mask;
  void* out;
  int64_t q_stride_t, q_stride_h, out_stride_t, out_stride_h;
  moe_cache_view_t k_cache, v_cache;
} moe_tree_attention_fp8_args_t;
size_t moe_tree_attention_fp8_workspace_size(int nodes, int batch, int q_heads, int k_heads, int dim);
moe_status_t moe_tree_attention_fp8(const moe_tree_attention_fp8_args_t* args, void* workspace, size_t workspace_bytes,
                                    moe_stream_t stream);

/*
 * Sampling from logits with given random numbers, and the filtered probabilities.  Of every
 * row l, with w_x = exp((l_x - max l) / temperature):
 *   the tokens in order of their logits, ties by the lower index first;
 *   of these the first top_k (0 or below, or vocab and above: all);
 *   of these the shortest prefix whose weight is at least top_p of theirs (1 and above or
 *   NaN: all; 0 and below: the first token);
 *   of these the ones with w_x >= min_p (0 and below or NaN: all; 1 and above: those of the
 *   largest logit).
 * tokens[row] is the first x, in order of indices, with (sum of kept w_i, i <= x) > coin *
 * (sum of kept w_i); probs[row, x] = w_x / (sum of kept w_i), 0 for what is not kept, fp32.
 * A temperature of 0 or below, or NaN: the first token of the largest logit alone.
 * Weights count in units of 2^-44, off by 2^-28 of themselves and a unit, and their sums are
 * exact: results do not depend on scheduling.  So a probability below e^-31 of the row's
 * largest is 0, and those just above it have few bits: their logarithms are not those of an
 * fp32 softmax.  NaN logits count as -infinity; a row
 * of nothing else gives the token -1 and probabilities of 0.  Tokens of an infinite logit
 * share the row alike; a logit below the largest by more than fp32's range has no weight.
 *   logits   [rows, vocab] of dtype, row stride of at least vocab; vocab <= 524,288
 *   temperature, top_p, min_p fp32 [rows], top_k int32 [rows]; each may be NULL (1, 1, 0, 0)
 *   coins    fp32 [rows] in [0, 1) (what lies outside is brought to the nearest end); only
 *            for tokens
 *   tokens   int32 [rows] out, or NULL
 *   probs    fp32 [rows, vocab] out by a row stride of at least vocab, or NULL; the
 *            target_probs and draft_probs that moe_verify_draft takes
 */
typedef struct moe_sample_args {
  int dtype; /* of the logits: MOE_DTYPE_BF16, _FP16 or _FP32 */
  int rows, vocab;
  const void* logits;
  int64_t logits_stride;
  const float* temperature;
  const int32_t* top_k;
  const float *top_p, *min_p, *coins;
  int32_t* tokens;
  float* probs;
  int64_t probs_stride;
} moe_sample_args_t;
moe_status_t moe_sample(const moe_sample_args_t* args, moe_stream_t stream);

/* Static English text for a status code. */
const char* moe_status_string(moe_status_t status);

/* Text of the last error raised on the calling host thread ("" if none). */
const char* moe_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* GBMOE_H */
