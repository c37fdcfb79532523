/*
 * moe.h -- C ABI of a GB300 (sm_103a) MoE expert layer for one serving step.
 *
 * One MoE layer on a batch of T tokens (a prefill chunk of `quantum` rows plus a few decode
 * or speculative-verify rows):
 *   router logits -> top-k with normalised gates -> expert histogram, exclusive scan and
 *   stable permutation -> grouped gate/up projection with SwiGLU -> down projection ->
 *   gate-weighted unpermute-combine, plus the always-on shared expert(s).
 * Sources (web pages, by title):
 *   "moe-prefill-quantum" (ds4-server on M3 Ultra): the cause section, the expected
 *     unique-experts formula, Table 9 (tokens per expert = Q*k/E, cost flattens at 48).
 *   "DeepSeek V4.1F Q4 with native DSpark MTP on M3 Ultra": Decode paragraph (router and
 *     top-k in one dispatch, fused shared-expert gate+up+SwiGLU, bf16 rounding inside the
 *     producer kernel) and DSpark paragraph (6 verify rows share one weight stream).
 *   "Why SSD-streamed MoE was slow: 8GB Jetson Orin Nano, part 2": gate -> up -> down as
 *     SwiGLU(gate, up); `mul_mat_id` grouped expert matmul; every chosen expert must be
 *     computed exactly once (the section on generated text changing between runs).
 *
 * Conventions for every entry point below:
 *   - Tensor pointers are DEVICE pointers unless stated otherwise.  They are borrowed: the
 *     caller owns them and keeps them alive until the work queued on `stream` has finished.
 *   - Layouts are row-major with the last index contiguous.  bf16 tensors are passed as
 *     `void*` holding IEEE bfloat16 bit patterns.
 *   - The activation tensors x, y, shared_y and out of moe_layer_forward, moe_route,
 *     moe_experts and moe_combine are moved as 16-byte vectors: their base addresses must be
 *     16-byte aligned (MOE_ERR_INVALID_ARG otherwise).
 *   - Calls that take a plan and a stream only enqueue work; they never synchronise the host,
 *     never allocate device memory and are safe to capture in a CUDA graph once the plan has its
 *     weights and workspace.  T == 0 is a no-op that returns MOE_OK.
 *   - A non-MOE_OK status means nothing was enqueued (argument errors are found before any
 *     launch) or, for MOE_ERR_CUDA, that a launch failed; moe_last_error() explains it.
 *   - Problems found on the device (an expert id out of range in moe_permute input, a
 *     non-finite router logit, a wait that timed out) never trap: they set bits of the
 *     plan's device error word, read with moe_plan_get_device_error().
 *   - A plan is not thread-safe: one host thread issues its calls, and calls that share the
 *     plan's workspace must be ordered on one stream.
 *   - moe_layer_forward may run part of its work on a second stream the plan owns: forked from
 *     `stream` (an event recorded on it) and joined back (`stream` waits for an event of the
 *     second stream) before the call's last launch, so every effect is ordered on `stream` as
 *     if all of it ran there, and a graph capture of `stream` captures both.
 */
#ifndef MOE_H_
#define MOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as the CUDA runtime's cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st* moe_stream_t;

typedef struct moe_plan moe_plan; /* opaque */

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1, /* null pointer, bad size, n_prefill outside [0, T] ... */
  MOE_ERR_UNSUPPORTED = 2, /* shape the kernels do not handle (see moe_plan_create) */
  MOE_ERR_NOT_READY = 3,   /* weights or workspace not set yet */
  MOE_ERR_WORKSPACE = 4,   /* workspace too small for this T, or misaligned */
  MOE_ERR_CUDA = 5,        /* a CUDA runtime call or kernel launch failed */
  MOE_ERR_DEVICE = 6,      /* moe_plan_get_device_error found device-side error bits */
  MOE_ERR_TIMEOUT = 7      /* (device error bit) a bounded wait inside a kernel gave up */
} moe_status;

typedef enum {
  MOE_W_BF16 = 0,  /* routed expert weights in bf16 */
  MOE_W_MXFP4 = 1, /* routed expert weights block-scaled 4-bit: e2m1 codes, two per byte
                      (even element in the low nibble, bit 3 = sign), one e8m0 scale byte
                      2^(s-127) per 32 consecutive K elements (OCP MX v1.0) */
  MOE_W_FP8 = 3    /* routed expert weights in e4m3 with one fp32 scale per 128 x 128 block
                      (rows and columns counted from 0, partial blocks at the edges); the
                      activations are quantised on the fly, see moe_quantize_rows */
} moe_wdtype;

/* Element types of tensors whose type is an argument. */
typedef enum { MOE_BF16 = 0, MOE_FP16 = 1, MOE_FP32 = 2 } moe_dtype;

/* Which kernels run the expert FFN (gate/up + SwiGLU + down). */
typedef enum {
  MOE_PATH_AUTO = 0, /* chosen by T: a step of at most 8 tokens with bf16 routed weights runs the
                        whole layer in one launch that streams the weights (a GEMV on the CUDA
                        cores); larger steps, and 4-bit weights, the tensor-core path where the
                        shape allows it */
  MOE_PATH_SIMT = 1, /* plain CUDA-core grouped FFN (debug/reference path, slow) */
  MOE_PATH_TC = 2    /* tcgen05/TMEM grouped GEMM at every T (requires d % 128 == 0, d_ff % 64 == 0) */
} moe_path;

/* Device error bits (moe_plan_get_device_error). */
#define MOE_DEVERR_EXPERT_RANGE 0x1u /* moe_permute saw an id outside [0, E) */
#define MOE_DEVERR_NONFINITE 0x2u    /* a selected router logit was NaN or infinite */
#define MOE_DEVERR_TIMEOUT 0x4u      /* a bounded in-kernel wait expired */
#define MOE_DEVERR_SEGMENT 0x8u      /* internal work-list overflow (should not happen) */
#define MOE_DEVERR_RANGE 0x10u       /* an intermediate (h or y) exceeded the fp16 range and was
                                        clamped to +-65504 */

/*
 * Create a plan for E routed experts, top-k, model width d_model, expert hidden width d_ff,
 * n_shared always-on shared experts (0 allowed; their width is set by moe_plan_set_shared) and
 * routed-weight format weight_dtype.  Source: the layer shapes of "moe-prefill-quantum" (cause
 * section: 256 experts, k chosen per token) and "DeepSeek V4.1F Q4 with native DSpark MTP on M3
 * Ultra" (Decode paragraph: a 384-expert router and an always-run shared expert).
 * Host-side only; no device memory is touched.
 * Limits: 1 <= k <= E <= 1024, k <= 32, d_model and d_ff multiples of 8 (multiples of 32
 * for MOE_W_MXFP4; MOE_W_FP8 runs every such shape on the tensor cores and has no CUDA-core path,
 * its shared experts need d_model % 128 == 0 and d_ff_shared % 64 == 0).  Returns NULL on bad arguments (moe_last_error() says why).
 */
moe_plan* moe_plan_create(int E, int k, int d_model, int d_ff, int n_shared, moe_wdtype weight_dtype);

/* Free the plan and the device memory it owns (its weight copies).  NULL is a no-op.
   Synchronises the device first so no queued work still reads the plan's memory.  (No
   counterpart on the pages: resource management of this library.) */
void moe_plan_destroy(moe_plan* plan);

/* Message for the most recent failing call on this host thread ("" if none).  (No counterpart
   on the pages: error reporting of this library.) */
const char* moe_last_error(void);

/*
 * Source: the expert FFN weights gate, up, down of "Why SSD-streamed MoE was slow: 8GB Jetson
 * Orin Nano, part 2" (section re-checking part 1) and their block-scaled 4-bit form ("moe-prefill-
 * quantum", hardware-check paragraph: MXFP4 unpack times scale).
 * Copy the layer's weights into plan-owned device memory (repacked for the kernels); the
 * caller's buffers may be freed when this returns.  Synchronous.  All pointers are device
 * pointers.  bf16 down-projection weights are held as fp16 (the down GEMM multiplies them with
 * the fp16 hidden vector): exact for 2^-17 <= |w| <= 65504 and zero, smaller magnitudes land
 * on the fp16 subnormal grid (absolute error <= 2^-25); a weight above 65504 in magnitude
 * makes the call fail with MOE_ERR_UNSUPPORTED.
 *   w_router  fp32 [E][d_model]                 router weight (logit = x . w_router[e] + b[e])
 *   b_router  fp32 [E] or NULL (zero bias)
 *   w_gate    [E][d_ff][d_model]                bf16, or e2m1 codes [E][d_ff][d_model/2]
 *   w_up      [E][d_ff][d_model]                same format as w_gate
 *   w_down    [E][d_model][d_ff]                bf16, or codes [E][d_model][d_ff/2]
 *   s_gate, s_up  uint8 [E][d_ff][d_model/32]   e8m0 scales (MOE_W_MXFP4), else NULL
 *   s_down        uint8 [E][d_model][d_ff/32]
 * MOE_W_FP8: the weights are e4m3 codes of one byte in the bf16 shapes, the scales fp32
 *   s_gate, s_up  [E][ceil(d_ff/128)][ceil(d_model/128)],  s_down [E][ceil(d_model/128)][ceil(d_ff/128)].
 */
moe_status moe_plan_set_weights(moe_plan* plan, const float* w_router, const float* b_router,
                                const void* w_gate, const void* w_up, const void* w_down,
                                const void* s_gate, const void* s_up, const void* s_down);

/*
 * Source: "DeepSeek V4.1F Q4 with native DSpark MTP on M3 Ultra", Decode paragraph (the shared
 * expert's gate+up+SwiGLU runs for every token).
 * Shared experts (bf16), added to every token with weight 1:
 *   w_gate, w_up [n_shared][d_ff_shared][d_model],  w_down [n_shared][d_model][d_ff_shared].
 * Required before forward when n_shared > 0 (and before moe_plan_set_workspace, whose size
 * depends on d_ff_shared).  Copies into plan memory (w_down as fp16, as above); synchronous.
 */
moe_status moe_plan_set_shared(moe_plan* plan, int d_ff_shared, const void* w_gate,
                               const void* w_up, const void* w_down);

/* Bytes of device workspace forward/route/permute/experts need for up to T_max tokens (no
   counterpart on the pages: the library's memory contract, so that no call allocates). */
size_t moe_plan_workspace_bytes(const moe_plan* plan, int T_max);

/*
 * (No counterpart on the pages: the library's memory contract.)
 * Give the plan a caller-owned device workspace of `bytes` (>= moe_plan_workspace_bytes(T_max),
 * 256-byte aligned).  The plan keeps the pointer until the next call or destroy; it never
 * allocates device memory itself after this point.
 */
moe_status moe_plan_set_workspace(moe_plan* plan, void* dev_ptr, size_t bytes, int T_max);

/* Choose the expert-FFN kernels (default MOE_PATH_AUTO; env MOE_FORCE_PATH=simt|tc overrides
   the default at plan creation).  No counterpart on the pages: a testing and debugging switch. */
moe_status moe_plan_set_path(moe_plan* plan, moe_path path);

/*
 * How the plan's routing scores and selects experts (moe_route, moe_route_logits, moe_layer_forward).
 * Source: "moe-prefill-quantum", cause section (k of E experts chosen per token); the pages do not
 * give a scoring rule, so the forms here have no counterpart on the pages.
 *   s_e = softmax over all E logits, or sigmoid(l_e);
 *   key_e = s_e + bias[e] (the bias selects and does not weigh); key_e = -inf where l_e = -inf (a
 *     masked expert: chosen only when nothing else is left, with weight 0);
 *   n_groups > 1: groups of E / n_groups consecutive experts are ranked by the sum of their group_top
 *     (1 or 2) largest keys, and the experts outside the topk_groups best get key -inf;
 *   ids: the k largest keys in order; weights w = s of those (0 where the key is -inf),
 *     w / (sum of w + 1e-20) with renormalize, times scale.
 * Orders are (value desc, index asc; +0 == -0; NaN lowest), all arithmetic fp32.  With sigmoid scores a
 * selected logit that is NaN or +inf sets MOE_DEVERR_NONFINITE; with softmax scores any such logit of the
 * token does, selected or not: a NaN logit's score is NaN and is left out of the sum, logits of +inf
 * share the score 1.  Softmax scores, one group, renormalize, scale 1
 * and no bias weigh like the default up to rounding; NULL restores the default (the softmax of the
 * k largest logits).  bias: device fp32 [E] or NULL, copied into plan memory (synchronous when given).
 * n_groups divides E, 1 <= n_groups <= 32, 1 <= topk_groups <= n_groups with topk_groups * E / n_groups
 * >= k, group_top <= E / n_groups, scale finite; else MOE_ERR_INVALID_ARG.
 */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;
typedef struct {
  moe_score score;
  const float* bias;
  int n_groups, topk_groups, group_top;
  int renormalize;
  float scale;
} moe_routing;
moe_status moe_plan_set_routing(moe_plan* plan, const moe_routing* routing);

/*
 * The kernels the expert FFN will actually run on (no counterpart on the pages): MOE_PATH_TC
 * or MOE_PATH_SIMT, as MOE_PATH_AUTO (or a forced path) resolves for the plan's shapes and
 * weights -- the tensor-core path needs d_model % 128 == 0, d_ff % 64 == 0, d_ff_shared % 64
 * == 0 and, for MOE_W_MXFP4, every e8m0 scale byte in [104, 140] (where e2m1 x 2^(s-127) is exact
 * in fp16).  MOE_PATH_SIMT is the CUDA-core reference path, orders of magnitude slower; a caller
 * that must not run it checks this after moe_plan_set_weights / moe_plan_set_shared, and
 * moe_last_error() then names the reason.  Returns -1 for a NULL plan.
 */
int moe_plan_resolved_path(const moe_plan* plan);

/*
 * The whole layer on one serving step.  Source: "moe-prefill-quantum", the cause section and
 * Table 9 (a step's batch is a prefill chunk of `quantum` rows plus the decode rows of the
 * generating sessions, and every row goes through the MoE layer) and "DeepSeek V4.1F Q4 with
 * native DSpark MTP on M3 Ultra", Decode and DSpark paragraphs (decode and 6-row verify steps).
 * x bf16 [T][d_model] -> out bf16 [T][d_model]:
 *   out[t] = sum_j g[t,j] * FFN_{ids[t,j]}(x[t]) + sum_s FFN_shared_s(x[t]),
 * the sum taken in fp32 in slot order j = 0..k-1, then the shared term, then one
 * round-to-nearest-even to bf16.  Rows [0, n_prefill) are prefill rows and the rest decode or
 * verify rows; the layer is per token, so the result does not depend on n_prefill.
 * 0 <= T <= T_max of the workspace.
 */
moe_status moe_layer_forward(moe_plan* plan, const void* x, int T, int n_prefill, void* out,
                             moe_stream_t stream);

/*
 * The layer for a step whose routing is already known (a router that lives elsewhere, or ids and
 * gates from moe_route_logits): grouping, expert FFNs, combine and the shared experts, as
 * moe_layer_forward does after its own routing.  Source: "moe-prefill-quantum", cause section (each
 * token goes to k of the E experts); the pages have no counterpart to the separate call.
 *   ids int32 [T][k], gates fp32 [T][k].  An id outside [0, E), or one that repeats an earlier slot
 * of its token, sets MOE_DEVERR_EXPERT_RANGE and contributes nothing.  gates enter as they are (they
 * need not sum to one).
 */
moe_status moe_layer_forward_routed(moe_plan* plan, const void* x, int T, const int32_t* ids, const float* gates,
                                    void* out, moe_stream_t stream);

/*
 * Router + top-k.  Source: "DeepSeek V4.1F Q4 with native DSpark MTP on M3 Ultra", Decode
 * paragraph (router logits and top-k selection, one dispatch); "moe-prefill-quantum", cause
 * section (k of E experts per token).  The tie rule (lower index first) is this library's.
 * logits fp32 [T][E] (may be NULL: then kept in the workspace),
 * ids int32 [T][k], gates fp32 [T][k].  Slot j holds the (j+1)-th largest logit under the
 * order (value desc, index asc; +0 == -0; NaN lowest); gates are the softmax of the k
 * selected logits, computed in fp32.  moe_plan_set_routing replaces this rule.
 */
moe_status moe_route(moe_plan* plan, const void* x, int T, float* logits, int32_t* ids,
                     float* gates, moe_stream_t stream);

/* Top-k and gates from given fp32 logits [T][E] (the same selection code as moe_route; the
   Decode paragraph's top-k step of "DeepSeek V4.1F Q4 with native DSpark MTP on M3 Ultra").
   Exists so that selection can be compared bit for bit on identical logits. */
moe_status moe_route_logits(moe_plan* plan, const float* logits, int T, int32_t* ids,
                            float* gates, moe_stream_t stream);

/*
 * Grouping of the T*k assignments a = t*k + j by expert.  Source: "Why SSD-streamed MoE was
 * slow: 8GB Jetson Orin Nano, part 2" -- the grouped expert matmul (`mul_mat_id`, first-cache
 * section) needs the rows of each expert together, and the section on generated text changing
 * between runs requires every chosen expert to be computed exactly once (a bijection here):
 *   counts int32 [E], offsets int32 [E+1] (exclusive scan, offsets[E] = T*k),
 *   perm int32 [T*k] (perm[r] = a, a stable counting sort: rows of one expert ascend by a),
 *   inv_perm int32 [T*k] (inv_perm[perm[r]] = r).
 * An id outside [0, E), or one that repeats an earlier slot of the same token, sets
 * MOE_DEVERR_EXPERT_RANGE and is dropped: it is not counted, gets no row, and its inv_perm entry
 * is -1; perm then holds offsets[E] < T*k rows and its tail is left untouched.  With T == 0,
 * counts and offsets are zeroed and ids, perm, inv_perm may be NULL.
 */
moe_status moe_permute(moe_plan* plan, const int32_t* ids, int T, int32_t* counts,
                       int32_t* offsets, int32_t* perm, int32_t* inv_perm, moe_stream_t stream);

/*
 * moe_permute without a plan and without any device allocation.  The pages have no counterpart
 * to this call; it exists for callers that cannot allocate device memory: engines whose memory
 * planner owns the whole device and forbids components from allocating outside its pool, and
 * code on a latency-critical path, where cudaMalloc would synchronise the device.  Same inputs and outputs as moe_permute
 * (ids int32 [T][k] -> counts [E], offsets [E+1], perm and inv_perm [T*k], all device
 * pointers; invalid or repeated ids are dropped with inv_perm = -1, but there is no error word).
 * Scratch is a fixed 1 MiB device array inside the library, present on every GPU that loads it
 * until the process exits; ceil(ceil(T / 32) / 4) * 4 * E must not exceed 262144 (T <= 32768 at
 * E = 256),
 * else MOE_ERR_WORKSPACE and nothing is enqueued.  The first call in a CUDA context (the first
 * on a device, and the first after that device's context was destroyed and re-created, e.g. by
 * cudaDeviceReset) looks up the array's device address (cudaGetSymbolAddress); make that first
 * call before any stream capture.  All calls share the array: two calls that may run at the same time on the GPU
 * (unordered streams) race; calls ordered on one stream do not.  Every scratch word a call
 * reads is rewritten by that call, so no clearing is needed between calls.
 */
moe_status moe_permute_static(int E, int k, const int32_t* ids, int T, int32_t* counts,
                              int32_t* offsets, int32_t* perm, int32_t* inv_perm, moe_stream_t stream);

/*
 * Self-test of the bounded waits' expiry path (failure detection; the pages have no counterpart).
 * Launches one CTA whose first warp waits on an mbarrier phase nothing completes, with the same
 * bounded wait the layer's kernels use, while its second warp holds a TMEM allocation: after
 * about one second (the kernels' wait limit) the wait gives up, sets MOE_DEVERR_TIMEOUT in *err
 * and raises the CTA's abort flag, and the CTA takes the GEMM kernels' abort teardown (waits out
 * in-flight copies, frees TMEM) and returns, leaving the context usable.
 *   err     device uint32, OR-ed with the error bits (the caller clears it first);
 *   result  device uint32 [3]: [0] = 2 when the wait expired (1 if it completed), [1] = the
 *           milliseconds it waited, [2] = 1 if the abort flag was raised.
 * Returns MOE_ERR_INVALID_ARG for NULL pointers, MOE_ERR_CUDA if the launch fails.
 */
moe_status moe_selftest_wait_expiry(uint32_t* err, uint32_t* result, moe_stream_t stream);

/*
 * Expert FFNs on grouped rows (testing entry point for the grouped GEMMs).  Source: "Why
 * SSD-streamed MoE was slow: 8GB Jetson Orin Nano, part 2", section re-checking part 1 (gate ->
 * up -> down, SwiGLU(gate, up)); "DeepSeek V4.1F Q4 with native DSpark MTP on M3 Ultra", Decode
 * paragraph (intermediates rounded inside the producing kernel):
 *   y[r] = FFN_e(x[perm[r] / k]) for r in [offsets[e], offsets[e+1]),  fp16 [T*k][d_model],
 *   shared_y[t] = sum_s FFN_shared_s(x[t]) fp16 [T][d_model] (may be NULL if n_shared == 0).
 * FFN(x) = W_d (silu(W_g x) * (W_u x)) with fp32 accumulation; the hidden vector is rounded to
 * fp16 (it is the fp16 operand of the down GEMM; with MOE_W_FP8 x and the hidden vector are
 * quantised in blocks of 128 instead, see moe_quantize_rows) and y is rounded to fp16.  Values beyond the
 * fp16 range are clamped and set MOE_DEVERR_RANGE.  offsets and perm as produced by
 * moe_permute (device pointers).
 */
moe_status moe_experts(moe_plan* plan, const void* x, int T, const int32_t* offsets,
                       const int32_t* perm, void* y, void* shared_y, moe_stream_t stream);

/*
 * Gate-weighted unpermute-combine.  Source: the combine is implicit in the pages -- every token's
 * output is the gate-weighted sum of its chosen experts' outputs ("moe-prefill-quantum", cause
 * section: each token is sent to k of the E experts; "Why SSD-streamed MoE was slow", part 2,
 * the section on generated text changing between runs: each chosen expert counted exactly once).
 *   out[t] = sum_{j<k} gates[t,j] * y[inv_perm[t*k+j]]  (+ shared_y[t]),
 * fp32 accumulation in slot order, then the shared term, one round-to-nearest-even to bf16.
 *   y         fp32 [T*k][d_model] in grouped (permuted) row order (device);
 *   gates     fp32 [T][k];  inv_perm int32 [T*k] (entries < 0 are skipped);
 *   shared_y  fp32 [T][d_model] or NULL;  out bf16 [T][d_model].
 * Needs no workspace and no weights (only the plan's k and d_model).  d_model % 8 != 0 gives
 * MOE_ERR_UNSUPPORTED.  (moe_layer_forward runs the same kernel on its own fp16 intermediates.)
 */
moe_status moe_combine(moe_plan* plan, const float* y, const float* gates, const int32_t* inv_perm,
                       const float* shared_y, int T, void* out, moe_stream_t stream);

/* Synchronise the device, return the device error word in *code (host pointer) and clear
   it.  Returns MOE_ERR_DEVICE when *code != 0.  No counterpart on the pages (failure detection
   of this library: device-side problems never trap). */
moe_status moe_plan_get_device_error(moe_plan* plan, uint32_t* code);

/*
 * Per-kernel timing for profiling (no counterpart on the pages).  When enabled, every kernel launched by the calls above
 * is bracketed by CUDA events recorded on the launching stream (a few microseconds of
 * overhead per launch).  moe_plan_timing_report synchronises, writes one line per kernel
 * name, "name launches total_ms\n", into buf (host memory, NUL-terminated, truncated to
 * len) and resets the counters.  Returns the number of bytes the full report needs.
 */
moe_status moe_plan_enable_timing(moe_plan* plan, int enable);
size_t moe_plan_timing_report(moe_plan* plan, char* buf, size_t len);

/* Number of kernels the most recent moe_layer_forward call launched (no counterpart on the
   pages; the Decode paragraph of "DeepSeek V4.1F Q4 with native DSpark MTP on M3 Ultra" counts
   dispatches per layer the same way). */
int moe_plan_last_launch_count(const moe_plan* plan);

/*
 * Step composer: the layer calls (serving steps) a prompt's prefill is cut into.
 * Source: "moe-prefill-quantum" -- the cause section's source excerpt (the server hands the
 * prompt over in pieces of `quantum` tokens while any request is generating, else of 2048) and
 * the section on prefill_cap boundaries with its code excerpt and Table 11 (the engine cuts a
 * piece where the absolute context position crosses a multiple of prefill_cap; a prompt that
 * starts off a boundary keeps being cut, e.g. 2048, 509, 1539, ... from 1539 mod 4096).
 * Reading where the excerpt is silent: no call exceeds prefill_cap tokens.
 *
 * Host-only and pure (no device work, no plan).  Prefilling n_tokens prompt tokens from
 * context position start_pos: writes the first min(total, max_calls) calls, in order, to
 * `calls` (host memory; may be NULL when max_calls == 0) and the total number of calls to
 * *n_calls (host pointer).  Each call's `n` prompt rows go to moe_layer_forward as its
 * n_prefill rows, followed by one row per generating request.
 * MOE_ERR_INVALID_ARG when start_pos < 0, n_tokens < 0, quantum < 1, prefill_cap < 1 or
 * n_calls is NULL.
 */
typedef struct {
  int64_t pos;   /* context position of the call's first prompt token */
  int32_t n;     /* prompt tokens in the call, 1 <= n <= prefill_cap */
  int32_t piece; /* index of the server piece the call belongs to */
} moe_prefill_call;

moe_status moe_compose_prefill(int64_t start_pos, int64_t n_tokens, int32_t quantum,
                               int32_t generation_active, int32_t prefill_cap,
                               moe_prefill_call* calls, int64_t max_calls, int64_t* n_calls);

/*
 * 8-bit blocks.  Source: "moe-prefill-quantum", hardware-check paragraph (a quantised weight read
 * is unpack, times scale, accumulate) and the DSpark paragraph of "DeepSeek V4.1F Q4 with native
 * DSpark MTP on M3 Ultra" (8-bit projections of a 6-row verify block); the format is this
 * library's choice.  A block of values with largest magnitude amax is stored as e4m3 codes q
 * (sign, 4 exponent bits, 3 mantissa bits, largest value 448, 0x7F / 0xFF NaN) and one fp32 scale s:
 *   s = max(amax * (1 / 448), 2^-126),  q = e4m3(v * (1 / s)),  v ~ q * s,
 * every quotient and product rounded to fp32 (1 / 448 too), q to nearest even.  A NaN element keeps the code
 * of NaN; an infinite element makes its block's scale infinite and the block NaN.
 *
 * moe_quantize_rows: rows [T][K] of x_dtype (row pitch ldx elements) in blocks of 1 x 128 along K
 *   (the last one partial): codes uint8 [T][ldq] (ldq >= K rounded up to 128, a multiple of 16; the
 *   columns from K to the end of the last block are zeroed), scales fp32 [T][lds], lds >= ceil(K / 128).
 * moe_quantize_blocks: a matrix [rows][K] in blocks of 128 x 128: codes [rows][K] without
 *   padding, scales [ceil(rows / 128)][ceil(K / 128)].
 * Both only enqueue work; moe_quantize_rows' codes must be 16-byte aligned; K <= 2^31 - 2048.  T == 0 or rows == 0 enqueues nothing.
 */
moe_status moe_quantize_rows(const void* x, moe_dtype x_dtype, int64_t ldx, int T, int K, uint8_t* q, int64_t ldq,
                            float* s, int64_t lds, moe_stream_t stream);
moe_status moe_quantize_blocks(const void* w, moe_dtype w_dtype, int rows, int K, uint8_t* q, float* s,
                                   moe_stream_t stream);

/*
 * A projection with 8-bit weights: out[t][n] = sum_b sa[t][b] sw[n / 128][b] (sum over block b of
 * a[t][k] w[n][k]).  Source: the 8-bit projections of the DSpark paragraph (above); the pages have
 * no counterpart to the 8-bit activations.  The sums of one block of 128 are formed by the tensor
 * core and added up in fp32.
 *   moe_linear_create       N output features, K input features, both >= 1 (<= 2^20).  Host only.
 *   moe_linear_set_weights  codes [N][K] and scales [ceil(N/128)][ceil(K/128)] (device), copied into
 *                               memory of the handle in the kernel's layout; synchronous.
 *   ..._workspace_bytes / set_workspace   caller-owned memory for the quantised rows of up to T_max rows,
 *                               256-byte aligned; one call at a time uses it (order them on a stream).
 *   moe_linear_forward      x [T][K] of x_dtype (pitch ldx) is quantised (moe_quantize_rows) and
 *                               multiplied; out [T][N] (pitch ldo) in out_dtype, MOE_BF16 or MOE_FP32.
 *   moe_linear_forward_quantized   the same for rows that are already codes (pitch ldq, a multiple
 *                               of 16, 16-byte aligned) with their scales (pitch lds, a multiple of 4,
 *                               16-byte aligned); neither columns beyond K nor scales beyond
 *                               ceil(K / 128) are read; needs no workspace.
 *   moe_linear_get_device_error    as moe_plan_get_device_error, for the handle's calls.
 * The forward calls only enqueue work, and a NULL or not-ready handle, T < 0 or T > T_max, a pitch
 * below the width or an unknown type is an error before any launch; so are more than 2^31 - 2048 rows.
 */
typedef struct moe_linear moe_linear; /* opaque */

moe_linear* moe_linear_create(int N, int K);
void moe_linear_destroy(moe_linear* lin);
moe_status moe_linear_set_weights(moe_linear* lin, const uint8_t* q, const float* s);
size_t moe_linear_workspace_bytes(const moe_linear* lin, int T_max);
moe_status moe_linear_set_workspace(moe_linear* lin, void* dev_ptr, size_t bytes, int T_max);
moe_status moe_linear_forward(moe_linear* lin, const void* x, moe_dtype x_dtype, int64_t ldx, int T, void* out,
                                  moe_dtype out_dtype, int64_t ldo, moe_stream_t stream);
moe_status moe_linear_forward_quantized(moe_linear* lin, const uint8_t* q, int64_t ldq, const float* s,
                                            int64_t lds, int T, void* out, moe_dtype out_dtype, int64_t ldo,
                                            moe_stream_t stream);
moe_status moe_linear_get_device_error(moe_linear* lin, uint32_t* code);

/*
 * Rows between token order and expert order, in any element type, with the gradients.  Source:
 * "Why SSD-streamed MoE was slow: 8GB Jetson Orin Nano, part 2", first-cache section (the grouped
 * expert matmul needs each expert's rows together); the pages have no counterpart to the gradients.
 * For experts computed outside this library (moe_experts gathers and scatters on its own).
 * inv_perm int32 [T][k] as moe_permute writes it: the row, in expert order, of token t's assignment
 * j.  An entry below 0 or at n_rows and above is a dropped assignment and contributes nothing; no
 * two entries may name the same row.  weights fp32 [T][k], or NULL for 1.
 *   moe_sort_rows              out[inv[t,j]] = w[t,j] x[t]
 *   moe_sort_rows_backward     dx[t] = sum_j w[t,j] grad[inv[t,j]],  dweights[t,j] = <x[t], grad[inv[t,j]]>
 *   moe_combine_rows           out[t] = sum_j w[t,j] y[inv[t,j]] + shared[t]
 *   moe_combine_rows_backward  dy[inv[t,j]] = w[t,j] grad[t],  dweights[t,j] = <grad[t], y[inv[t,j]]>
 *     (the gradient of shared is grad itself)
 * Token rows [T][d] and rows in expert order [n_rows][d] have any pitch (elements) >= d, aligned to
 * their elements; 16-byte aligned rows with d % 8 == 0 take the faster accesses.  Rows of out / dy
 * that no entry names are left as they are.  Sums are fp32 in slot order, the shared term last, rounded
 * once to the output's type (beyond fp16's range: infinity); sums over d are fp32 in a fixed order.
 * dweights fp32 [T][k] or NULL (x / y is then not read and may be NULL); 0 for a dropped assignment.
 * moe_sort_rows without weights copies the bits.  Outputs do not overlap inputs.  1 <= k <= 32,
 * T k and n_rows <= 2^31 - 1, d <= 2^24.  The calls only enqueue work, need no plan and no workspace.
 */
moe_status moe_sort_rows(const void* x, moe_dtype x_dtype, int64_t ldx, int T, int k, int d, const int32_t* inv_perm,
                         const float* weights, void* out, int64_t ldo, int64_t n_rows, moe_stream_t stream);
moe_status moe_sort_rows_backward(const void* grad, moe_dtype dtype, int64_t ldg, int64_t n_rows, int T, int k, int d,
                                  const int32_t* inv_perm, const float* weights, const void* x, int64_t ldx, void* dx,
                                  int64_t lddx, float* dweights, moe_stream_t stream);
moe_status moe_combine_rows(const void* y, moe_dtype y_dtype, int64_t ldy, int64_t n_rows, int T, int k, int d,
                            const int32_t* inv_perm, const float* weights, const void* shared, moe_dtype shared_dtype,
                            int64_t lds, void* out, moe_dtype out_dtype, int64_t ldo, moe_stream_t stream);
moe_status moe_combine_rows_backward(const void* grad, moe_dtype grad_dtype, int64_t ldg, int T, int k, int d,
                                     const int32_t* inv_perm, const float* weights, const void* y, int64_t ldy, void* dy,
                                     moe_dtype y_dtype, int64_t lddy, int64_t n_rows, float* dweights,
                                     moe_stream_t stream);

/*
 * Verification of drafted tokens.  Source: "DeepSeek V4.1F Q4 with native DSpark MTP on M3 Ultra", DSpark
 * paragraph (a block of 6 rows verifies drafted tokens); the acceptance rule has no counterpart on the pages.
 * B requests own consecutive rows of the step's R verify rows: request b the rows offsets[b] .. offsets[b+1] - 1
 * (int32 [B+1], device; requests share no row), one for each of its n = rows - 1 drafts and one behind the last.  Row r of target [R][V]
 * holds the probabilities of the token that follows; drafts[r] (int32 [R]; not read in a request's last row) is the
 * token that row r verifies, and row r of draft_probs [R][V] the distribution q it was drawn from (not read in a
 * request's last row; NULL: the draft was certain, q = 1 at the drafted token and 0 elsewhere).  u fp32 [R] and
 * u_sample fp32 [B] are uniform numbers in [0, 1).
 *   Draft i is accepted while u_i q_i(draft) < p_i(draft), up to the first that is not.
 *   Behind the accepted drafts comes one token: from r = max(p - q, 0) of the refused row (without draft_probs: p
 *   without the refused draft), or from p of the last row when no draft was refused: the lowest index whose
 *   cumulative sum of r exceeds u_sample[b] * (sum of r); the last index with r > 0 if none does.  Where r sums to 0
 *   the token is drawn from that row's p, where p does too it is -1.
 * Probabilities need not sum to one.  A value that is NaN, negative or above 2^64 counts as 0; a draft outside
 * [0, V) is refused.  The products u q are exact, sums and u_sample times them have
 * some 47 bits (where the sum is above 2^-100).
 *   tokens   int32 [R]: the accepted drafts, the drawn token, then -1, in the request's rows; rows of no request
 *            are left as they are.
 *   accepted int32 [B]: the number of accepted drafts; 0 for a request without rows; -1 (and no token is written)
 *            where offsets[b] < 0, offsets[b] > offsets[b+1] or offsets[b+1] > R.
 * target and draft_probs have one element type and row pitches ldt, ldd >= V.  V <= 2^30, B <= 65535.  Only
 * enqueues work (one launch), needs no plan and no workspace.
 */
moe_status moe_verify_drafts(const void* target, moe_dtype dtype, int64_t ldt, const void* draft_probs, int64_t ldd,
                             int R, int V, const int32_t* drafts, const int32_t* offsets, int B, const float* u,
                             const float* u_sample, int32_t* tokens, int32_t* accepted, moe_stream_t stream);

/*
 * Low-rank adapters of many requests beside a shared projection.  Source: the projections of "DeepSeek V4.1F Q4
 * with native DSpark MTP on M3 Ultra", Decode and DSpark paragraphs; the adapters have no counterpart on the pages.
 *   out[t] = base[t] + B_a (s_a A_a x[t]),  a = ids[t];  out[t] = base[t], bit for bit, where ids[t] == -1 or
 * slot a is empty.
 * A handle holds n slots of one shape: A_a [r_a][K], B_a [N][r_a], r_a <= r_max, s_a a number.
 *   moe_adapters_create     1 <= n <= 1024, 1 <= N, K <= 2^20, 1 <= r_max <= 128; dtype (bf16 or fp16) is that of A,
 *                           B and x.  Host only.  (Slots are held padded to rank 16, 32, 64 or 128 of r_max, and twice:
 *                           as small and as large steps read them.)
 *   moe_adapters_set        contiguous A and B (device) copied into slot `slot` of the handle's memory in the kernel's
 *                           layout; r = 0 empties the slot.  Synchronous: waits for the whole device before and after, so
 *                           that queued calls finish with the old contents (not while a stream is being captured).  Other
 *                           slots keep theirs.
 *   ..._workspace_bytes / set_workspace   caller-owned memory for grouping up to T_max rows, 256-byte aligned; one call
 *                           at a time uses it (order them on a stream).
 *   moe_adapters_forward    x [T][K] (pitch ldx), ids int32 [T], base [T][N] (pitch ldb; NULL: zero) and out [T][N]
 *                           (pitch ldo) of out_dtype (bf16, fp16 or fp32).  base may be out (same pitch), else they do not
 *                           overlap.  Rows may ask for any adapters in any order.  An id outside [-1, n) sets
 *                           MOE_DEVERR_EXPERT_RANGE and counts as -1.
 *   moe_adapters_get_device_error   as moe_plan_get_device_error, for the handle's calls.
 * The device that is current when the first slot or the workspace is set holds the handle's memory: these calls, the
 * forward call and the error query are refused with another one current.
 * Both products accumulate in fp32; u = s_a A_a x is held as terms of the 16-bit type: three in bf16 for an fp32 result
 * (all of u's 24 bits), two for a 16-bit one (relative error 2^-16 of u), two in fp16 (2^-22 of u, or 2^-39 of the row's
 * largest where that is more); base is added in fp32 and the sum rounded once.  A row's result does not depend on its
 * place or on the other rows; steps of another T may split the sums otherwise.  T_max <= 2^26.
 * The forward call only enqueues work; a NULL or not-ready handle, T < 0 or T > T_max, a pitch below the width or an
 * unknown type is an error before any launch.
 */
typedef struct moe_adapters moe_adapters; /* opaque */

moe_adapters* moe_adapters_create(int n, int N, int K, int r_max, moe_dtype dtype);
void moe_adapters_destroy(moe_adapters* h);
moe_status moe_adapters_set(moe_adapters* h, int slot, const void* a, const void* b, int r, float scale);
size_t moe_adapters_workspace_bytes(const moe_adapters* h, int T_max);
moe_status moe_adapters_set_workspace(moe_adapters* h, void* dev_ptr, size_t bytes, int T_max);
moe_status moe_adapters_forward(moe_adapters* h, const void* x, int64_t ldx, int T, const int32_t* ids, const void* base,
                                int64_t ldb, void* out, moe_dtype out_dtype, int64_t ldo, moe_stream_t stream);
moe_status moe_adapters_get_device_error(moe_adapters* h, uint32_t* code);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H_ */
