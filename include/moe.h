/*
 * moe.h -- C ABI of the GB300 (sm_103a) sparse Mixture-of-Experts FFN layer.
 *
 * The layer, as the source pages state it:
 *   logits = x W_g                                   (router projection)
 *   (ids, w) = top-k of softmax(logits), renormalised (gating_top_k_softmax)
 *   rows grouped by expert                            (init_routing)
 *   h_e = act(x W13_e[:, :I]) * (x W13_e[:, I:])      (grouped matmul + swiglu)
 *   y_e = h_e W2_e                                    (grouped matmul)
 *   out = sum_j w_j y_{ids_j} + SharedExpert(x)       (finalize_routing)
 *
 * Conventions shared by every call
 * --------------------------------
 * - All tensors are device pointers, row-major and contiguous, owned by the
 *   caller.  The library allocates no device memory; scratch space comes from
 *   the caller's workspace `ws` of at least moe_workspace_size(cfg) bytes
 *   (256-byte aligned).  The first 256 bytes of `ws` are a control block that
 *   holds the device error word (and, with MOE_OPT_DYNAMIC_TILES, the GEMMs'
 *   tile counters).
 * - `stream` is a cudaStream_t (NULL = legacy default stream).  Every call is
 *   asynchronous on that stream and returns after enqueueing its kernels.
 *   The compute calls enqueue only kernels and event records / waits (no
 *   host synchronisation, no allocation), so they can be captured into a
 *   CUDA graph; the first call on a device does one-time set-up (kernel
 *   attributes, moe_layer's side stream), so make it before capturing.
 * - Return value: MOE_OK or a negative moe_status_t.  Argument errors are
 *   detected on the host before anything is enqueued.  Data errors found on
 *   the device (an expert id outside [0, E), non-monotone offsets, a permuted
 *   position outside [0, T*k), non-finite router logits) never fault: the
 *   offending element is skipped or clamped and a code is recorded in the
 *   device error word, which moe_read_device_status() reads.
 * - Pointers must be 16-byte aligned and every row pitch a multiple of 16
 *   bytes, which makes D, I and I_shared multiples of 8 (16 for fp8 weights).
 * - The control block has to be zero when a workspace is first used (zero-fill
 *   it once); the calls leave it ready for the next.  A workspace serves one
 *   call at a time: calls that may overlap on the GPU need one each.  What
 *   moe_linear_w4 uses as a workspace serves its own calls only.
 * - Dtypes: act_dtype applies to x, W_g, the permuted rows and out.  w_dtype
 *   applies to W13, W2 and the shared expert's weights.  Supported pairs:
 *   (F32, F32), (BF16, BF16), (BF16, FP8_E4M3), (BF16, FP8_E4M3_NK),
 *   (BF16, FP8_E4M3_NK_A8), and for moe_layer_few (BF16, W4_*).
 *   Router logits and gate weights are always fp32; the expert outputs
 *   y_perm and the shared-expert output are fp32, or bf16 for fp8-weight
 *   layers (one rounding each, inside the 6e-2 RMS bar of those layers).
 *   The intermediate h takes 4 bytes per element: fp32 for fp32 layers and
 *   for FP8_E4M3 weights; for bf16 weights two bf16 planes [M, I] -- h_hi =
 *   bf16(h) followed by h_lo = bf16(h - h_hi) -- which the down projection
 *   consumes as two bf16 tensor-core products, so that h keeps about 16
 *   significant bits.  FP8_E4M3 weights (W8A16, in the pages' [.., K, N]
 *   layout) run on the fp16 tensor-core kind: e4m3 expands exactly to fp16,
 *   and the A rows (x, then h) are fp16 rows times exact powers of two, so
 *   each product equals the bf16-activation product up to fp32 summation
 *   order (x exactly; h rounded once to 11 significant bits relative to its
 *   row).
 * - FP8_E4M3_NK: the same e4m3 values and per-column scales, with each
 *   expert's matrix stored transposed (W13 [E, 2I, D], W2 [E, D, I], W13s
 *   [2 I_shared, D], W2s [D, I_shared]: the reduction dimension contiguous),
 *   as moe_pack_weights_nk writes it once from the [.., K, N] layout.  These
 *   layers run on the 8-bit tensor-core kind (kind::f8f6f4) with no weight
 *   expansion: every A row (x, then h) is scaled by an exact power of two so
 *   that its largest element lies in [128, 256) and carried as two e4m3
 *   terms, hi = e4m3(v) and lo = e4m3(v - hi), multiplied by the weights in
 *   two products into one fp32 accumulator.  A bf16 x is represented exactly
 *   except for elements below 2^-9 of their row's largest, which keep an
 *   absolute error under 2^-17 of it.  h is stored in bf16 (2 bytes per
 *   element; 8 significant bits) and reaches the down projection the same
 *   way, so both products see exactly the bf16 rows but for those small
 *   elements.
 * - FP8_E4M3_NK_A8 (W8A8, opt-in): the weights of FP8_E4M3_NK, and the
 *   activations quantised per row to one e4m3 term with a dynamic scale, as
 *   "用SGLang-JAX在TPU上优化Ling-2.6-1T" §5 ("激活量化", "逐通道
 *   direct_scaled_dot") describes: s = max|row| / 448 and q = e4m3(v / s)
 *   (fp32 divisions, nearest even, saturating); x per token before the
 *   permutation, h per row after it is stored in bf16; one 8-bit product per
 *   multiply-add, (sum q_a q_w) * s_a * s_w[n] after the reduction.  The
 *   router still projects the bf16 x.  This changes the result (e4m3 keeps
 *   4 significant bits of each activation); the bf16-activation layouts
 *   above are the configured arithmetic.
 * - W4_G32 / W4_G64 / W4_G128: 4-bit weights with group scales, taken by
 *   moe_layer_few and moe_block (moe_layer and moe_grouped_ffn return
 *   MOE_ERR_UNSUPPORTED; moe_dequantize_w4 gives them bf16 weights).  A matrix
 *   with N outputs and K inputs is [N, K/2] bytes: byte j of a row holds the
 *   codes 0..15 of inputs 2j (low nibble) and 2j + 1 (high nibble); with a
 *   bf16 scale per row and group, [N, K/group], the weight is
 *   (code - 8) * scale.  W13 [E, 2I, D/2] (rows [0, I) gate, [I, 2I) up), s13
 *   [E, 2I, D/group], W2 [E, D, I/2], s2 [E, D, I/group], the shared expert's
 *   likewise without E.  D, I and I_shared are multiples of the group.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_F32 = 0,
  MOE_BF16 = 1,
  MOE_FP8_E4M3 = 2,   /* weights [.., K, N] as the pages write them */
  MOE_FP8_E4M3_NK = 3, /* the same weights transposed per matrix (moe_pack_weights_nk) */
  MOE_FP8_E4M3_NK_A8 = 4, /* FP8_E4M3_NK weights, activations quantised per row (W8A8) */
  MOE_W4_G32 = 5,  /* 4-bit weights, a scale per row and group of 32 inputs (moe_layer_few) */
  MOE_W4_G64 = 6,  /* groups of 64 */
  MOE_W4_G128 = 7  /* groups of 128 */
} moe_dtype_t;

/* SwiGLU: SiLU(gate) * up.  GEGLU: tanh-approximated GELU(gate) * up. */
typedef enum { MOE_ACT_SWIGLU = 0, MOE_ACT_GEGLU_TANH = 1 } moe_act_t;

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = -1,  /* null pointer, bad shape, misalignment, k > E, E > 512 */
  MOE_ERR_UNSUPPORTED = -2,  /* dtype / activation combination not built */
  MOE_ERR_CUDA = -3,         /* a CUDA runtime or driver call failed */
  MOE_ERR_DEVICE_CHECK = -4, /* the device error word is set (see moe_read_device_status) */
  MOE_ERR_WORKSPACE = -5     /* workspace missing, misaligned or too small */
} moe_status_t;

/* Codes stored in the device error word (bit flags, OR-ed together). */
#define MOE_DEV_BAD_EXPERT_ID 0x1   /* an id outside [0, E) reached routing */
#define MOE_DEV_BAD_OFFSETS 0x2     /* offsets not monotone or beyond T*k */
#define MOE_DEV_BAD_DEST 0x4        /* a permuted position outside [0, T*k) */
#define MOE_DEV_NONFINITE_LOGIT 0x8 /* NaN / Inf router logit or biased score (treated as -Inf) */
#define MOE_DEV_WAIT_TIMEOUT 0x10   /* a bounded pipeline wait gave up */

typedef struct {
  int32_t T;           /* tokens */
  int32_t D;           /* hidden size */
  int32_t E;           /* routed experts, 1..512 */
  int32_t k;           /* experts per token, 1..min(E, 16) */
  int32_t I;           /* routed expert intermediate size */
  int32_t I_shared;    /* shared expert / dense MLP intermediate, 0 = none */
  int32_t act;         /* moe_act_t */
  int32_t act_dtype;   /* moe_dtype_t: MOE_F32 or MOE_BF16 */
  int32_t w_dtype;     /* moe_dtype_t: MOE_F32, MOE_BF16 or MOE_FP8_E4M3 */
  int32_t renormalize; /* 1: gate weights renormalised over the k chosen experts */
} moe_config_t;

/* Bytes of workspace that every call below accepts for this configuration.
 * The last region, at T <= 32, is the scratch of moe_layer_few's kernel, and only
 * that call, and moe_block where it takes that kernel, ask for it: moe_layer, the
 * stage calls and other batches of moe_block accept what comes before (of which
 * moe_layer needs all; the stage calls use the control block and their own
 * scratch).  So a workspace that holds moe_layer's largest batch holds its smaller
 * ones, while few tokens of moe_layer_few or moe_block can ask for more than a
 * larger batch: for these, take the maximum over the configurations.
 * Returns 0 for an invalid configuration. */
size_t moe_workspace_size(const moe_config_t* cfg);

/* Router projection and gating_top_k_softmax.
 * Pages: "千问 3.5 MoE 在 TPU 上的系统优化实战" (routed MoE paragraph: the
 * router projects each token and picks the top 10 experts by softmax);
 * "CANN/cann-recipes-infer：Qwen3-MoE优化", section "GMM使能和Routing优化"
 * (npu_moe_gating_top_k_softmax fuses top-k and softmax) and section
 * "融合RMSNorm + Cast" (the gate is computed in fp32).
 *   x          [T, D] act_dtype, or NULL: then `logits` is an input.
 *   Wg         [D, E] act_dtype (ignored when x is NULL).
 *   logit_bias [E] fp32 or NULL, added to x W_g (must be NULL when x is NULL).
 *   logits     [T, E] fp32: x W_g + bias with fp32 accumulation (output), or
 *              the input logits when x is NULL.
 *   topk_ids   [T, k] int32 out: experts by descending logit, the lower index
 *              first among equal logits.
 *   topk_w     [T, k] fp32 out: softmax over the k chosen logits when
 *              cfg->renormalize, else the full-softmax probabilities. */
int moe_route(const moe_config_t* cfg, const void* x, const void* Wg, const float* logit_bias,
              float* logits, int32_t* topk_ids, float* topk_w, void* ws, size_t ws_bytes,
              void* stream);

/* init_routing + compute_expert_tokens + the permutation gather.
 * Pages: "CANN/cann-recipes-infer：Qwen3-MoE优化", section "GMM使能和Routing优化"
 * (npu_moe_init_routing orders rows by expert; npu_moe_compute_expert_tokens
 * counts tokens per expert); "千问 3.5 MoE 在 TPU 上的系统优化实战", SparseCore
 * paragraph (gather rows by routing index into one contiguous unpadded buffer).
 * Expanded row r = t*k + j is token t's j-th choice.
 *   topk_ids    [T, k] int32 in.
 *   x           [T, D] act_dtype in (may be NULL: no gather, x_perm unused).
 *   counts      [E] int32 out: rows per expert.
 *   offsets     [E+1] int32 out: exclusive scan of counts; offsets[E] = T*k.
 *   sorted_rows [T*k] int32 out: expanded row at each permuted position,
 *               grouped by expert, ascending r inside an expert (stable).
 *   dest        [T*k] int32 out: permuted position of each expanded row
 *               (inverse of sorted_rows; -1 for a row with an invalid id).
 *   x_perm      [T*k, D] act_dtype out: x_perm[p] = x[sorted_rows[p] / k]. */
int moe_permute(const moe_config_t* cfg, const int32_t* topk_ids, const void* x, int32_t* counts,
                int32_t* offsets, int32_t* sorted_rows, int32_t* dest, void* x_perm, void* ws,
                size_t ws_bytes, void* stream);

/* moe_permute for callers that cannot allocate device memory.  The source
 * pages have no counterpart: this is an interface for hosts that hand an
 * operator only its input and output buffers and forbid device allocation
 * while a request runs (a serving runtime that plans all device memory at
 * start-up, a plugin interface without a workspace argument), so they cannot
 * provide the workspace moe_permute takes.
 *   Same arguments, argument checks and results as moe_permute, without
 *   ws / ws_bytes (the configuration is validated exactly as there).  Its
 *   scratch (one expert histogram per routing segment: E <= 512 experts times
 *   at most 128 segments) is a fixed 256 KiB array in the library's device
 *   memory, held on every GPU that loads the library until the process exits.
 *   Limit: T*k <= 2^30 expanded rows, the same as every other call; larger
 *   sizes return MOE_ERR_INVALID_ARG before anything is enqueued.
 *   The first call on each device looks up the array's device address
 *   (cudaGetSymbolAddress) with that device current; make that first call
 *   before any stream capture.  Nothing is allocated or freed, by this call
 *   or by any library routine it uses.
 *   Every call shares the one array, and it keeps the last call's contents:
 *   calls that overlap on the GPU (different streams, or different host
 *   threads, without ordering between them) race on it.
 *   There is no error word to read: a row with an id outside [0, E) gets
 *   dest = -1, is left out of sorted_rows, and offsets[E] < T*k. */
int moe_permute_noalloc(const moe_config_t* cfg, const int32_t* topk_ids, const void* x,
                        int32_t* counts, int32_t* offsets, int32_t* sorted_rows, int32_t* dest,
                        void* x_perm, void* stream);

/* Grouped matmul over expert segments, with the gate/up activation epilogue,
 * plus the shared expert (or dense MLP) over all tokens.
 * Pages: "CANN/cann-recipes-infer：Qwen3-MoE优化", sections "MoE TP优化 /
 * 计算分解" (w13 = [gate | up], swiglu = SiLU(first half) * second half) and
 * "GMM使能和Routing优化" (npu_grouped_matmul); "Gemma-4 模型优化报告" §2
 * (GEGLU experts; dense MLP added to the MoE output); "用SGLang-JAX在TPU上优化
 * Ling-2.6-1T" §5 "逐通道 direct_scaled_dot" (per-output-channel fp8 scale
 * applied after the K reduction).
 *   x_perm  [T*k, D] act_dtype: expert-ordered rows.
 *   offsets [E+1] int32: segment bounds (from moe_permute).
 *   W13     [E, D, 2I] w_dtype: columns [0, I) gate, [I, 2I) up
 *           (FP8_E4M3_NK: [E, 2I, D], rows [0, I) gate, [I, 2I) up).
 *   s13     [E, 2I] fp32 per-column scales (fp8 only, else NULL).
 *   W2      [E, I, D] w_dtype (FP8_E4M3_NK: [E, D, I]);
 *   s2      [E, D] fp32 (fp8 only, else NULL).
 *   h       out: act(gate) * up, [T*k, I] fp32 (fp32 layers and FP8_E4M3
 *           weights), [T*k, I] bf16 (FP8_E4M3_NK weights), or the bf16 pair
 *           [2, T*k, I] (hi plane, then lo plane) for bf16 weights.
 *   y_perm  [T*k, D] out: h W2 per segment (times s2 for fp8); fp32, or
 *           bf16 for fp8-weight layers (their 6e-2 bar leaves room, and the
 *           combine then reads half the bytes).
 *   x, W13s [D, 2*I_shared], s13s [2*I_shared], W2s [I_shared, D], s2s [D]:
 *           the shared expert (FP8_E4M3_NK: W13s [2*I_shared, D], W2s
 *           [D, I_shared]); x NULL (or I_shared == 0) skips it.
 *   h_s     shared intermediate, same layout as h with T rows.
 *   s_out   [T, D] out: shared expert output, fp32 (bf16 for fp8 weights). */
int moe_grouped_ffn(const moe_config_t* cfg, const void* x_perm, const int32_t* offsets,
                    const void* W13, const float* s13, const void* W2, const float* s2, void* h,
                    void* y_perm, const void* x, const void* W13s, const float* s13s,
                    const void* W2s, const float* s2s, void* h_s, void* s_out, void* ws,
                    size_t ws_bytes, void* stream);

/* finalize_routing fused with the shared-expert add.
 * Pages: "CANN/cann-recipes-infer：Qwen3-MoE优化", section "GMM使能和Routing优化"
 * (npu_moe_finalize_routing restores token order and takes the weighted sum);
 * "千问 3.5 MoE 在 TPU 上的系统优化实战": y = Router(x) + SharedExpert(x).
 *   out[t] = round( sum_{j<k} w[t, j] * y_perm[dest[t*k + j]] + s[t] ),
 *   accumulated in fp32 with j ascending, the shared row added last, one
 *   rounding to act_dtype.
 *   y_perm [T*k, D] fp32 (bf16 for fp8-weight layers), dest [T*k] int32,
 *   topk_w [T, k] fp32, s [T, D] of y_perm's type or NULL, out [T, D]
 *   act_dtype. */
int moe_finalize(const moe_config_t* cfg, const void* y_perm, const int32_t* dest,
                 const float* topk_w, const void* s, void* out, void* ws, size_t ws_bytes,
                 void* stream);

/* The whole layer: moe_route, moe_permute, moe_grouped_ffn, moe_finalize on
 * one stream, with every intermediate carved from `ws`.  Arguments as above;
 * the shared-expert weights may be NULL when cfg->I_shared == 0. */
int moe_layer(const moe_config_t* cfg, const void* x, const void* Wg, const float* logit_bias,
              const void* W13, const float* s13, const void* W2, const float* s2,
              const void* W13s, const float* s13s, const void* W2s, const float* s2s, void* out,
              void* ws, size_t ws_bytes, void* stream);

/* The whole layer for a few tokens (1 <= T <= 32) as one kernel launch: the
 * decode step of a small batch.  When to take it rather than moe_layer, measured
 * with weights read from HBM (1 to 32 tokens, five layers in bf16, one in both
 * e4m3 layouts): it is faster for FP8_E4M3 weights at every T (90 us against 178 at
 * one token of a Ling-style layer, 1239 against 2079 at 32), for FP8_E4M3_NK up to
 * 16 tokens (90 : 126, 799 : 813; 32: 1280 : 1234), for bf16 up to 8 tokens (34 : 41
 * at one token of a Qwen3-style layer, 94 : 107 at 8) and mostly beyond (176 : 183 at
 * 32).  moe_layer is faster where bf16 layers have many small experts and a wide
 * shared one (Gemma-style: 138 : 140 at 8 tokens, 205 : 198 at 16, 264 : 246 at 32).
 * 4-bit weights have no other call.  Pages: "用SGLang-JAX在TPU上优化Ling-2.6-1T" §4 (decode
 * near the weight-read bound); "CANN/cann-recipes-infer：Qwen3-MoE优化" (the
 * single-batch decode it is measured on, and its 4-bit weights).
 *   Arguments, layouts and results as moe_layer, with any E in 1..512 (W_g's
 *   rows need no padding here) and with the weight types BF16, FP8_E4M3,
 *   FP8_E4M3_NK and W4_*.  s13 / s2 / s13s / s2s: fp32 per column for e4m3
 *   weights, bf16 per row and group for 4-bit weights, NULL for bf16.
 *   Other types and T > 32 return MOE_ERR_UNSUPPORTED.
 *   Arithmetic: bf16 weights are multiplied in bf16, x as it is and h as two bf16
 *   terms (16 significant bits).  e4m3 weights and 4-bit codes minus 8 are
 *   multiplied as fp16 (exact there) by rows of x and h in fp16, each row times a
 *   power of two that puts its largest element in [2^14, 2^15): x keeps its bits
 *   but where an element is less than 2^-31 of the row's largest (it then errs by
 *   at most 2^-39 of that one), h is rounded to 11 significant bits (same floor).
 *   (Rows whose largest element is below 2^-86 keep fewer bits.)  All sums are
 *   fp32; e4m3 scales multiply the finished sums, group scales the fp32 sums of their
 *   group.  The weighted sum over a token's experts
 *   is fp32 in a fixed order (a tree over j mod 8, the shared expert as j = k),
 *   rounded once to bf16.  The same inputs give the same bits on every call.
 *   Logits, ids and weights are left in the workspace (MOE_WS_LOGITS,
 *   MOE_WS_TOPK_IDS, MOE_WS_TOPK_W), no other intermediate is.
 *   The kernel is launched cooperatively, one CTA on every SM: it starts when
 *   every SM has room for it.  Waits inside it are bounded; one that gives up
 *   sets MOE_DEV_WAIT_TIMEOUT (zero-fill the control block before the next
 *   call then).  Capturable into a CUDA graph after a first call per shape
 *   class outside of one. */
int moe_layer_few(const moe_config_t* cfg, const void* x, const void* Wg, const float* logit_bias,
                  const void* W13, const void* s13, const void* W2, const void* s2, const void* W13s,
                  const void* s13s, const void* W2s, const void* s2s, void* out, void* ws,
                  size_t ws_bytes, void* stream);

/* y = x W^T for a few rows of x and 4-bit weights with group scales:
 *   y[m, n] = sum_k x[m, k] * (code[n, k] - zero[n, k / group]) * scale[n, k / group]
 * for the projections around the layer (a dense or shared projection, the
 * logits of a decode step).  No page has this operator by itself; the Qwen3-MoE
 * page's 4-bit weights are its source.
 *   M       rows of x, 0..32 (more: MOE_ERR_UNSUPPORTED; 0: nothing is done, x and y may be NULL).
 *   K, N    inputs, a multiple of `group`, at most 65535 groups; outputs, any N
 *           from 1 to 2^31 - 512.
 *   group   32, 64 or 128.
 *   x       [M, K] bf16.
 *   Wq      [N, K/2] bytes as MOE_W4_* describes.
 *   scales  [N, K/group] bf16.
 *   zeros   [N, K/group] bytes, zero points in their low four bits, or NULL: 8.
 *   y       [M, N] bf16 or fp32 (y_dtype MOE_BF16 / MOE_F32), one rounding.
 *   ws      moe_linear_w4_workspace_size(M, K, N) bytes, 256-byte aligned,
 *           zero-filled once (all of it); its control block takes the device
 *           error word.  Calls of other sizes may follow in it when it is large
 *           enough for each, other functions' calls may not: it holds counts that
 *           are zero between calls.  After MOE_DEV_WAIT_TIMEOUT, zero-fill it
 *           before the next call.
 *   x, Wq, scales and y 16-byte aligned, zeros not.  x and code - zero are
 *   multiplied in bf16, exactly; a group's sum is fp32, its scale multiplies that,
 *   and the groups are added in fp32.  The same inputs give the same bits on every
 *   call (of one M, K and N: which kernel runs depends on them). */
size_t moe_linear_w4_workspace_size(int32_t M, int32_t K, int32_t N);
int moe_linear_w4(int32_t M, int32_t K, int32_t N, int32_t group, const void* x, const void* Wq,
                  const void* scales, const void* zeros, void* y, int32_t y_dtype, void* ws,
                  size_t ws_bytes, void* stream);

/* Weights [G, K, N] (the pages' layout, bf16 or fp32: w_dtype) to the 4-bit form:
 * Wq [G, N, K/2] and scales [G, N, K/group].  Per row and group: scale =
 * bf16(max |w| / 7), code = round(w / scale) (nearest, ties to even, clamped to
 * -8..7) + 8; an all-zero group gets scale 1; a group with an infinity or NaN
 * gets a NaN scale, so that its products are NaN.  1 <= G <= 65535.
 * Run once when weights are loaded. */
int moe_quantize_w4(const void* W, int32_t w_dtype, int64_t G, int32_t K, int32_t N, int32_t group,
                    void* Wq, void* scales, void* stream);
/* The way back: W [G, K, N] bf16 = bf16((code - zero) * scale), for moe_layer
 * (prefill) on weights kept in 4 bits.  zeros [G, N, K/group] or NULL: 8. */
int moe_dequantize_w4(const void* Wq, const void* scales, const void* zeros, int64_t G, int32_t K,
                      int32_t N, int32_t group, void* W, void* stream);

/* How moe_route_gated and moe_block choose experts.  With logits l [E] of a token
 * (x W_g + logit_bias, fp32) and its scores p, all in fp32 (what is compared to 2^-22
 * and 2^-23 of |l| relative, the weights as expf and division have them):
 *   p       softmax over the E experts, or sigmoid of each logit (score).
 *   c       p + select_bias: takes part in the choice, not in the weights.
 *   groups  the experts in n_group runs of E / n_group; a group's value is the
 *           largest c in it, or the sum of the two largest (group_score); the
 *           topk_group largest groups stay, the others' experts cannot be chosen.
 *   ids     the k largest c, descending.
 *   w       p of the chosen (cfg->renormalize: divided by their sum), times scale.
 * Ties, of groups and of experts, go to the lower index.  Without select_bias the
 * order of experts (and of groups by their largest) is taken from the logits, which
 * order as p does and differ where p no longer does.  Renormalised weights of a
 * softmax are the softmax over the chosen logits; of sigmoids below e^-57 the same
 * (their ratios there, kept from underflow).  A non-finite logit (or c) counts as
 * -infinity: p is 0, the expert is chosen last and not part of a group's sum,
 * MOE_DEV_NONFINITE_LOGIT is set; a token that has only such experts to choose gets
 * weights scale / k.  (So a select_bias of -infinity takes an expert out.  A softmax's sum
 * is over all finite logits, those of such experts too.) */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score_t;
typedef enum { MOE_GROUP_MAX = 0, MOE_GROUP_TOP2_SUM = 1 } moe_group_score_t;
typedef struct {
  int32_t score;       /* moe_score_t */
  int32_t n_group;     /* 1..32, divides E; 1: no groups */
  int32_t topk_group;  /* 1..n_group, topk_group * E / n_group >= k */
  int32_t group_score; /* moe_group_score_t */
  float scale;         /* factor of the weights, finite */
} moe_gate_t;

/* moe_route with the choice above.  Arguments as there (x NULL: `logits` is the
 * input), and
 *   gate         not NULL.
 *   select_bias  [E] fp32 or NULL. */
int moe_route_gated(const moe_config_t* cfg, const moe_gate_t* gate, const void* x, const void* Wg,
                    const float* logit_bias, const float* select_bias, float* logits,
                    int32_t* topk_ids, float* topk_w, void* ws, size_t ws_bytes, void* stream);

/* The residual's addition and the root-mean-square norm of rows of D values, and the
 * normed rows in 8 bits:
 *   s = x + residual,  y = s / sqrt(mean(s^2) + eps) * weight
 * in fp32 (a row whose squares leave fp32's range is scaled by a power of two first).
 * Pages: "CANN/cann-recipes-infer：Qwen3-MoE优化", section "融合RMSNorm + Cast" (the
 * norm writes the forms that its readers take); "用SGLang-JAX在TPU上优化
 * Ling-2.6-1T" §5 "激活量化" (8-bit rows with dynamic scales).
 *   rows, D   rows >= 0; D a multiple of 8, 8..32768 (more: MOE_ERR_UNSUPPORTED).
 *   dtype     MOE_BF16 or MOE_F32: x, residual, weight, sum_out and y.
 *   x         [rows, D].
 *   residual  [rows, D] or NULL: nothing is added.
 *   weight    [D].
 *   eps       finite, >= 0.
 *   sum_out   [rows, D] out or NULL: s, rounded once.  May be x or residual itself.
 *   y         [rows, D] out or NULL, rounded once.  May be x or residual itself.
 *   q         [rows, D] e4m3 out or NULL; y or q is needed.
 *   q_group   values to a scale: 0 (the whole row), 32, 64 or 128 (dividing D).
 *   q_scales  [rows, D / q_group] fp32 out ([rows] for q_group 0), with q.
 * A scale is max |y| / 448 of its values (1 where all are zero, at least 2^-126, NaN where one
 * is an infinity or NaN), q = e4m3(y / scale) from y before any other rounding (fp32
 * division, nearest even).  All pointers 16-byte aligned; outputs overlap nothing but as
 * said (sum_out and y are two buffers).  NULL tensors are taken when rows is 0.  No
 * workspace. */
int moe_add_rms_norm(int32_t rows, int32_t D, int32_t dtype, const void* x, const void* residual,
                     const void* weight, float eps, void* sum_out, void* y, void* q, int32_t q_group,
                     float* q_scales, void* stream);

/* The low-rank adapter of each row's own request, beside a projection that all rows
 * share (moe_linear_w4's, or any):
 *   y[t, n] = base[t, n] + scales[a] * sum_j (sum_k x[t, k] A[a, j, k]) B[a, n, j],  a = ids[t]
 *   T         rows, 0..2^30.
 *   K, N, r   inputs and outputs, multiples of 8 to 2^24; rank, a multiple of 8 to 256 (more:
 *             MOE_ERR_UNSUPPORTED).  Adapters of smaller ranks are padded with zeros.
 *   n         adapters, 1..16384 (more: MOE_ERR_UNSUPPORTED).
 *   x         [T, K] bf16.
 *   ids       [T] int32 in any order; a row whose id is not in [0, n) has no adapter:
 *             its y is its base.
 *   A, B      [n, r, K] and [n, N, r] bf16.
 *   scales    [n] fp32, or NULL: 1.
 *   base      [T, N] of y's type, y itself (in place), or NULL: 0.
 *   y         [T, N] bf16 or fp32 (y_dtype), one rounding.  Overlaps nothing else (y == x:
 *             MOE_ERR_INVALID_ARG).
 *   ws        moe_lora_workspace_size(T, K, N, r, n) bytes (0: sizes not taken), which hold
 *             every batch of up to T rows with the same K, N, r and n; 256-byte aligned;
 *             holds nothing between calls but the control block (its first 256 bytes,
 *             zero-filled once), which takes the device error word.
 * x A^T is summed in fp32 and multiplied by B as two bf16 terms (16 significant bits),
 * as three (24) where y is fp32; its sums are fp32.  Infinities of x are the formula's; an
 * infinite B may give NaN (its product with a term that is 0), and s x A^T beyond bf16's largest
 * number counts as infinite.  The same inputs give the same bits
 * on every call of the same sizes.  Pointers but ids and scales 16-byte aligned, those 4. */
size_t moe_lora_workspace_size(int32_t T, int32_t K, int32_t N, int32_t r, int32_t n);
int moe_lora(int32_t T, int32_t K, int32_t N, int32_t r, int32_t n, const void* x,
             const int32_t* ids, const void* A, const void* B, const float* scales, const void* base,
             void* y, int32_t y_dtype, void* ws, size_t ws_bytes, void* stream);

/* A pre-norm residual MoE block: moe_add_rms_norm, then moe_layer or moe_layer_few with
 * moe_route_gated's choice, on one stream:
 *   sum_out = x + residual,  y = norm(x + residual) * norm_weight,  out = layer(y)
 * (the sum is normed before it is rounded for sum_out).
 *   gate        NULL: moe_layer's choice (softmax top-k), select_bias NULL then.
 *   norm_weight [D] act_dtype, or NULL: no norm, the layer takes x (residual, sum_out
 *               and y NULL, eps 0).
 *   y           [T, D] act_dtype out: the normed rows, which the router projects.  May
 *               not overlap anything else.
 *   sum_out     and out are two buffers.
 *   s13, s2, s13s, s2s  fp32 per column (e4m3 weights), bf16 per row and group (4-bit
 *               weights, as moe_layer_few has them), or NULL.
 *   ws          moe_workspace_size(cfg) bytes (as said there, for batches of up to 32
 *               tokens and larger ones the maximum over both).
 *   x, residual, sum_out, eps as in moe_add_rms_norm; the other arguments and the errors
 *   as in moe_layer (E a multiple of 8 for bf16 activations).
 * moe_layer_few's kernel takes 4-bit weights (T <= 32, else MOE_ERR_UNSUPPORTED),
 * FP8_E4M3 up to 32 tokens, FP8_E4M3_NK up to 16 and BF16 up to 8 (with a gate 4), and
 * leaves in the workspace what it does; with a gate it is given the choice of the
 * launches before it.
 * FP8_E4M3_NK_A8 layers take their 8-bit rows from the norm (rounded once, from fp32),
 * instead of from y: one launch and one reading of y less. */
int moe_block(const moe_config_t* cfg, const moe_gate_t* gate, const void* x, const void* residual,
              const void* norm_weight, float eps, const void* Wg, const float* logit_bias,
              const float* select_bias, const void* W13, const void* s13, const void* W2,
              const void* s2, const void* W13s, const void* s13s, const void* W2s, const void* s2s,
              void* sum_out, void* y, void* out, void* ws, size_t ws_bytes, void* stream);

/* One of the calls above with its arguments in a block of 8-byte words, in their
 * order: integers and addresses (0: NULL) as they are, eps as a double.  For bindings
 * that take longer for a call the more arguments it has; same results and errors,
 * MOE_ERR_INVALID_ARG for another call, NULL words or an int32 argument of more bits. */
#define MOE_CALL_ADD_RMS_NORM 0
#define MOE_CALL_ROUTE_GATED 1
#define MOE_CALL_LORA 2
int moe_call(int32_t call, const void* words);

/* Device byte offsets inside `ws` where moe_layer keeps its intermediates,
 * for inspection (logits, ids, weights, counts, offsets, sorted_rows, dest,
 * x_perm, h, y_perm, h_s, s).  `which` is one of the MOE_WS_* indices;
 * returns (size_t)-1 for an unknown index, an invalid configuration, or an
 * fp8-only region of a layer without fp8 weights. */
#define MOE_WS_LOGITS 0
#define MOE_WS_TOPK_IDS 1
#define MOE_WS_TOPK_W 2
#define MOE_WS_COUNTS 3
#define MOE_WS_OFFSETS 4
#define MOE_WS_SORTED_ROWS 5
#define MOE_WS_DEST 6
#define MOE_WS_X_PERM 7
#define MOE_WS_H 8
#define MOE_WS_Y_PERM 9
#define MOE_WS_H_SHARED 10
#define MOE_WS_S 11
/* fp8-weight layers only: x times exact powers of two [T, D] -- as fp16
 * rows (FP8_E4M3) or as two-term e4m3 rows [T, 2D], hi in bytes [0, D) and
 * lo in [D, 2D) (FP8_E4M3_NK) -- their inverse scales per token [T] and per
 * permuted row [T*k] (fp32); for these layers MOE_WS_X_PERM holds rows of
 * the same form. */
#define MOE_WS_X16 12
#define MOE_WS_TOK_INV 13
#define MOE_WS_ROW_INV 14
size_t moe_workspace_offset(const moe_config_t* cfg, int which);

/* Synchronises `stream`, reads and clears the device error word of `ws`.
 * Returns MOE_OK, MOE_ERR_DEVICE_CHECK (flags written to *flags when not
 * NULL) or MOE_ERR_CUDA. */
int moe_read_device_status(void* ws, void* stream, int32_t* flags);

/* Transposes one-byte (e4m3) weight matrices into the layout of
 * MOE_FP8_E4M3_NK layers; run once when the weights are loaded.
 * Pages: "用SGLang-JAX在TPU上优化Ling-2.6-1T" §5 "逐通道 direct_scaled_dot"
 * (fp8 tokens and fp8 weights fed straight to the matrix unit, f32 partial
 * sums, per-token and per-channel scales after the reduction).  The pages
 * write each projection input dimension first; this library's 8-bit
 * tensor-core path reads both operands with the reduction dimension
 * contiguous, hence this one-time copy.
 *   W     [G, K, N] device, one byte per element (the pages' layout: W13 with
 *         G = E, K = D, N = 2I; W2 with K = I, N = D; G = 1 for the shared
 *         expert's matrices).
 *   W_nk  [G, N, K] device out: W_nk[g][n][c] = W[g][c][n].  Must not
 *         overlap W.
 *   1 <= G <= 65535; K and N positive multiples of 16; both pointers
 *   16-byte aligned and the two buffers disjoint, else MOE_ERR_INVALID_ARG
 *   before anything is enqueued.
 *   Asynchronous on `stream`; needs no workspace. */
int moe_pack_weights_nk(const void* W, int64_t G, int32_t K, int32_t N, void* W_nk, void* stream);

/* Human-readable text of a moe_status_t. */
const char* moe_status_string(int status);

/* Kernel launches one moe_layer call enqueues for this configuration. */
int moe_layer_launch_count(const moe_config_t* cfg);

/* Kernel-variant options (process-wide; set them from the thread that
 * launches, between calls).  Returns the previous value, or
 * MOE_ERR_INVALID_ARG for an unknown option.
 *   MOE_OPT_PAIR_TILES: how grouped GEMMs with a full 256-column B tile
 *   use 2-CTA clusters (tcgen05 cta_group::2, M = 256 rows per tile, each CTA
 *   loading half of B; a group's last tile with at most 64 (gate/up) or 128
 *   (down) rows runs swapped, with the weights as the M = 256 operand and the
 *   rows as N): 3 (default) = when there are at least 150 rows per group on
 *   average; 1 = always; 2 = always, without swapped tails; 0 = never (one
 *   CTA per 128-row tile).  FP8_E4M3 GEMMs always use one CTA per tile;
 *   FP8_E4M3_NK GEMMs follow the same policy (their swapped tails stack the
 *   hi and lo e4m3 rows along N).  Results are the same up to fp32
 *   summation order. */
#define MOE_OPT_PAIR_TILES 1
/*   MOE_OPT_GATHER_A: where moe_layer's routed gate/up GEMM takes its A
 *   rows.  0 = a permuted copy of x written by the gather kernel, read by
 *   tiled TMA loads; 1 = no copy: the GEMM reads the rows of x (for fp8
 *   weights, x's fp16 or two-term e4m3 rows) with TMA tile::gather4 loads, on
 *   one-CTA tiles (measured 2.5-2.8x slower on GB300); 2 = no copy, for bf16
 *   layers: four extra warps of the GEMM copy each tile row's 128 bytes per
 *   k-block from x by 16-byte cp.async, eight lanes per row (fp8 layers take
 *   1); 3 (default) = 2 for bf16 layers with at least 32 routed rows per
 *   expert on average (prefill: Qwen3-MoE-style layer 526 -> 490 us,
 *   Gemma-4-style 491 -> 469 us on GB300), 0 otherwise and when
 *   MOE_OPT_SHARED_IN_GEMM is set for a layer that can take it.  Same
 *   results. */
#define MOE_OPT_GATHER_A 2
/*   MOE_OPT_DECODE_KERNEL: 1 (default) = the swap-AB decode kernel (weights
 *   as the 128-row MMA operand, 16 or 64 rows per tile, each active expert's
 *   weights streamed once) for decode-size passes where it measured faster: a
 *   single group (shared expert) of at most 64 rows, at most one row per group
 *   on average, up to 4 rows per group with at most 256 groups (bf16), or fp8
 *   weights at up to 16 rows per group; 0 = always the 128-row-tile kernel;
 *   2 / 3 = the decode kernel with 64 / 16 rows per tile for every routed or
 *   shared FFN pass (testing).  Same results up to fp32
 *   summation order. */
#define MOE_OPT_DECODE_KERNEL 3
/*   MOE_OPT_PDL: 1 (default) = kernels are launched with programmatic
 *   dependent launch (each kernel may be scheduled while its predecessor in
 *   the stream runs and waits on the device, with griddepcontrol.wait, for
 *   the predecessor's completion before it touches memory); 0 = plain stream
 *   order.  Same results. */
#define MOE_OPT_PDL 4
/*   MOE_OPT_SHARED_STREAM: 1 (default) = moe_layer runs the shared expert
 *   on a second stream owned by the library (one per device, created on the
 *   first call that needs it) that forks from the caller's stream once x is
 *   ready and joins it before the finalize kernel, so that the shared GEMMs
 *   overlap routing and the routed GEMMs; 2 = the same stream, forked after
 *   init_routing instead (the shared GEMMs then start beside the permutation
 *   kernel, which needs no shared memory, rather than ahead of the routing
 *   kernels, which do); 0 = everything on the caller's stream.  Same results.
 *   Fork and join are event record / wait pairs made under a lock, so calls
 *   from several host threads stay correct (their shared experts then
 *   serialise on the one side stream). */
#define MOE_OPT_SHARED_STREAM 5
/*   MOE_OPT_FUSED_COMBINE: 1 = moe_layer fuses the combine into the routed
 *   down projection (NEXT-1's second half: "千问 3.5 MoE 在 TPU 上的系统优化实战",
 *   SparseCore paragraph -- un-permute and reduce without the intermediate
 *   expert rows): the down pass multiplies each row by its routing weight and
 *   adds it, with fp32 atomics, into [T, D] fp32 sums (the y_perm region of the
 *   workspace, zeroed first), and the last kernel adds the shared row and
 *   rounds once; no y_perm rows are written or read.  The k rows of a token
 *   are then summed in whatever order they arrive, so the output may differ
 *   from the default's fixed j-ascending order in the last bit (run to run as
 *   well).  Layers with bf16 weights or K-contiguous e4m3 weights; others
 *   (and 0, the default) keep finalize's fixed order. */
#define MOE_OPT_FUSED_COMBINE 6
/*   MOE_OPT_TILE_ORDER: 1 = the grouped GEMMs schedule the experts heaviest
 *   first (most rows; the lower index first among equal counts), the
 *   longest-processing-time order of "企业官网建设流程全解析" §4 (sort the
 *   experts' work heaviest first so that the largest ones do not trail);
 *   every CTA sorts the expert counts itself (a bitonic sort in one warp)
 *   while it builds its tile schedule; 0 (default) = expert order.  Same
 *   results. */
#define MOE_OPT_TILE_ORDER 7
/*   MOE_OPT_SHARED_IN_GEMM: 1 = moe_layer runs the shared expert as one more
 *   group of the routed grouped GEMMs (NEXT-3: "用SGLang-JAX在TPU上优化
 *   Ling-2.6-1T" §5 "核内共享专家", the shared expert moved into the routed
 *   kernel): its token rows are appended to the permuted rows (rows R .. R+T-1
 *   of x_perm, h and y_perm), its tiles follow the routed tiles in the same
 *   persistent launches, and the layer makes no launches of its own for it.
 *   Layers whose I_shared equals I with bf16 or K-contiguous e4m3 weights
 *   (the workspace of such a layer always holds those T extra rows); other
 *   layers, and 0 (default), run the shared expert in its own launches (on
 *   the side stream, MOE_OPT_SHARED_STREAM).  Same results. */
#define MOE_OPT_SHARED_IN_GEMM 9
/*   MOE_OPT_FUSED_ROUTING: 1 (default) = the routing chain in fewer
 *   launches ("CANN/cann-recipes-infer：Qwen3-MoE优化", section "GMM使能和
 *   Routing优化": fused gate + gating_top_k_softmax, fused init_routing):
 *   (a) for more than 64 tokens of bf16 activations (64 <= E <= 512), the
 *   router projection and the top-k softmax are one kernel: a cluster of up
 *   to 4 CTAs per 128 tokens splits the fp32 sum over D into consecutive
 *   slices on the tensor core and hands the partial rows through distributed
 *   shared memory to the CTA that adds them in slice order and takes the
 *   top-k; inside moe_layer each of its CTAs also counts its tokens' ids per
 *   expert, and init_routing (above the one-launch size) is one kernel with
 *   a CTA per router CTA that sorts that CTA's rows from those histograms;
 *   (b) otherwise, for 8193 to 65536 expanded rows, the histogram, scan and
 *   stable scatter of init_routing are one cluster of 8 CTAs that exchange
 *   their expert histograms through distributed shared memory.
 *   (a) applies where its grid has at least 64 CTAs (prefill; decode batches
 *   take the split-K projection); 2 = (a) wherever the shape allows it, 3 =
 *   the same without the histogram sort (testing).  0 = a grouped-GEMM launch
 *   writing split-K planes, then the top-k kernel; a histogram kernel, then a
 *   scan + scatter kernel.  The logits may differ in the last bits between
 *   the two (another split of the fp32 sum over D); ids and weights follow
 *   from each one's own logits by the same rule, and the permutation is the
 *   same. */
#define MOE_OPT_FUSED_ROUTING 10
/*   MOE_OPT_B_PREFETCH: n > 0 = the grouped GEMMs' TMA producer also
 *   prefetches its weight box n k-blocks ahead into L2 (near the end of a
 *   tile, the first k-blocks of its next tile), so that more weight bytes are
 *   in flight from HBM than the shared-memory ring holds; for the weights
 *   read in one box per stage (bf16 as 64-column blocks, K-contiguous e4m3).
 *   0 (default) = off; at most 16.  Same results. */
#define MOE_OPT_B_PREFETCH 11
/*   MOE_OPT_DYNAMIC_TILES: the persistent grouped GEMMs (128-row and 2-CTA
 *   tiles) can hand out their tiles dynamically: each CTA's producer (the
 *   leader's, in a pair) takes tiles from a counter in the workspace's
 *   control block with an atomic add and passes them to the CTA's (pair's)
 *   other roles through a small queue in shared memory, one tile ahead, so
 *   that CTAs whose tiles run faster take more of them; the calls that launch
 *   those GEMMs zero the counters first (one memset).  2 (default) = for the
 *   prefill-sized gate/up passes (at least 1024 rows and 32 per group) whose
 *   tiles are at least 64 k-blocks long (D >= 4096 for bf16 weights, D >=
 *   8192 for K-contiguous e4m3 weights; Ling-style prefill layer 11.35-11.39
 *   -> 11.04-11.07 ms on GB300); 1 = every pass (the short
 *   down-pass tiles measured 3-8 % slower); 0 = tile t to CTA (pair) t modulo
 *   the grid.  Same results. */
#define MOE_OPT_DYNAMIC_TILES 12
/*   MOE_OPT_SHARED_CTAS: n > 0 = the shared expert's GEMMs on the library's
 *   side stream use at most n CTAs (their persistent grid), leaving the other
 *   SMs to the routed path's kernels that run beside them; 0 (default) = one
 *   CTA per SM.  Same results. */
#define MOE_OPT_SHARED_CTAS 13
int moe_set_option(int option, int value);

/* Per-kernel timing hook (process-wide, off by default).  `events` holds
 * n_events cudaEvent_t handles created by the caller; while set, each
 * moe_layer call records events[i] on its stream right before its i-th kernel
 * launch and events[L] after the last one (L = moe_layer_launch_count), so
 * consecutive events bracket exactly one kernel.  Calls with fewer than L+1
 * events record nothing.  Pass NULL / 0 to switch it off.  Not thread-safe:
 * set it from the thread that calls moe_layer.  Returns MOE_OK. */
int moe_set_trace_events(void* const* events, int n_events);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
