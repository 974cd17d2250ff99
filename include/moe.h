/*
 * moe.h -- C ABI of the GB300 (sm_103a) routed-expert hot path.
 *
 * One call runs, on one GPU, the routed-expert layer whose caller owns the
 * activations x[T,d] (bf16), the top-k expert ids[T,k] (int32, distinct per
 * row), the routing scores[T,k] (fp32) and the expert weights W13[E,2I,d] and
 * W2[E,d,I] (bf16):
 *
 *     dispatch (expert-major permutation) -> W13 grouped GEMM -> SwiGLU
 *       -> W2 grouped GEMM x score -> deterministic combine
 *
 * and its backward (input gradients, weight gradients accumulated in place,
 * score gradients).  Sources: "Dist-MoE: Meta's Blackwell SM100 MoE Kernels"
 * (section "What it is selling": caller-owned inputs, one library-owned
 * context, the pipeline, FPROP/DGRAD/WGRAD, BF16 with FP32 accumulate, MXFP8
 * E4M3 after routing with prepared weights, plain/clamped SwiGLU, in-place
 * WGRAD; section "Caveats": fixed physical token count with zero-score padding,
 * sequentially reusable, non-reentrant contexts, fatal scratch overflow) and
 * the "nvfp4moe" README (section "Grouped GEMM": expert-major rows, m_indptr of
 * length E+1, empty experts; section "MoE layer": distinct int32 ids, fp32
 * weights, workspace overwritten by the next call, one plan per stream,
 * allocation-free warmed plans; sections "Training" and "Supported kernel
 * surface": deterministic dispatch, combine and router gradients; "Limits").
 *
 * Conventions shared by every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller unless the
 *     argument name ends in _host.  The library never frees them.
 *   - bf16 tensors are passed as void* holding IEEE bfloat16 values; all
 *     tensors are dense row-major (C order) with the shapes given.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *     Work is enqueued on it; no entry point below synchronises unless it says
 *     so.  A plan is not reentrant: use one plan per concurrent stream.
 *   - Return value: MOE_OK (0) or one of the MOE_ERR_* codes.  Argument errors
 *     are detected on the host before anything is enqueued.  Errors found by
 *     the device (bad ids, a wait that gave up) are recorded in the plan's
 *     device error word and reported by moe_plan_check().
 *   - No entry point allocates device memory after moe_plan_set_workspace();
 *     forward and backward enqueue kernels and async copies only, so they may
 *     be captured in a CUDA graph.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes -------------------------------------------------------- */
#define MOE_OK                0
#define MOE_ERR_INVALID_ARG   1  /* bad size, null pointer, misaligned pointer   */
#define MOE_ERR_WORKSPACE     2  /* workspace missing or too small               */
#define MOE_ERR_STATE         3  /* e.g. backward without a saving forward       */
#define MOE_ERR_BAD_IDS       4  /* device found an id outside [0,E) or repeated */
#define MOE_ERR_TIMEOUT       5  /* a device-side wait gave up                   */
#define MOE_ERR_CUDA          6  /* a CUDA runtime/driver call failed            */
#define MOE_ERR_UNSUPPORTED   7  /* combination not implemented                  */

/* ---- precisions ------------------------------------------------------------ */
#define MOE_PREC_BF16   0   /* bf16 operands, fp32 accumulate                     */
#define MOE_PREC_MXFP8  1   /* E4M3 operands with E8M0 scales per 32 along K      */
#define MOE_PREC_NVFP4  2   /* E2M1 operands with E4M3 scales per 16 along K and
                               per-tensor scales; inference only                   */

/* ---- workspace flags ------------------------------------------------------- */
#define MOE_WS_TRAINING     1  /* keep forward activations and backward buffers */
#define MOE_WS_HOST_STAGING 2  /* device copies of per-step host inputs/outputs  */

typedef struct moe_plan moe_plan;

/*
 * moe_plan_create -- describe one routed-expert layer.
 *   T  physical tokens per call (a fixed shape: callers with fewer tokens pad
 *      and give the padding rows zero scores -- "Caveats", item 2)
 *   d  hidden size, I expert intermediate size, E experts, k experts per token
 *   precision  MOE_PREC_BF16 or MOE_PREC_MXFP8
 * Limits ("Limits" section of the nvfp4moe README, adapted to whole tiles):
 *   d % 128 == 0, I % 64 == 0, 1 <= k <= E <= 256, T >= 1, T*k < 2^31.
 * Returns a host-side plan object (owned by the caller, free with
 * moe_plan_destroy) or NULL on invalid arguments.  Does not touch the GPU
 * except to query the current device's properties.  A plan belongs to the
 * device current at creation (its grids are sized for that device's SMs): make
 * that device current for every later call with the plan.  Plans on different
 * devices may be used from different host threads at once.
 */
moe_plan* moe_plan_create(int T, int d, int I, int E, int k, int precision);

/* Free the plan (host memory only; the caller frees its workspace). */
void moe_plan_destroy(moe_plan* plan);

/*
 * Clamped SwiGLU ("What it is selling": plain or clamped SwiGLU).  limit = 0
 * selects plain silu(gate)*up; limit > 0 clips gate and up to [-limit, limit]
 * before the activation, and the backward passes gradient only where the
 * pre-activation lies inside the closed interval.  A NaN gate or up value of a
 * plan with a limit counts as -limit, except in moe_decode_nvfp4, where it stays
 * NaN.
 */
int moe_plan_set_swiglu_clamp(moe_plan* plan, float limit);

/*
 * Bytes of device workspace the plan needs for `flags` (MOE_WS_*).  The size
 * covers the worst case of padded expert-major rows,
 *   Rpad <= T*k + E*(G-1)    (G = the plan's row granule, 128 or 256),
 * so it never depends on the routing.  Returns 0 for a NULL plan.
 */
size_t moe_plan_workspace_bytes(const moe_plan* plan, int flags);

/*
 * Hand the plan a caller-allocated device buffer (256-byte aligned) of at least
 * moe_plan_workspace_bytes(plan, flags) bytes.  The plan owns its contents from
 * now on ("MoE layer": the workspace is overwritten by the next call).  Clears
 * the device error word (a synchronous cudaMemset on the legacy stream).
 * Returns MOE_ERR_WORKSPACE if `bytes` is too small.  An NVFP4 plan also takes a
 * workspace without the scratch of moe_decode_nvfp4 at its end, which is, with n =
 * min(T, MOE_DECODE_MAX_TOKENS) * k, 4*n*I, 4*n*d and n bytes, each rounded up to 256;
 * decoding then returns MOE_ERR_WORKSPACE.
 */
int moe_plan_set_workspace(moe_plan* plan, void* workspace, size_t bytes, int flags);

/*
 * Forward.  Inputs (device):
 *   x       [T, d]  bf16         ids  [T, k] int32      scores [T, k] fp32
 *   w13     [E, 2I, d] bf16: rows [0,I) gate, [I,2I) up (not interleaved)
 *   w2      [E, d, I]  bf16
 *   For MOE_PREC_MXFP8, w13/w2 hold E4M3 codes (uint8, same shapes) and
 *   w13_sf / w2_sf their E8M0 scales in the tiled layout, both produced by
 *   moe_prepare_weights_mxfp8; for bf16 pass NULL.  An MXFP8 plan quantises
 *   the routed activation rows along d and h along I (32-element blocks) and
 *   runs block-scaled E4M3 GEMMs; it needs I % 128 == 0, d <= 4096, I <= 4096.
 *   With save_for_backward = 1 it also keeps a and the routed x rows
 *   quantised along the rows for moe_backward_mxfp8 (h is kept as its E4M3
 *   codes only; the backward recomputes the bf16 h from a).
 * Output: y [T, d] bf16, overwritten:
 *   y[t] = bf16( sum_{j=0..k-1} bf16( scores[t,j] * W2[e] . h ) ),
 *   h = bf16(silu(G) * U),  (G, U) = bf16(W13[e] . x[t]),  e = ids[t,j]
 * (sum in fixed j order).  save_for_backward = 1 keeps what moe_backward needs
 * in the workspace (requires a MOE_WS_TRAINING workspace).
 * Ids outside [0,E) or repeated within a row set MOE_ERR_BAD_IDS in the device
 * error word (detail = smallest offending flat index t*k+j); such elements are
 * dropped, so memory stays safe, but y is then not meaningful.
 */
int moe_forward(moe_plan* plan, const void* x, const int32_t* ids, const float* scores,
                const void* w13, const void* w2, const uint8_t* w13_sf, const uint8_t* w2_sf,
                void* y, int save_for_backward, void* stream);

/*
 * Forward over rows the caller has already laid out expert-major (nvfp4moe
 * README, "MoE layer": its run_routed entry takes such rows with m_indptr and
 * the padded offsets, for callers that route on their own).  Dispatch and gather are
 * skipped; the W13 GEMM + SwiGLU and the W2 GEMM run over the caller's layout,
 * and the combine runs when row_of and y are given.  Inputs (device):
 *   x_e      [rows, d] bf16: expert e's routed rows at [off_pad[e], off_pad[e] + m_e)
 *            with m_e = m_indptr[e+1] - m_indptr[e]; the rows up to off_pad[e+1]
 *            are padding (computed like routed rows; zero rows give zero outputs)
 *   m_indptr [E+1] int32: m_indptr[0] = 0, non-decreasing (exact row counts)
 *   off_pad  [E+1] int32: off_pad[0] = 0, every entry a multiple of
 *            moe_tile_rows() (128), off_pad[e+1] - off_pad[e] >= m_e,
 *            off_pad[E] <= rows
 *   score_of [rows] fp32 routing score of each row, or NULL (no score)
 *   w13, w2  as moe_forward (bf16 plans)
 *   row_of   [T, k] int32 row of x_e holding token t's j-th contribution (-1:
 *            none), or NULL
 * Outputs (device):
 *   ys [rows, d] bf16: ys[r] = bf16(score_of[r] * W2[e] . h),
 *      h = bf16(silu(G) * U), (G, U) = bf16(W13[e] . x_e[r]), for the m tiles
 *      that hold routed rows (rows in other tiles are not written)
 *   y  [T, d] bf16 (with row_of, else NULL): y[t] = bf16(sum_j ys[row_of[t,j]])
 *      in fixed j order
 * On the same layout, inputs and weights, ys and y equal those of moe_forward
 * bit for bit.  rows <= the plan's worst-case padded row count
 * (T*k + E*127 rounded down to a multiple of 128), else MOE_ERR_INVALID_ARG.
 * The layout is checked on the device: an inconsistent m_indptr / off_pad runs
 * no tile and records MOE_ERR_INVALID_ARG in the device error word (detail:
 * the first offending expert index e, 0..E); on a consistent layout a row_of
 * entry outside [0, off_pad[E]) is treated as -1 and records
 * MOE_ERR_INVALID_ARG with detail E + 1 + its flat index t*k + j.  bf16 plans
 * only (MOE_ERR_UNSUPPORTED otherwise).  The call uses the plan's workspace
 * (h, the tile list, a checked copy of row_of), so it overwrites the tables of
 * the previous call and cannot be followed by moe_backward.
 */
int moe_forward_routed(moe_plan* plan, const void* x_e, long long rows, const int32_t* m_indptr,
                       const int32_t* off_pad, const float* score_of, const void* w13,
                       const void* w2, void* ys, const int32_t* row_of, void* y, void* stream);

/*
 * Backward of the last saving forward on this plan ("What it is selling":
 * DGRAD and WGRAD; nvfp4moe "Training": router gradients).  Inputs: dy [T, d]
 * bf16 and the same w13/w2 as the forward.  Outputs:
 *   dx      [T, d]      bf16, overwritten
 *   dscores [T, k]      fp32, overwritten (gradient w.r.t. the given scores)
 *   dw13    [E, 2I, d]  fp32, ACCUMULATED in place (+=); experts with no rows
 *   dw2     [E, d, I]   fp32, ACCUMULATED in place      are left untouched
 * Returns MOE_ERR_STATE if no saving forward preceded it, MOE_ERR_UNSUPPORTED
 * for an MXFP8 plan (use moe_backward_mxfp8).
 */
int moe_backward(moe_plan* plan, const void* dy, const void* w13, const void* w2,
                 void* dx, float* dw13, float* dw2, float* dscores, void* stream);

/*
 * Backward of an MXFP8 plan ("What it is selling": MXFP8 E4M3 for FPROP, DGRAD
 * and WGRAD; nvfp4moe "Training").  Every block-scaled GEMM takes its operands
 * quantised in 32-element blocks along its own K (block rule of
 * moe_quantize_mxfp8):
 *   DGRAD-W2:  dY rows along d, W2[e]^T prepared along d         -> g
 *   DGRAD-W13: dA rows along 2I, W13[e]^T prepared along 2I       -> dX_e
 *   WGRAD-W2:  dY and hs along the rows of each expert            -> dW2[e]
 *   WGRAD-W13: dA and x along the rows of each expert             -> dW13[e]
 * (row blocks start at each expert's first padded row; the zero padding rows do
 * not change a block's scale).  Rounding points and outputs are those of
 * moe_backward: dx, dscores overwritten, dw13/dw2 accumulated in place.
 * w13t/w13t_sf and w2t/w2t_sf come from moe_prepare_weights_mxfp8_backward.
 * Needs a MOE_WS_TRAINING workspace and a saving forward (MOE_ERR_STATE
 * otherwise); MOE_ERR_UNSUPPORTED for a bf16 plan.
 */
int moe_backward_mxfp8(moe_plan* plan, const void* dy, const uint8_t* w13t,
                       const uint8_t* w13t_sf, const uint8_t* w2t, const uint8_t* w2t_sf,
                       void* dx, float* dw13, float* dw2, float* dscores, void* stream);

/*
 * One training (or, with dy_host == NULL, inference) step from HOST buffers:
 * copies x_host, ids_host, scores_host (and dy_host) into the plan's staging
 * area, runs moe_forward (+ moe_backward), and copies y (and dx, dscores) back
 * into the host buffers, all enqueued on `stream`; the caller synchronises the
 * stream before reading the host outputs.  The copies run on a plan-owned side
 * stream (created with the host-staging workspace) that joins `stream` at the
 * end of the step, overlapped with compute: x and dY upload during dispatch and
 * the forward, y downloads during the backward, dx and dscores during the
 * weight-gradient GEMMs.  After a training step on the plan, the next step's
 * uploads need not wait for that step to end (its last reads of the staged
 * inputs came before its dX combine), so in a loop of training steps they
 * overlap the previous step's weight-gradient GEMMs.  The host buffers are read
 * and written asynchronously: the caller keeps the inputs unchanged and leaves
 * the outputs alone until the stream has passed the step.  Host buffers should
 * be pinned (page-locked) for the copies to be asynchronous.  Weights and weight
 * gradients stay on the device.  Needs a MOE_WS_HOST_STAGING workspace (plus
 * MOE_WS_TRAINING when dy_host != NULL).
 */
int moe_step_host(moe_plan* plan, const void* x_host, const int32_t* ids_host,
                  const float* scores_host, const void* dy_host,
                  const void* w13, const void* w2, float* dw13, float* dw2,
                  void* y_host, void* dx_host, float* dscores_host, void* stream);

/*
 * MXFP8 block quantiser ("What it is selling": MXFP8 E4M3 with prepared
 * weights).  in [rows, K] bf16 -> codes [rows, K] E4M3, scales [rows, K/32]
 * E8M0, per 32-element block along K: X = floor(log2(amax)) - 8 clamped to
 * [-127,127], scale code X+127 (0 for an all-zero block), code =
 * E4M3(v * 2^-X) rounded to nearest even and saturated to +-448.
 * K % 32 == 0.  Used to prepare weights and exported for bit-exact tests.
 */
int moe_quantize_mxfp8(const void* in, long rows, int K, uint8_t* codes, uint8_t* scales,
                       void* stream);

/*
 * Prepared MXFP8 weights ("What it is selling": MXFP8 E4M3 accepts prepared
 * weights; nvfp4moe "Training": re-prepare after each optimizer step).
 * Quantises w13 [E,2I,d] along d and w2 [E,d,I] along I with the block rule of
 * moe_quantize_mxfp8 into
 *   w13_codes [E,2I,d], w2_codes [E,d,I]  (E4M3 bytes, same layout as the input)
 *   w13_scales, w2_scales                 (E8M0 bytes in the tiled layout the
 *                                           block-scaled GEMMs read; sizes from
 *                                           moe_mxfp8_weight_scale_bytes)
 * Tiled scale layout: rows are grouped in blocks of 128 and K in groups of 128
 * elements (four 32-element blocks); each (row block, K group) is a 512-byte
 * chunk, chunk index block*(K/128) + kb/4, in which row r = row%128 and block
 * j = kb%4 sit at byte 16*(r%32) + 4*(r/32) + j.  For W13 the row
 * blocks are, per expert, the 64 gate rows and 64 up rows of each 64-column
 * n-tile (block e*(I/64)+t holds gate rows [64t,64t+64) then up rows
 * [I+64t, I+64t+64)); for W2 they are consecutive 128-row blocks of [E*d].
 * d % 128 == 0, I % 128 == 0.
 */
size_t moe_mxfp8_weight_scale_bytes(int d, int I, int E,
                                    int which /* 0: W13, 1: W2, 2: W13^T, 3: W2^T */);
int moe_prepare_weights_mxfp8(const void* w13, const void* w2, int d, int I, int E,
                              uint8_t* w13_codes, uint8_t* w13_scales, uint8_t* w2_codes,
                              uint8_t* w2_scales, void* stream);

/*
 * Weights prepared for the MXFP8 backward (moe_backward_mxfp8): each expert's
 * matrix transposed so that the DGRAD GEMMs read it K-major, and quantised
 * along that K:
 *   w13t_codes [E, d, 2I]  W13[e]^T quantised along 2I
 *   w2t_codes  [E, I, d]   W2[e]^T  quantised along d
 * Scales in the tiled layout above with plain 128-row blocks of the transposed
 * matrices ([E*d] and [E*I] rows); sizes from moe_mxfp8_weight_scale_bytes
 * (which = 2, 3).  d % 128 == 0, I % 128 == 0.
 */
int moe_prepare_weights_mxfp8_backward(const void* w13, const void* w2, int d, int I, int E,
                                       uint8_t* w13t_codes, uint8_t* w13t_scales,
                                       uint8_t* w2t_codes, uint8_t* w2t_scales, void* stream);

/*
 * NVFP4 inference ("Dist-MoE" note, "What it is selling": the FP4 mode serves
 * inference only, with weights prepared ahead of the call; nvfp4moe README,
 * "Dense GEMM" / "Grouped GEMM": E2M1 codes two to a byte, one E4M3 scale per
 * block, one dequantisation scale per tensor, the GEMM scaled by the product of
 * its operands' tensor scales; "MoE layer": fixed activation scales from a
 * calibration pass or a checkpoint).  Block rule: a tensor with per-tensor dequantisation
 * scale s has encode scale g = 1/s; each 16-element block along K with amax A
 * gets the E4M3 scale code E4M3((A / 6) * g) and its elements
 * E2M1(v * (g / S)), S the scale's value (fp32 arithmetic, round to nearest
 * even, saturating; S = 0 gives zero codes).  Codes are packed two per byte,
 * element 2i in the low nibble.
 *
 * An NVFP4 plan (precision MOE_PREC_NVFP4; d % 256 == 0, I % 256 == 0) takes
 * only an inference workspace (flags 0; MOE_ERR_UNSUPPORTED for
 * MOE_WS_TRAINING or MOE_WS_HOST_STAGING) and runs moe_forward_nvfp4 and
 * moe_decode_nvfp4 only (moe_forward returns MOE_ERR_UNSUPPORTED).
 */

/*
 * Static activation scales of an NVFP4 plan: the per-tensor dequantisation
 * scales of the routed activation rows (x_scale) and of h (h_scale), e.g.
 * amax / (6 * 448) of calibration data (moe_amax_bf16).  Values beyond the
 * calibrated range saturate.  Both > 0 and finite (MOE_ERR_INVALID_ARG).
 */
int moe_plan_set_activation_scales(moe_plan* plan, float x_scale, float h_scale);

/*
 * Prepared NVFP4 weights: W13 [E,2I,d] quantised along d and W2 [E,d,I] along I,
 * each expert with its own dequantisation scale amax(W[e]) / (6 * 448) (1 for
 * an all-zero expert):
 *   w13_codes [E, 2I, d/2], w2_codes [E, d, I/2]   packed E2M1
 *   w13_sf, w2_sf                                  E4M3 scales, tiled: rows in
 *       blocks of 128, K in groups of 64 elements (four 16-element blocks); each
 *       (row block, K group) a 512-byte chunk, chunk index block*(K/64) + k/64,
 *       row r = row%128 and block j = (k/16)%4 at byte 16*(r%32) + 4*(r/32) + j;
 *       W13 row blocks per expert and 64-column n-tile (64 gate rows, then the
 *       same 64 up rows), W2 plain 128-row blocks of [E*d]
 *   w13_scale, w2_scale [E] fp32 (device)
 * Buffer sizes from moe_nvfp4_weight_bytes (which: 0 W13 codes, 1 W13 scales,
 * 2 W2 codes, 3 W2 scales).  d % 256 == 0, I % 256 == 0.
 */
size_t moe_nvfp4_weight_bytes(int d, int I, int E, int which);
int moe_prepare_weights_nvfp4(const void* w13, const void* w2, int d, int I, int E,
                              uint8_t* w13_codes, uint8_t* w13_sf, float* w13_scale,
                              uint8_t* w2_codes, uint8_t* w2_sf, float* w2_scale, void* stream);

/*
 * NVFP4 inference forward: x [T,d] bf16, ids, scores as moe_forward; weights
 * from moe_prepare_weights_nvfp4.  The routed x rows are quantised along d with
 * the static x scale; gate/up = bf16(alpha13 * sum) with alpha13 = x_scale *
 * w13_scale[e] (R1); h = bf16(silu(G) * U) (R2) quantised along I with the
 * static h scale; ys = bf16(s * (alpha2 * sum)), alpha2 = h_scale * w2_scale[e]
 * (R3); y = the fixed-order combine (R6).  MOE_ERR_STATE if the activation
 * scales were not set.
 */
int moe_forward_nvfp4(moe_plan* plan, const void* x, const int32_t* ids, const float* scores,
                      const uint8_t* w13_codes, const uint8_t* w13_sf, const float* w13_scale,
                      const uint8_t* w2_codes, const uint8_t* w2_sf, const float* w2_scale,
                      void* y, void* stream);

/*
 * The routed experts of a few tokens: what moe_forward_nvfp4 is for prompts, for
 * the single tokens of a decoding loop, on the same prepared weights.  The
 * activations are not quantised (no activation scales are needed): x stays bf16,
 * h is rounded to 11 significant bits (elements below 2^-28 of the largest of their
 * row: to within 2^-39 of that one), every sum is fp32, and
 *   y[t] = bf16( sum_j scores[t,j] * (w2_scale[e] * W2[e] . h) ),
 *   h = silu(G) * U, (G, U) = w13_scale[e] * W13[e] . x[t] (clipped to the plan's
 *   clamp), e = ids[t,j], in fixed j order.
 * tokens: 0 <= tokens <= min(T, MOE_DECODE_MAX_TOKENS) of the plan's T; x [tokens,
 * d] bf16, ids and scores [tokens, k], y [tokens, d] bf16 (x, y and the weights
 * 16-byte aligned).  Each chosen expert is read and converted once for every 8 of its
 * tokens, fewer where rows are wide (4 at 4096 elements).  moe_forward_nvfp4 is the faster
 * call, with k = 8, from about 56 tokens on 8 experts, 72 on 16 and 176 on 128 (d = 2048,
 * I = 768), 72 on 128 experts of d = 4096, I = 1536 and 6 on 256 experts of d = 7168, I =
 * 2048.  Bad ids are dropped and reported as
 * by moe_forward; a token's NaN or infinity stays in its own row of y.  Two launches
 * for one token of up to 8 experts, else three.  NVFP4 plans only; MOE_ERR_UNSUPPORTED
 * also where the list of tokens*k pairs (4 bytes each) and one token's row of fp16
 * do not fit in 200 KB together.  The workspace holds h and the experts' outputs of
 * the call, apart from what the other calls of the plan use.
 */
#define MOE_DECODE_MAX_TOKENS 256
int moe_decode_nvfp4(moe_plan* plan, const void* x, const int32_t* ids, const float* scores,
                     int tokens, const uint8_t* w13_codes, const uint8_t* w13_sf,
                     const float* w13_scale, const uint8_t* w2_codes, const uint8_t* w2_sf,
                     const float* w2_scale, void* y, void* stream);

/*
 * amax = max |in[i]| over n bf16 values (device pointers; amax is one fp32 on
 * the device), for calibrating static NVFP4 scales.
 */
int moe_amax_bf16(const void* in, long long n, float* amax, void* stream);

/*
 * Synchronise the device, read and clear the plan's device error word.
 * Returns MOE_OK or the first recorded device error; *detail (may be NULL)
 * receives its detail (for MOE_ERR_BAD_IDS the smallest offending flat index).
 */
int moe_plan_check(moe_plan* plan, long long* detail);

/* Human-readable name of a status code (static string). */
const char* moe_status_string(int status);

/*
 * Inspection of the plan's workspace (for tests and tools).  Returns the device
 * address and byte size of one internal tensor of the last call:
 *   MOE_BUF_M_INDPTR  int32 [E+1]    expert-major row offsets (exact counts)
 *   MOE_BUF_OFF_PAD   int32 [E+1]    row offsets with segments padded to BM
 *   MOE_BUF_ROW_OF    int32 [T*k]    padded row of element t*k+j (-1: dropped)
 *   MOE_BUF_TOKEN_OF  int32 [Rpad]   token of each padded row (-1: padding)
 *   MOE_BUF_SCORE_OF  fp32  [Rpad]   score of each padded row (0: padding)
 *   (NVFP4 plans: MOE_BUF_XQ / XSF / HQ / HSF hold packed E2M1 codes [Rpad, d/2],
 *   [Rpad, I/2] and their tiled E4M3 scales)
 *   MOE_BUF_XE        bf16  [Rpad,d] gathered activations
 *   MOE_BUF_A         bf16  [Rpad,2I] gate/up pre-activations (training)
 *   MOE_BUF_H         bf16  [Rpad,I] SwiGLU output (bf16 plans; MXFP8 plans keep
 *                                    only its E4M3 codes, MOE_BUF_HQ)
 *   MOE_BUF_YS        bf16  [Rpad,d] score-weighted expert outputs
 *   MOE_BUF_DYE       bf16  [Rpad,d] gathered upstream gradient
 *   MOE_BUF_DA        bf16  [Rpad,2I] gradient at gate/up (bf16 plans; MXFP8 plans
 *                                    keep only its E4M3 codes, MOE_BUF_DAQ / DAQT)
 *   MOE_BUF_HS        bf16  [Rpad,I] score * h, the WGRAD-W2 operand (bf16 plans;
 *                                    MXFP8 plans keep only MOE_BUF_HSQT)
 *   MOE_BUF_DXE       bf16  [Rpad,d] per-row input gradients
 * Rows are valid up to off_pad[E].  Sizes are the worst-case capacities.  A
 * tensor the plan does not hold returns MOE_ERR_WORKSPACE.
 * off_pad rounds each expert's segment up to moe_plan_row_granule(plan) rows.
 */
#define MOE_BUF_M_INDPTR 0
#define MOE_BUF_OFF_PAD  1
#define MOE_BUF_ROW_OF   2
#define MOE_BUF_TOKEN_OF 3
#define MOE_BUF_SCORE_OF 4
#define MOE_BUF_XE       5
#define MOE_BUF_A        6
#define MOE_BUF_H        7
#define MOE_BUF_YS       8
#define MOE_BUF_DYE      9
#define MOE_BUF_DA       10
#define MOE_BUF_HS       11
#define MOE_BUF_DXE      12
#define MOE_BUF_XQ       13   /* u8   [Rpad,d] E4M3 activations (MXFP8 plans) */
#define MOE_BUF_XSF      14   /* u8   tiled E8M0 scales of XQ                   */
#define MOE_BUF_HQ       15   /* u8   [Rpad,I] E4M3 h (MXFP8 plans)             */
#define MOE_BUF_HSF      16   /* u8   tiled E8M0 scales of HQ                   */
#define MOE_BUF_XQT      17   /* MXFP8 training: E4M3 [d, Rpad], routed x quantised along the rows */
#define MOE_BUF_XQTSF    18   /* its tiled scales (row blocks over d, K groups over Rpad)      */
#define MOE_BUF_DAQ      19   /* MXFP8 training: E4M3 [Rpad, 2I], dA quantised along 2I        */
#define MOE_BUF_DASF     20   /* its tiled scales (row blocks over Rpad, K groups over 2I)     */
#define MOE_BUF_DAQT     21   /* MXFP8 training: E4M3 [2I, Rpad], dA quantised along the rows  */
#define MOE_BUF_DAQTSF   22   /* its tiled scales (row blocks over 2I, K groups over Rpad)     */
#define MOE_BUF_HSQT     23   /* MXFP8 training: E4M3 [I, Rpad], hs quantised along the rows   */
#define MOE_BUF_HSQTSF   24   /* its tiled scales (row blocks over I, K groups over Rpad)      */
int moe_plan_buffer(const moe_plan* plan, int which, void** dev_ptr, size_t* bytes);

/*
 * Stage timing (for benchmarks and tools).  `events` holds caller-created
 * cudaEvent_t handles (as void*); while set, each call records them on its
 * stream at its stage boundaries:
 *   which = 0 (moe_forward, n >= 6):  [0] start, [1] after dispatch (3 launches),
 *     [2] after gather, [3] after W13+SwiGLU, [4] after W2 x score, [5] after combine
 *   which = 1 (moe_backward, n >= 7): [0] start, [1] after dY gather,
 *     [2] after DGRAD-W2 + SwiGLU backward, [3] after DGRAD-W13,
 *     [4] after dX/dscores combine, [5] after WGRAD-W2, [6] after WGRAD-W13
 * n = 0 (or events = NULL) stops recording.  The plan keeps the pointer: the
 * array must stay valid while set.  The records are "external" ones
 * (cudaEventRecordExternal), so events captured in a CUDA graph still time
 * each replay.
 */
int moe_plan_set_timing_events(moe_plan* plan, int which, void* const* events, int n);

/*
 * Failure-path testing (the pages' kernels trap on fatal conditions, see
 * "Caveats"; this library records errors instead).  wait_limit_ns > 0 makes
 * every bounded device wait of this plan's GEMM kernels give up after that many
 * nanoseconds (0 restores the default of 2 s); stall_w13 = 1 makes the MMA role
 * of the W13 GEMM wait on a barrier that nothing arrives at, so that wait runs
 * out: the kernel then records MOE_ERR_TIMEOUT (detail = the wait's site), stops
 * every role, drains its outstanding copies and MMAs with bounded waits, frees
 * its tensor memory and exits, leaving the CUDA context usable.  The outputs of
 * such a call are not meaningful.  stall_w13 = 0 restores normal operation.
 */
int moe_plan_set_debug(moe_plan* plan, long long wait_limit_ns, int stall_w13);

/*
 * Concurrent backward.  wgrad_sms > 0 makes moe_backward run the two
 * weight-gradient GEMMs (bound by the fp32 gradient traffic) on a plan-owned
 * stream, with persistent grids of wgrad_sms CTAs, while DGRAD-W13 (bound by
 * the tensor pipe and its operand loads) and the dX combine run on the
 * caller's stream on the other SMs; the caller's stream then waits for the
 * weight gradients, so the call's semantics are unchanged and the results are
 * bit-identical (every tile is computed the same way).  0 (the default)
 * launches every GEMM on every SM, one after the other.  With stage timing
 * events set, the events of the weight-gradient stages are recorded on the
 * plan's stream.  The first call with wgrad_sms > 0 creates the stream and two
 * events (no device memory).  0 <= wgrad_sms < the number of SMs, else
 * MOE_ERR_INVALID_ARG.  Applies to moe_backward and moe_backward_mxfp8.
 */
int moe_plan_set_backward_split(moe_plan* plan, int wgrad_sms);

/*
 * Weight-gradient tile order.  Each SM walks its weight-gradient tiles
 * longest expert first; a tile of a heavy expert is bound by its K loop over
 * the expert's rows and leaves DRAM idle, a tile of a light expert by the
 * read-modify-write of its fp32 gradient.  With min_rows > 0, the tiles of
 * experts with more than min_rows routed rows (padded) run in pieces on one
 * accumulator, each piece followed by a whole tile of a lighter expert on the
 * other, so that the light tiles' gradient traffic overlaps the heavy tiles'
 * K loops.  Every tile still sums its K range in the same order, so the
 * gradients are bit-identical to those of the plain order (min_rows = 0).
 * Default 2560.  min_rows < 0 or > 2^30: MOE_ERR_INVALID_ARG.  Applies to
 * moe_backward and moe_backward_mxfp8.
 */
int moe_plan_set_wgrad_interleave(moe_plan* plan, long long min_rows);

/* Number of SMs of the plan's device (the persistent kernels' grid size). */
int moe_plan_num_sms(const moe_plan* plan);

/* Number of kernels this plan has launched so far (all entry points). */
long long moe_plan_launch_count(const moe_plan* plan);

/*
 * moe_dispatch_static -- the expert-major dispatch of moe_forward (per-expert
 * histogram, prefix scan, stable scatter) for callers that cannot allocate
 * device memory: code that runs inside another framework's allocator or
 * memory-pool callbacks, hosts whose device memory is already carved into
 * fixed pools, or processes that may only touch memory they are handed.  It
 * calls no cudaMalloc, cudaFree or other allocating routine; the kernels'
 * scratch (chunk histograms, counts, tile table, error word) lives in one
 * static __device__ array of about 280 KB that every GPU loading this library
 * keeps until the process exits.  The source pages have no counterpart of this
 * entry point.
 *   ids [T,k] int32, scores [T,k] fp32                       (inputs, device)
 *   m_indptr [E+1], off_pad [E+1], row_of [T*k] int32,
 *   token_of [rows_capacity] int32, score_of [rows_capacity] fp32,
 *   status [2] int32: {MOE_OK or MOE_ERR_BAD_IDS, smallest bad flat index or -1}
 *                                                            (outputs, device)
 * Same contents as the tables moe_forward builds (see moe_plan_buffer) for a
 * plan whose row granule is 128.
 * Limits: T*k <= MOE_STATIC_MAX_ROUTED (else MOE_ERR_WORKSPACE: the static
 * scratch is too small), k <= E <= 256, rows_capacity >=
 * floor((T*k + E*(BM-1)) / BM) * BM (else MOE_ERR_INVALID_ARG).
 * The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current.  The address is kept per
 * device and CUDA context: the first call from another context on the device
 * (a non-primary context, or the primary context re-created after
 * cudaDeviceReset) looks it up again and is a first call in the same sense.  All calls on a device share the one array,
 * which keeps the last call's contents (the error word is cleared at the start
 * of each call): calls whose work overlaps on the GPU (for example on two
 * streams) race and must not be issued.
 */
#define MOE_STATIC_MAX_ROUTED 262144
int moe_dispatch_static(const int32_t* ids, const float* scores, int T, int k, int E,
                        int32_t* m_indptr, int32_t* off_pad, int32_t* row_of, int32_t* token_of,
                        float* score_of, long long rows_capacity, int32_t* status, void* stream);

/* Rows per GEMM m tile (128). */
int moe_tile_rows(void);

/*
 * Row GEMMs on CTA pairs.  on = 1 runs W13, W2 and DGRAD-W13 of a bf16 plan on
 * pairs of CTAs of a thread-block cluster with 256 x 256 tiles (tcgen05
 * cta_group::2), each CTA reading a third less operand data per product: the
 * 128-row m tiles of each expert go to the pair kernel two at a time, and an
 * expert's odd last m tile to the one-CTA kernel (dispatch builds both lists),
 * so expert segments stay padded to 128 rows.  DGRAD-W2 stays on one CTA.
 * Must be called before moe_plan_workspace_bytes / moe_plan_set_workspace
 * (MOE_ERR_STATE afterwards); needs d % 256 == 0 and I % 256 == 0 (else
 * MOE_ERR_UNSUPPORTED).
 */
int moe_plan_set_cta_pairs(moe_plan* plan, int on);

/* Padding granule of this plan's expert segments (off_pad): 128. */
int moe_plan_row_granule(const moe_plan* plan);

/*
 * Dense bf16 GEMM through the same tcgen05 kernels (for tests):
 *   mode 0: C[M,N] bf16  = A[M,K] . B[N,K]^T      (both operands K-major)
 *   mode 1: C[M,N] bf16  = A[M,K] . B[K,N]        (B MN-major)
 *   mode 2: C[M,N] fp32 += A[K,M]^T . B[K,N]      (both operands MN-major)
 *   mode 3: as mode 0 on CTA pairs (256 x 256 tiles, M % 256 == N % 256 == 0)
 *   mode 4: as mode 1 on CTA pairs
 * M % 128 == 0, N % 64 == 0, K % 64 == 0 (mode 2: K % 128 == 0).  `scratch`
 * is a device buffer of moe_gemm_scratch_bytes(M, K) bytes for the tile tables.
 */
size_t moe_gemm_scratch_bytes(int M, int K);
int moe_gemm_bf16(int mode, const void* A, const void* B, void* C, int M, int N, int K,
                  void* scratch, void* stream);

/* ---- element types of the entry points that take one ------------------------ */
#define MOE_DTYPE_BF16  0
#define MOE_DTYPE_FP32  1

/*
 * Router: top-k expert ids and scores from logits, per-expert counts, the balance
 * and z losses, and their gradient.  It makes the ids and scores that moe_forward
 * takes, and takes the dscores that moe_backward makes.
 *   E experts (1..256), k of them per token (1..E)
 *   dtype    MOE_DTYPE_* of the logits and of their gradient
 *   scoring  how the scores follow from the logits l of the chosen experts:
 *     MOE_ROUTER_SOFTMAX_TOPK  softmax over the chosen
 *     MOE_ROUTER_SOFTMAX       their share of the softmax over all experts
 *     MOE_ROUTER_SIGMOID       sigmoid(l), divided by the chosen experts' sum
 *   scale    factor on the scores (finite)
 */
#define MOE_ROUTER_SOFTMAX_TOPK 0
#define MOE_ROUTER_SOFTMAX      1
#define MOE_ROUTER_SIGMOID      2
typedef struct moe_router_desc {
  int E, k;
  int dtype;
  int scoring;
  float scale;
} moe_router_desc;

/*
 * Bytes of device workspace for T tokens (0 for an invalid description).  It is
 * scratch: its contents mean nothing before or after a call.  Calls that may
 * overlap on the GPU need one each.
 */
size_t moe_router_workspace_bytes(const moe_router_desc* desc, int T);

/*
 * Router forward.  Inputs (device):
 *   logits      [T, E] of dtype, rows ld elements apart (ld >= E)
 *   bias        [E] fp32 or NULL: added to the logits (in fp32) for the choice
 *               only; scores and probabilities do not see it
 *   token_mask  [T] uint8 or NULL: 0 marks a padding token, whose logits are not
 *               read; it gets the ids (t*k + j) % E and scores 0
 * Outputs (device, overwritten):
 *   ids       [T, k] int32: the k largest of l + bias, largest first, ties to the
 *             lowest index; a NaN ranks below every number
 *   scores    [T, k] fp32
 *   counts    [E+1] int32: how often each expert was chosen, and in counts[E] the
 *             number of live tokens
 *   prob_sum  [E] fp32: sum over live tokens of p, the softmax over all experts
 *             (MOE_ROUTER_SIGMOID: sigmoid(l) divided by its sum over all experts)
 *   losses    [2] fp32: balance = E / (k N^2) * sum_e counts[e] * prob_sum[e] (N =
 *             counts[E]; 1 when perfectly balanced) and z = mean of
 *             logsumexp(l)^2 (0 for MOE_ROUTER_SIGMOID)
 *   row_stat  [T] fp32: logsumexp(l), or for MOE_ROUTER_SIGMOID the logarithm of
 *             the sum of the sigmoids; what moe_router_backward needs of the forward
 * A token is live when it is not padding and some logit is above -inf.  A logit of
 * -inf switches its expert off: it is chosen only when nothing else is left, with
 * score 0 and without being counted.  A row of -inf only has scores 0 and row_stat
 * -inf, as padding has.  NaN and +inf logits give NaN
 * where the formulas do.  Sums run in a fixed order, so results repeat bit for bit.
 * Exponentials are the hardware's: a score, probability or gradient term whose logit
 * lies D below the row's largest errs by up to 4 D 2^-24 of itself, on top of 2^-18
 * at most.
 * T >= 0, T*k < 2^31; T = 0 writes counts, prob_sum and losses as zeros.
 */
int moe_router_forward(const moe_router_desc* desc, int T, const void* logits, long long ld,
                       const float* bias, const uint8_t* token_mask, int32_t* ids,
                       float* scores, int32_t* counts, float* prob_sum, float* losses,
                       float* row_stat, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Router backward: the gradient of
 *   sum d_scores * scores + d_losses[0] * balance + d_losses[1] * z
 * with respect to the logits (the choice and the counts are constants).  logits,
 * ids, counts and row_stat are the forward's; d_scores [T, k] fp32 (dscores of
 * moe_backward) and d_losses [2] fp32 (device) may each be NULL for zeros.
 *   d_logits  [T, E] of dtype, rows ld_d elements apart, overwritten; rows of
 *             tokens that are not live become 0.  May be logits itself (same ld).
 */
int moe_router_backward(const moe_router_desc* desc, int T, const void* logits, long long ld,
                        const int32_t* ids, const int32_t* counts, const float* row_stat,
                        const float* d_scores, const float* d_losses, void* d_logits,
                        long long ld_d, void* stream);

/*
 * The norms around a block with its gate and residual scale.  On rows of d
 * elements, with rms(v) = sqrt(mean(v^2) + eps):
 *   n   = y / rms(y) * w_post             (n = y where w_post is NULL)
 *   out = residual + alpha * gate * n
 *   u   = out / rms(out) * w_pre
 * y is the block's output (as y of moe_forward), out the residual stream after it
 * and u the next block's input.  y = NULL leaves the first two lines out (u is the
 * norm of residual); u = w_pre = NULL leaves the last one out.
 *   d               row width, 1..16384
 *   dtype           MOE_DTYPE_* of y, u and their gradients
 *   residual_dtype  of the residual stream and its gradients (MOE_DTYPE_FP32 if
 *                   dtype is)
 *   param_dtype     of w_post, w_pre and gate (their gradients are fp32)
 *   gate            MOE_GATE_NONE, MOE_GATE_CHANNEL (gate [d]) or MOE_GATE_TOKEN
 *                   (gate [T])
 *   alpha           the residual scale
 * Arithmetic is fp32, rounded once on the way out; u follows from the unrounded
 * out.  Every [T, d] tensor comes with the distance of its rows in elements
 * (ld >= d) and needs no alignment beyond its elements' (16-byte aligned rows of a
 * width that 8 divides run faster).
 */
#define MOE_GATE_NONE    0
#define MOE_GATE_CHANNEL 1
#define MOE_GATE_TOKEN   2
typedef struct moe_block_norm_desc {
  int d;
  int dtype, residual_dtype, param_dtype;
  int gate;
  float alpha, eps;
} moe_block_norm_desc;

/* Bytes of scratch moe_block_norm_backward needs for T rows (0 if desc is invalid). */
size_t moe_block_norm_workspace_bytes(const moe_block_norm_desc* desc, int T);

/*
 * Forward.  residual_out (needed with y) may be residual itself and u may be y
 * itself (same ld).  gate is given exactly when desc->gate is not MOE_GATE_NONE
 * and y is given; w_pre exactly when u is.  T >= 0.
 */
int moe_block_norm_forward(const moe_block_norm_desc* desc, int T, const void* residual,
                           long long ld_residual, const void* y, long long ld_y,
                           const void* w_post, const void* gate, const void* w_pre,
                           void* residual_out, long long ld_out, void* u, long long ld_u,
                           void* stream);

/*
 * Backward.  residual_out is the stream after the block (for y = NULL: the
 * residual that was normed), y, w_post, gate, w_pre as in the forward; the row
 * statistics are computed again, nothing is kept from the forward.
 *   d_residual_out  [T, d] gradient at residual_out from what reads it later, or
 *                   NULL for zeros
 *   d_u             [T, d] gradient at u, or NULL with w_pre = NULL
 * Outputs:
 *   d_residual  [T, d] gradient at residual, overwritten (may be d_residual_out)
 *   dy          [T, d] gradient at y, overwritten (may be d_u), or NULL
 *   dw_post [d], dw_pre [d], dgate [d] or [T]: fp32, overwritten, or added to with
 *               accumulate = 1; each may be NULL
 * Sums over rows run in a fixed order.  workspace: 16-byte aligned, at least
 * moe_block_norm_workspace_bytes(desc, T); calls that may overlap need one each.
 */
int moe_block_norm_backward(const moe_block_norm_desc* desc, int T, const void* residual_out,
                            long long ld_out, const void* y, long long ld_y,
                            const void* d_residual_out, long long ld_dout, const void* d_u,
                            long long ld_du, const void* w_post, const void* gate,
                            const void* w_pre, void* d_residual, long long ld_dres, void* dy,
                            long long ld_dy, float* dw_post, float* dgate, float* dw_pre,
                            int accumulate, void* workspace, size_t workspace_bytes,
                            void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_GB300_H */
