/*
 * cq.h -- C ABI of the MI355X (gfx950) library for exact minimax FP16
 * group-scale selection in symmetric 4-bit, group-size-128 weight
 * quantization, and GPTQ-v1 packing of the result.
 *
 * The operation (CliffQuant repository README, "What CliffQuant changes",
 * displayed objective and the paragraph after it): for one group of 128
 * weights w_i and E environment diagonals d_{e,i} >= 0, choose the positive
 * finite IEEE binary16 scale s (bit patterns 0x0001..0x7BFF, 31,743 values)
 * that minimises
 *        F(s) = max_e sum_i d_{e,i} (w_i - s q_i(s))^2,
 *        q_i(s) = clip(round-half-even(w_i / s), -8, 7)   (round, then clip),
 * an exact objective tie going to the lower binary16 bit pattern.  The
 * quotient w_i/s is taken as one correctly rounded binary32 division and the
 * reported objective is summed in binary64, i = 0..127 in order, each
 * operation rounded on its own.
 *
 * Conventions for every entry point:
 *  - Array arguments are DEVICE pointers (HIP global memory on the current
 *    device) owned by the caller; the library never frees or keeps them.
 *  - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *    Calls are asynchronous on that stream and return after enqueueing; the
 *    outputs are valid once the stream has reached that point.
 *  - No entry point allocates device memory: scratch space comes from the
 *    caller's `workspace` (device memory, 256-byte aligned, at least
 *    cq_workspace_size(...) bytes, not shared between calls that may overlap).
 *  - Pointers to float32 inputs (w, d) and to int8 codes must be 16-byte
 *    aligned, other arrays naturally aligned (torch allocations are).
 *  - Argument errors are reported before anything is enqueued; data errors
 *    (non-finite weights or diagonals, negative diagonals) are reported per
 *    group through CQ_FLAG_BAD_INPUT, never through the status.
 *  - The library keeps no state between calls; distinct streams may be used
 *    from distinct host threads at once.
 *
 * Layouts:
 *   w      float32 [n_groups][128]   group g: 128 consecutive input channels
 *                                    of one output row (row-major [out][in]
 *                                    matrices give g = row*(in/128) + chunk).
 *   d      float32 [n_d][E][128]     group g uses slice (g % d_period); a
 *                                    matrix has d_period = in/128 (groups
 *                                    inherit the diagonals of their input
 *                                    channels), per-group diagonals have
 *                                    d_period = n_groups.
 *   scales uint16  [n_groups]        binary16 bit patterns (0x0001..0x7BFF).
 *   codes  int8    [n_groups][128]   q_i in [-8, 7] at the chosen scale.
 */
#ifndef CQ_H
#define CQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define CQ_ABI_VERSION 2
#define CQ_GROUP 128
#define CQ_MAX_GROUP 256 /* longest group cq_quantize_groups_spec takes */
#define CQ_MAX_ENVS 32
#define CQ_MAX_POLICIES 64
#define CQ_MAX_BOOT (1 << 20)

/* Status codes. */
#define CQ_OK 0
#define CQ_EINVAL (-1)       /* null required pointer, bad size or enum */
#define CQ_EWORKSPACE (-2)   /* workspace missing, misaligned or too small */
#define CQ_EHIP (-3)         /* a HIP launch failed (hipGetLastError) */
#define CQ_EUNSUPPORTED (-4) /* valid arguments this entry point does not serve */
#define CQ_ELIMIT (-5)       /* more groups than cq_quantize_groups_noalloc's fixed scratch holds */

/* Solvers (cq_quantize_groups `method`); all three return the same result.
 *  CQ_EXHAUSTIVE  the independent full-grid enumerator (README, "What CliffQuant changes": a
 *                 separate reference evaluates every one of the 31,743 binary16 values): the
 *                 binary32 objective of every weight at every scale, then binary64 rescoring of
 *                 every scale its error bound cannot rule out.  No scale is skipped.
 *  CQ_CANDIDATE   the production solver's idea (same section): candidates from code transitions,
 *                 quadratic vertices and environment intersections; groups whose direct
 *                 candidates tie exactly go to CQ_BOUNDED (CQ_EXHAUSTIVE for another quantizer;
 *                 README and model card, "Verification").
 *  CQ_BOUNDED     branch and bound over the grid: stops at the first scale >= 2 max|w| (every
 *                 larger one ties with it exactly and loses to it), takes chunk-constant codes in
 *                 closed form and skips chunks of scales whose proven lower bound exceeds the
 *                 best value screened; the outputs are those of the full grid. */
#define CQ_EXHAUSTIVE 0
#define CQ_CANDIDATE 1
#define CQ_BOUNDED 2

/* Baseline policies (cq_baseline_scales `which`), the two the pages compare the minimax
 * scales with (CliffQuant README, the opening question and the "Held-out reconstruction
 * proxy" table; model card, "Held-out reconstruction proxy"):
 *  CQ_ABSMAX       the matched AbsMax checkpoint's scale, s = fp16(fl32(max_i |w_i| / 7));
 *                  0 -> 0x0001, overflow -> 0x7BFF.
 *  CQ_POOLED_WMSE  the environments averaged before the scale is chosen: minimise
 *                  P(s) = (1/E) sum_e F_e(s) over the same grid with the same tie rule. */
#define CQ_ABSMAX 0
#define CQ_POOLED_WMSE 1

/* Per-group flag bits (cq_quantize_groups `flags`). */
#define CQ_FLAG_BAD_INPUT 1u  /* non-finite w or d, or d < 0: scale 0, codes 0, objective NaN */
#define CQ_FLAG_NEAR_TIE 2u   /* more than one scale survived the binary32 screen */
#define CQ_FLAG_EXACT_TIE 4u  /* the winner's binary64 objective equals another scale's */
#define CQ_FLAG_FALLBACK 8u   /* the candidate solver handed the group to the exhaustive one */
#define CQ_FLAG_FP64_SWEEP 16u /* decided by a full binary64 sweep (screen inconclusive) */

/* ABI version of the loaded library (CQ_ABI_VERSION). */
int32_t cq_abi_version(void);

/* Static description of a status code. */
const char *cq_status_string(int32_t status);

/* Bytes of workspace cq_quantize_groups (and cq_quantize_groups_spec) needs for
 * `method`, E and n_groups (any group length); CQ_EXHAUSTIVE and CQ_BOUNDED
 * return the same size, which is also what cq_baseline_scales with
 * CQ_POOLED_WMSE needs.  Returns 0 for invalid arguments. */
size_t cq_workspace_size(int32_t method, int32_t E, int64_t n_groups);

/*
 * Minimax scale, codes and objective for n_groups groups.
 *   method       CQ_EXHAUSTIVE, CQ_CANDIDATE or CQ_BOUNDED; all return the same result.
 *   scales       out, required.
 *   codes        out, nullable.
 *   objective    out, nullable: F(s) at the chosen scale, binary64.
 *   flags        out, nullable: CQ_FLAG_* bits.
 *   pooled_scales / pooled_objective
 *                out, nullable, CQ_EXHAUSTIVE only (else CQ_EUNSUPPORTED):
 *                the pooled-WMSE policy decided in the same sweep.
 * E in 1..32, n_groups >= 0 (0 enqueues nothing), 1 <= d_period.
 * The binary32 screen is followed by binary64 rescoring of every scale the
 * screen's error bound cannot rule out, so the pick equals the binary64
 * argmin over all scales with the lower-bit-pattern tie rule.
 */
int32_t cq_quantize_groups(const float *w, const float *d, int64_t d_period, int32_t E,
                           int64_t n_groups, int32_t method,
                           uint16_t *scales, int8_t *codes, double *objective, uint8_t *flags,
                           uint16_t *pooled_scales, double *pooled_objective,
                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * cq_quantize_groups for another quantizer (CliffQuant README, "Use the solver": the
 * solver takes a quantizer specification with qmin and qmax and a group of any length,
 * its example four weights): codes q_i = clip(round-half-even(w_i / s), qmin, qmax),
 * groups of group_len weights.
 *   w      float32 [n_groups][group_len], 4-byte aligned.
 *   d      float32 [n_d][E][group_len], 4-byte aligned; group g uses slice g % d_period.
 *   codes  out, nullable, int8 [n_groups][group_len].
 * 1 <= group_len <= CQ_MAX_GROUP, -128 <= qmin <= 0 <= qmax <= 127, qmin < qmax (else
 * CQ_EINVAL).  (128, -8, 7) is cq_quantize_groups itself, with its alignment rules.  Any
 * other quantizer is served by CQ_EXHAUSTIVE, and by CQ_CANDIDATE when group_len <= 128 and
 * -8 <= qmin, qmax <= 8 (its tied groups then go to CQ_EXHAUSTIVE, flag CQ_FLAG_FALLBACK;
 * pooled outputs CQ_EUNSUPPORTED); other methods and quantizers return CQ_EUNSUPPORTED.
 * Other outputs, workspace and errors as for cq_quantize_groups.
 */
int32_t cq_quantize_groups_spec(const float *w, const float *d, int32_t group_len, int32_t qmin, int32_t qmax,
                                int64_t d_period, int32_t E, int64_t n_groups, int32_t method,
                                uint16_t *scales, int8_t *codes, double *objective, uint8_t *flags,
                                uint16_t *pooled_scales, double *pooled_objective,
                                void *workspace, size_t workspace_bytes, void *stream);

/*
 * cq_quantize_groups for callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same arguments without
 * the workspace, and the same results.  The scratch space lives in a fixed array of the library
 * on each GPU (about 12.6 MB, held until the process ends), found at the first call on that
 * device; the call itself allocates nothing.
 *   n_groups  0..CQ_NOALLOC_MAX_GROUPS, else CQ_ELIMIT before anything is enqueued.
 * Every call on one GPU uses that GPU's one array; the kernels clear what must start at zero,
 * but calls that overlap on one GPU (other streams, other host threads) race.
 */
#define CQ_NOALLOC_MAX_GROUPS (1 << 20)
int32_t cq_quantize_groups_noalloc(const float *w, const float *d, int64_t d_period, int32_t E,
                                   int64_t n_groups, int32_t method,
                                   uint16_t *scales, int8_t *codes, double *objective, uint8_t *flags,
                                   uint16_t *pooled_scales, double *pooled_objective, void *stream);

/*
 * Baseline scale policies.
 *   CQ_ABSMAX       d may be NULL when objective is NULL; no workspace needed.
 *   CQ_POOLED_WMSE  the argmin of P(s) over every scale (the CQ_BOUNDED search of P);
 *                   workspace as for cq_workspace_size(CQ_EXHAUSTIVE, E, n_groups).
 *   objective  nullable: for CQ_ABSMAX the worst-environment objective F at
 *              the AbsMax scale; for CQ_POOLED_WMSE the pooled objective P.
 */
int32_t cq_baseline_scales(const float *w, const float *d, int64_t d_period, int32_t E,
                           int64_t n_groups, int32_t which,
                           uint16_t *scales, int8_t *codes, double *objective,
                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * cq_baseline_scales for another quantizer (CliffQuant README, "Use the solver": the solver takes
 * a quantizer specification; the baselines as in cq_baseline_scales).  w is [n_groups][group_len],
 * d [n_d][E][group_len]; codes in [qmin, qmax] as for cq_quantize_groups_spec.
 *   CQ_ABSMAX       s = fp16(fl32(max_i |w_i| / qmax)), 0 -> 0x0001, overflow -> 0x7BFF (the
 *                   largest magnitude maps to the largest positive code, as max|w| / 7 does for
 *                   [-8, 7]); needs qmax >= 1, else CQ_EINVAL.  workspace unused.
 *   CQ_POOLED_WMSE  the pooled policy of the full-grid search (cq_quantize_groups_spec's pooled
 *                   outputs alone); workspace as cq_workspace_size(CQ_EXHAUSTIVE, E, n_groups).
 * codes (nullable) are those of the chosen scale; objective (nullable) max_e F_e (AbsMax) or
 * (1/E) sum_e F_e (pooled), binary64.  Limits as for cq_quantize_groups_spec; w and d 4-byte
 * aligned.  The pages' quantizer (group_len 128, [-8, 7]) is cq_baseline_scales itself, with its
 * alignment rules.
 */
int32_t cq_baseline_scales_spec(const float *w, const float *d, int32_t group_len, int32_t qmin, int32_t qmax,
                                int64_t d_period, int32_t E, int64_t n_groups, int32_t which, uint16_t *scales,
                                int8_t *codes, double *objective, void *workspace, size_t workspace_bytes,
                                void *stream);

/*
 * GPTQ-v1 packing of one [out][in] matrix (Qwen3.5-0.8B-Base-CliffQuant-
 * W4A16-G128 model card, "Quantization configuration": GPTQ v1, 4-bit,
 * group size 128, symmetric).
 *   codes       int8 [out][in], values in [-8, 7] (the cq_quantize_groups
 *               codes of the matrix's groups, in group order).
 *   grp_scales  uint16 [out][in/128] (the matrix's per-group scales).
 *   qweight     out, int32 [in/8][out]: nibble j (bits 4j..4j+3) of
 *               qweight[r][o] is codes[o][8r+j] + 8.
 *   scales      out, uint16 [in/128][out]: scales[c][o] = grp_scales[o][c].
 * out >= 0, in >= 0, in % 128 == 0.  Codes outside [-8, 7] are packed
 * modulo 16 (the caller guarantees the range).
 */
int32_t cq_pack_gptq_v1(const int8_t *codes, const uint16_t *grp_scales, int64_t out, int64_t in,
                        int32_t *qweight, uint16_t *scales, void *stream);

/*
 * GPTQ-v1 packing of one [out][in] matrix for another quantizer (CliffQuant README, "Use the
 * solver": the solver takes a quantizer specification; the model card's format, "Quantization
 * configuration", with the field width and the group length as parameters).
 *   codes       int8 [out][in], values in [-2^(bits-1), 2^(bits-1) - 1].
 *   grp_scales  uint16 [out][in/group_len] (binary16 bit patterns).
 *   qweight     out, int32 [in*bits/32][out]: field j (bits j*bits .. j*bits + bits - 1, low
 *               field first) of qweight[r][o] is codes[o][(32/bits) r + j] + 2^(bits-1).
 *   scales      out, uint16 [in/group_len][out]: scales[c][o] = grp_scales[o][c].
 * bits in {2, 4, 8}; 1 <= group_len <= CQ_MAX_GROUP; out >= 0, in >= 0, in a multiple of
 * group_len and of 32/bits; else CQ_EINVAL (bits = 4 with group_len = 128 gives what
 * cq_pack_gptq_v1 gives).  Codes outside the range are packed modulo 2^bits (the caller
 * guarantees the range).  codes and qweight 4-byte aligned, grp_scales and scales 2-byte.
 * Two launches on `stream`.
 */
int32_t cq_pack_gptq_v1_spec(const int8_t *codes, const uint16_t *grp_scales, int64_t out, int64_t in,
                             int32_t bits, int32_t group_len, int32_t *qweight, uint16_t *scales, void *stream);

/*
 * GPTQ-v1 packing of n_mats matrices in one launch (model card, "Verification": the packed
 * checkpoint holds 150 module-buffer sets, each unpacked again; "Quantization configuration":
 * GPTQ v1, 4-bit, group size 128, symmetric).  Matrix k has shape outs[k] x ins[k]; every array
 * holds the matrices back to back in order, each block exactly what cq_pack_gptq_v1 takes or
 * writes for that matrix alone:
 *   codes       int8 [sum_k outs[k] * ins[k]], matrix k from offset sum_{j<k} outs[j] * ins[j].
 *   grp_scales  uint16, matrix k from offset sum_{j<k} outs[j] * ins[j] / 128.
 *   qweight     out, int32, matrix k's [ins[k]/8][outs[k]] from offset sum_{j<k} outs[j] * ins[j] / 8.
 *   scales      out, uint16, matrix k's [ins[k]/128][outs[k]] from offset sum_{j<k} outs[j] * ins[j] / 128.
 *   outs, ins   HOST int64 arrays [n_mats], read before the call returns.
 * 0 <= n_mats <= CQ_MAX_PACK_MATRICES; every ins[k] a multiple of 128 (ins[k] / 128 <= 65535);
 * shapes below 2^31 each and 2^46 elements in all; else CQ_EINVAL.  Alignment as for
 * cq_pack_gptq_v1.
 */
#define CQ_MAX_PACK_MATRICES 256
int32_t cq_pack_gptq_v1_multi(const int8_t *codes, const uint16_t *grp_scales, int32_t n_mats,
                              const int64_t *outs, const int64_t *ins, int32_t *qweight, uint16_t *scales,
                              void *stream);

/*
 * Module-macro worst-environment weighted MSE (Qwen3.5-0.8B-Base-CliffQuant-
 * W4A16-G128 model card, "Held-out reconstruction proxy"; CliffQuant README,
 * "Held-out reconstruction proxy").
 *   per group  p_g = max_e (1/128) sum_i d_eval_{e,i} (w_i - s_g q_i(s_g))^2
 *   per module mean of p_g over groups [module_offsets[m], module_offsets[m+1])
 *   macro      mean over the n_modules module means.
 *   scales          device uint16 [n_groups] binary16 patterns (0x0001..0x7BFF).
 *   module_offsets  device int64 [n_modules+1], non-decreasing, first 0, last
 *                   n_groups; a module whose range is empty or out of bounds
 *                   gets NaN.
 *   module_mean     out, double [n_modules].   macro  out, double [1].
 *   per_group       out, nullable, double [n_groups].
 * workspace: cq_proxy_workspace_size(n_groups) bytes.
 */
size_t cq_proxy_workspace_size(int64_t n_groups);
int32_t cq_proxy_worst_env_wmse(const float *w, const float *d_eval, int64_t d_period, int32_t E,
                                int64_t n_groups, const uint16_t *scales,
                                const int64_t *module_offsets, int32_t n_modules,
                                double *module_mean, double *macro, double *per_group,
                                void *workspace, size_t workspace_bytes, void *stream);

/*
 * The same proxy for n_policies scale policies of the same groups in one call
 * (the model card compares the minimax scales with the AbsMax baseline on this
 * proxy: Qwen3.5-0.8B-Base-CliffQuant-W4A16-G128 model card, "Held-out
 * reconstruction proxy"); w and d_eval are read once for all of them, and each
 * policy's results equal those of a cq_proxy_worst_env_wmse call on its own
 * scales bit for bit.
 *   scales       device uint16 [n_policies][n_groups].
 *   module_mean  out, double [n_policies][n_modules].
 *   macro        out, double [n_policies].
 *   per_group    out, nullable, double [n_policies][n_groups].
 * 1 <= n_policies <= CQ_MAX_POLICIES.  workspace (only when per_group is
 * NULL): cq_proxy_workspace_size(n_policies * n_groups) bytes.
 */
int32_t cq_proxy_worst_env_wmse_multi(const float *w, const float *d_eval, int64_t d_period, int32_t E,
                                      int64_t n_groups, int32_t n_policies, const uint16_t *scales,
                                      const int64_t *module_offsets, int32_t n_modules,
                                      double *module_mean, double *macro, double *per_group,
                                      void *workspace, size_t workspace_bytes, void *stream);

/*
 * cq_proxy_worst_env_wmse_multi for another quantizer (CliffQuant README, "Use the solver": a
 * quantizer specification; the proxy as in cq_proxy_worst_env_wmse, with 1/group_len for the
 * pages' 1/128: the mean over the group's weights).  w is [n_groups][group_len], d_eval
 * [n_d][E][group_len]; codes in [qmin, qmax].  Arguments, limits and workspace as for
 * cq_proxy_worst_env_wmse_multi (w and d_eval 4-byte aligned); the pages' quantizer is
 * cq_proxy_worst_env_wmse_multi itself, with its alignment rules.  Per-group sums run over the group's 16 lanes (each lane's weights in index order, then a
 * fixed butterfly): within rounding of the sequential definition, bit-identical across runs.
 */
int32_t cq_proxy_worst_env_wmse_multi_spec(const float *w, const float *d_eval, int32_t group_len, int32_t qmin,
                                           int32_t qmax, int64_t d_period, int32_t E, int64_t n_groups,
                                           int32_t n_policies, const uint16_t *scales,
                                           const int64_t *module_offsets, int32_t n_modules, double *module_mean,
                                           double *macro, double *per_group, void *workspace,
                                           size_t workspace_bytes, void *stream);

/*
 * W4A16 matmul over the GPTQ-v1 tensors, the consumer check of the packed
 * output (Qwen3.5-0.8B-Base-CliffQuant-W4A16-G128 model card, "Quantization
 * configuration": GPTQ v1, 4 bits, group 128, symmetric, 16-bit activations).
 *   x        device uint16 [M][in]: bfloat16 bit patterns, 16-byte aligned.
 *   qweight  device int32 [in/8][out], scales device uint16 [in/128][out]
 *            (binary16 bit patterns): the cq_pack_gptq_v1 outputs.
 *   y        out, float [M][out]: y[m][o] = sum_g s[g][o] sum_{k in g}
 *            x[m][k] (u[k][o] - 8), each group's sum in fp32 on the matrix
 *            cores (exact products), then one fp32 fma with its scale.
 * in a multiple of 128; M up to 64 * 65535; M == 0 or out == 0 enqueues nothing.
 */
int32_t cq_w4a16_matmul(const uint16_t *x, const int32_t *qweight, const uint16_t *scales, int64_t M,
                        int64_t out, int64_t in, float *y, void *stream);

/*
 * Running the packed checkpoint: the linear layer over the GPTQ-v1 tensors, the paged key/value
 * cache and the attention that reads it (model card, "Quantization configuration": 16-bit
 * activations; "Calibration and evaluation data": windows of 256 tokens, which these operators
 * carry through layers that are quantized already).  The conventions above hold: device pointers,
 * the caller's stream and workspace, argument errors before anything is enqueued.  Strides and
 * leading dimensions are in elements.
 */

/* Element types. */
#define CQ_BF16 0
#define CQ_F16 1
#define CQ_F32 2

/* Activations: max(z, 0); z / (1 + e^-z); z (1 + erf(z / sqrt 2)) / 2; and its tanh form
 * z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2. */
#define CQ_ACT_NONE 0
#define CQ_ACT_RELU 1
#define CQ_ACT_SILU 2
#define CQ_ACT_GELU 3
#define CQ_ACT_GELU_TANH 4

/*
 * Linear layer over the GPTQ-v1 tensors with its epilogue:
 *        z[m][c] = sum_g s[g][c] sum_{k in g} x[m][k] (u[k][c] - 8) + bias[c],
 *        y[m][o] = act(z[m][o]) + residual[m][o]                        (gated = 0)
 *        y[m][o] = act(z[m][o]) z[m][out + o] + residual[m][o]          (gated = 1)
 * the products exact and summed in fp32 on the matrix cores, the groups' scales applied in fp32, the
 * epilogue in fp32 and one rounding into y's type.  (Sums may be held divided by a group's scale:
 * below 2^100 in magnitude, nothing overflows that fp32 can hold.)
 *   x         x_type (CQ_BF16 or CQ_F16) [M] rows of `in`, ldx apart; 16-byte aligned, ldx a
 *             multiple of 8.
 *   qweight   int32 [in/8][cols], scales uint16 [in/128][cols] binary16 bits, as packed by
 *             cq_pack_gptq_v1; cols = out, or 2 out when gated (the gate's out columns first).
 *   bias      nullable, x_type [cols].
 *   residual  nullable, x_type [M] rows of `out`, ldr apart; it may be y itself where both have
 *             the same type and leading dimension.
 *   y         out, y_type (x_type or CQ_F32) [M] rows of `out`, ldy apart.
 * in a positive multiple of 128; cols < 2^31, in <= 2^24, M < 2^31; M == 0 or out == 0 enqueues
 * nothing.
 */
int32_t cq_w4a16_linear(const void *x, int64_t ldx, int32_t x_type, const int32_t *qweight, const uint16_t *scales,
                        const void *bias, const void *residual, int64_t ldr, int32_t activation, int32_t gated,
                        int64_t M, int64_t out, int64_t in, void *y, int64_t ldy, int32_t y_type, void *stream);

/*
 * Block tables and slot maps of a paged cache, built on the GPU from the requests' lengths.
 * Pages hold page_size tokens.  Request r holds ctx_len[r] tokens in the pages
 * block_table[r][0 .. ceil(ctx_len[r] / page_size)) and receives new_len[r] more.  In request order,
 * each takes the pages it needs beyond those from the end of the list free_pages[0 .. n_free), in
 * block order.  A request whose lengths are negative, or longer than max_pages pages, is invalid
 * (status 2) and takes nothing; from the first valid request on whose pages or tokens no longer
 * fit (n_free pages, max_tokens tokens), valid requests are refused (status 1).
 *   ctx_len, new_len  int32 [n_requests].
 *   free_pages        int32 [free_capacity]; n_free int32 [1] (clamped to 0 .. free_capacity).
 *   block_table       int32 rows of max_pages, table_stride apart; in and out: the entries of the
 *                     pages taken are written, the others kept.
 *   cu_q              out, int32 [n_requests + 1]: prefix sums of the new tokens served.
 *   kv_len            out, int32 [n_requests]: ctx_len + new_len where served, else max(ctx_len, 0).
 *   slots             out, int32 [max_tokens]: page * page_size + offset of each new token, requests
 *                     back to back; -1 from cu_q[n_requests] on (and where the token's page, one
 *                     held before, is entered as negative or gives a slot beyond 2^31 - 1).
 *   positions         out, int32 [max_tokens]: the token's position in its request; 0 past the end.
 *   status            out, int32 [n_requests]: 0 served, 1 refused, 2 invalid.
 *   n_left            out, int32 [1]: the pages left, free_pages[0 .. n_left); not n_free itself.
 * The call may be repeated: its inputs (block_table's taken entries apart) are left alone, so the
 * outputs must not overlap them.  0 <= n_requests <= CQ_MAX_REQUESTS, 0 <= max_tokens,
 * page_size >= 1, max_pages >= 1, max_pages * page_size < 2^31, table_stride >= max_pages.
 */
#define CQ_MAX_REQUESTS 4096
int32_t cq_kv_block_map(const int32_t *ctx_len, const int32_t *new_len, int32_t n_requests, int32_t page_size,
                        const int32_t *free_pages, const int32_t *n_free, int32_t free_capacity,
                        int32_t *block_table, int64_t table_stride, int32_t max_pages, int32_t max_tokens,
                        int32_t *cu_q, int32_t *kv_len, int32_t *slots, int32_t *positions, int32_t *status,
                        int32_t *n_left, void *stream);

/*
 * New keys and values into the pages of the cache.
 *   k, v              16-bit elements [n_tokens][kv_heads][head_dim]: *_token_stride and
 *                     *_head_stride apart, head_dim contiguous.
 *   k_cache, v_cache  in and out, [n_pages][kv_heads][page_size][head_dim]: page_stride, head_stride
 *                     and row_stride apart (the same for both), head_dim contiguous.
 *   slots             int32 [n_tokens]; a token whose slot is outside [0, n_pages * page_size) is
 *                     not written.  No slot may occur twice.
 * n_tokens, n_pages >= 0; kv_heads, page_size, head_dim >= 1; strides >= 0, those of the cache
 * at least what the layout's order needs is the caller's care.
 */
int32_t cq_kv_cache_write(const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                          int64_t v_token_stride, int64_t v_head_stride, void *k_cache, void *v_cache,
                          int64_t page_stride, int64_t head_stride, int64_t row_stride, int32_t n_pages,
                          int32_t page_size, int32_t kv_heads, int32_t head_dim, const int32_t *slots,
                          int32_t n_tokens, void *stream);

/*
 * Attention of new tokens over a paged cache.  Request r has the n = cu_q[r + 1] - cu_q[r] packed
 * query tokens from cu_q[r] on and kv_len[r] cached tokens, the new ones last: its i-th query token
 * stands at position p = kv_len[r] - n + i and sees the keys j < kv_len[r] with j <= p (causal) and
 * j > p - window (window > 0).  Query head h reads key/value head h / (heads / kv_heads).
 *        out = sum_j softmax_j(scale q . k_j) v_j,    lse = log sum_j exp(scale q . k_j)
 * over the keys seen; a token that sees none, or belongs to no request, gets out = 0, lse = -inf.
 * What a masked key or value holds (an unwritten slot, an infinity, a NaN) has no effect on the row
 * that does not see it.  Scores, softmax statistics and sums are fp32; the weights are rounded to the
 * 16-bit type for their product with V on the matrix cores (against a maximum that may lag by 2^8:
 * the sums of weights times V stay finite while 2^8 times their sum of magnitudes does).
 *   type              CQ_BF16 or CQ_F16: q, k_cache, v_cache and out.
 *   q, out            [n_tokens][heads][head_dim], strides as given, head_dim contiguous.
 *   k_cache, v_cache  as for cq_kv_cache_write.
 *   block_table       int32 rows of max_pages, table_stride apart: position j is in page
 *                     block_table[r][j / page_size]; keys of a page outside [0, n_pages) count as
 *                     masked.
 *   cu_q, kv_len      int32 [n_requests + 1], [n_requests], cu_q non-decreasing.  A kv_len below 0 is
 *                     taken as 0, one beyond max_pages * page_size (0 where n_pages is 0) as that: the
 *                     new tokens are then the last ones of the table's.
 *   max_q, max_kv     bounds of n and kv_len, from the host: they set how the work is divided.  Query
 *                     tokens past max_q are not computed (their out is left as it is); kv_len may
 *                     exceed max_kv, at a loss of speed.
 *   lse               out, nullable, float [n_tokens][heads].
 *   workspace         cq_paged_attention_workspace_size(...) bytes for the same sizes (none: may be
 *                     NULL).
 * q, k_cache, v_cache and out 16-byte aligned, all strides multiples of 8; head_dim a multiple of 8 up
 * to CQ_MAX_HEAD_DIM; heads a multiple of kv_heads; max_pages * page_size <= 2^30; window > 0 needs
 * causal; scale finite; n_requests and heads < 2^16, n_tokens * heads < 2^31.  CQ_EUNSUPPORTED, with nothing enqueued,
 * where requests may have more than 16 rows (tokens times heads / kv_heads) and (n_tokens * heads / 256 + (n_requests
 * + 1) * kv_heads) is 2^23 or more, unless n_requests * ceil(max_q * heads / kv_heads / 256) * kv_heads is less.
 */
#define CQ_MAX_HEAD_DIM 256
typedef struct cq_paged_attention_args {
    const void *q;
    const void *k_cache;
    const void *v_cache;
    const int32_t *block_table;
    const int32_t *cu_q;
    const int32_t *kv_len;
    void *out;
    float *lse;
    int64_t q_token_stride, q_head_stride;
    int64_t out_token_stride, out_head_stride;
    int64_t page_stride, head_stride, row_stride;
    int64_t table_stride;
    int32_t type;
    int32_t n_tokens, n_requests, max_q, max_kv;
    int32_t heads, kv_heads, head_dim;
    int32_t page_size, n_pages, max_pages;
    int32_t causal, window;
    float scale;
} cq_paged_attention_args;
size_t cq_paged_attention_workspace_size(int32_t n_tokens, int32_t n_requests, int32_t max_q, int32_t max_kv,
                                         int32_t heads, int32_t kv_heads, int32_t head_dim);
int32_t cq_paged_attention(const cq_paged_attention_args *args, void *workspace, size_t workspace_bytes,
                           void *stream);

/*
 * Microscaled blocks: 32 neighbouring values with a shared power of two as a byte b (2^(b - 127); 255: all 32 are NaN)
 * and an element of 4 or 8 bits each.
 *   CQ_MXFP4  e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives (bit 3), two a byte, the first in the low four bits.
 *   CQ_MXFP8  e4m3: up to 448 (0x7f, 0xff: NaN), one a byte.
 * A value is its element times 2^(b - 127).
 */
#define CQ_MXFP4 3
#define CQ_MXFP8 4
#define CQ_MX_BLOCK 32

/*
 * Rows of values as microscaled blocks along the row.  With A the largest magnitude of a block, its scale is
 * 2^(floor(log2 A) - 2) (CQ_MXFP8: - 8), at least 2^-127 (b = 0, also where A = 0), and its elements are the values over
 * the scale rounded to nearest, ties to the even code, and at most 6 (448) in magnitude.  A block with an infinity or
 * a NaN becomes NaN (b = 255, codes 0).
 *   x       x_type (CQ_BF16, CQ_F16 or CQ_F32) [rows] of `len`, ldx elements apart; 16-byte aligned, ldx a multiple of 8.
 *   codes   out, [rows] of len / 2 bytes (CQ_MXFP8: len), ldc bytes apart; 16-byte aligned, ldc a multiple of 16.
 *   scales  out, [rows] of len / 32 bytes, lds apart.
 * len a positive multiple of 32; rows * len < 2^34; rows == 0 enqueues nothing.
 */
int32_t cq_mx_quantize(const void *x, int64_t ldx, int32_t x_type, int64_t rows, int64_t len, int32_t format,
                       uint8_t *codes, int64_t ldc, uint8_t *scales, int64_t lds, void *stream);
/*
 * The values that microscaled blocks stand for, rounded once to y_type (what a 16-bit type cannot hold becomes an
 * infinity or a subnormal number, as the type has it).  Arguments as for cq_mx_quantize, y in x's place.
 */
int32_t cq_mx_dequantize(const uint8_t *codes, int64_t ldc, const uint8_t *scales, int64_t lds, int32_t format,
                         int64_t rows, int64_t len, void *y, int64_t ldy, int32_t y_type, void *stream);

/*
 * Linear layer over MXFP4 weights with its epilogue:
 *        z[m][c] = sum_k X[m][k] W[c][k] + bias[c],   y as for cq_w4a16_linear,
 * X being x's rows as cq_mx_quantize gives them in x_format, or those given as codes.  The products are exact and summed
 * in fp32 on the matrix cores, the epilogue is in fp32, with one rounding into y's type.  A block that is NaN (of x or
 * W) makes the outputs NaN that it takes part in.
 *   type       CQ_BF16 or CQ_F16: of bias and residual, of x where it is not codes, and of y unless y_type is CQ_F32.
 *   x_format   CQ_MXFP4 or CQ_MXFP8.
 *   x          x_scales NULL: [M] rows of `in` values, ldx elements apart (a multiple of 8).  Else [M] rows of codes, in / 2
 *              (CQ_MXFP8: in) bytes, ldx bytes apart (a multiple of 16 up to 2^23).  16-byte aligned.
 *   x_scales   nullable, [M] rows of in / 32 bytes, ldxs apart (a multiple of 4); 4-byte aligned.
 *   qweight    [cols] rows of in / 2 bytes without gaps, 16-byte aligned; scales [cols] rows of in / 32 bytes, 4-byte
 *              aligned: W in MXFP4, as cq_mx_quantize gives them for [cols][in].  cols = out, or 2 out when gated (the gate's first).
 *   bias, residual, y, activation, gated   as for cq_w4a16_linear.
 *   workspace  cq_mxfp4_linear_workspace_size(...) bytes for the same sizes (0: may be NULL); `codes`: whether x is.
 * in a positive multiple of 128 up to 2^22; cols <= 2^25, M * cols < 2^38, M * in < 2^34, M < 2^31; M == 0 or out == 0 enqueues nothing.
 */
typedef struct cq_mxfp4_linear_args {
    const void *x;
    const uint8_t *x_scales, *qweight, *scales;
    const void *bias, *residual;
    void *y;
    int64_t ldx, ldxs, ldr, ldy;
    int64_t M, out, in;
    int32_t type, x_format, y_type, activation, gated;
} cq_mxfp4_linear_args;
size_t cq_mxfp4_linear_workspace_size(int64_t M, int64_t out, int64_t in, int32_t gated, int32_t x_format,
                                      int32_t codes);
int32_t cq_mxfp4_linear(const cq_mxfp4_linear_args *args, void *workspace, size_t workspace_bytes, void *stream);

/*
 * A paged cache whose keys and values are microscaled blocks along head_dim (a multiple of 32 up to CQ_MAX_HEAD_DIM).
 *   k_codes, v_codes    [n_pages][kv_heads][page_size] rows of head_dim / 2 bytes (CQ_MXFP8: head_dim), 16-byte aligned:
 *                       page_stride, head_stride and row_stride bytes apart (multiples of 16, the same for both).
 *   k_scales, v_scales  [n_pages][kv_heads][page_size] rows of head_dim / 32 bytes: scale_*_stride bytes apart.
 * Strides >= 0; that the rows do not overlap is the caller's care.
 */
typedef struct cq_mx_cache {
    void *k_codes, *v_codes, *k_scales, *v_scales;
    int64_t page_stride, head_stride, row_stride;
    int64_t scale_page_stride, scale_head_stride, scale_row_stride;
    int32_t format;
    int32_t n_pages, page_size, kv_heads, head_dim;
} cq_mx_cache;

/*
 * New keys and values into the pages of such a cache, each block quantized as by cq_mx_quantize.
 *   type   CQ_BF16 or CQ_F16, of k and v; they and slots as for cq_kv_cache_write.
 * n_tokens * kv_heads * head_dim < 2^34.
 */
int32_t cq_kv_cache_write_mx(const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                             int64_t v_token_stride, int64_t v_head_stride, int32_t type, const cq_mx_cache *cache,
                             const int32_t *slots, int32_t n_tokens, void *stream);

/*
 * cq_paged_attention over such a cache.  Keys and values are those the blocks stand for, in q's 16-bit type: exact where they
 * were quantized from values of that type; what it cannot hold is an infinity or rounded (in bfloat16 values from 2^128 on
 * and bits below 2^-133).
 *   args   as for cq_paged_attention, whose k_cache, v_cache and their strides are not read; kv_heads, head_dim, page_size
 *          and n_pages are the cache's.
 * Masks, outputs, limits and errors as there; a NaN block has no effect on a row that does not see it.  The workspace is of
 * cq_paged_attention_mx_workspace_size(...) bytes for the same sizes.
 */
size_t cq_paged_attention_mx_workspace_size(int32_t n_tokens, int32_t n_requests, int32_t max_q, int32_t max_kv,
                                            int32_t heads, int32_t kv_heads, int32_t head_dim);
int32_t cq_paged_attention_mx(const cq_paged_attention_args *args, const cq_mx_cache *cache, void *workspace,
                              size_t workspace_bytes, void *stream);

/*
 * Separately normalized environment diagonals from calibration activations
 * (CliffQuant README, "What CliffQuant changes": each channel's sensitivity
 * weighted by its activations, per calibration environment, each environment
 * normalized on its own; model
 * card, "Calibration and evaluation data": environments of 256-token windows,
 * a 16-bit model runtime).
 *   x   device uint16 [E][T][in]: bfloat16 bit patterns of the activations
 *       entering one matrix, T tokens per environment, row-major.
 *   d   out, float [in/128][E][128]: d_{e,i} = mean_t x_{t,i}^2 divided by its
 *       mean over the channels i (binary64, rounded once), the layout
 *       cq_quantize_groups takes with d_period = in/128.  An environment whose
 *       activations are all zero gives NaN (the solver flags it).
 * 1 <= E <= CQ_MAX_ENVS, T >= 1, in a multiple of 128 up to 2^24; x 16-byte
 * aligned.  workspace: cq_diagonals_workspace_size(E, T, in) bytes.
 */
size_t cq_diagonals_workspace_size(int32_t E, int64_t T, int64_t in);
int32_t cq_environment_diagonals(const uint16_t *x, int32_t E, int64_t T, int64_t in, float *d,
                                 void *workspace, size_t workspace_bytes, void *stream);

/*
 * Held-out comparison of two scale policies on the proxy's per-group values
 * (CliffQuant README, "Held-out reconstruction proxy": the minimax policy's
 * wins, ties and losses against Pooled-WMSE by group, and a 95% interval for
 * the effect from a bootstrap resampling within modules, paired across the
 * policies).
 *   pa, pb          device double [n_groups]: per-group proxy values p_g of
 *                   policies A and B (e.g. two rows of the per_group output of
 *                   cq_proxy_worst_env_wmse_multi on held-out diagonals).
 *   module_offsets  device int64 [n_modules+1] as for the proxy; a module whose
 *                   range is empty or out of bounds makes the effect NaN.
 *   boot_idx        device int32 [n_boot][n_groups], drawn by the caller:
 *                   replicate r takes, at position j of module m's range, group
 *                   boot_idx[r][j], which must lie in m's range (else that
 *                   replicate is NaN).  The same draw serves both policies.
 *   alpha           0 < alpha < 1: the interval runs from the 100 alpha/2 to
 *                   the 100 (1 - alpha/2) percentile.
 *   counts          out, device int64 [3]: groups with p_A < p_B, ==, >.
 *   effect          out, device double [1]: the mean over modules of each
 *                   module's mean of (p_B - p_A), every sum left to right.
 *   boot            out, device double [n_boot]: the replicate effects (the same
 *                   formula on each draw), sorted ascending, NaN last.
 *   ci              out, device double [2]: the percentiles of boot by linear
 *                   interpolation at position q (n_boot - 1); NaN when n_boot is
 *                   0 or a replicate is NaN.
 * 0 <= n_boot <= CQ_MAX_BOOT; (n_boot + 1) * n_modules <= 2^31 - 1.
 * workspace: cq_heldout_workspace_size(n_boot, n_modules) bytes.
 */
size_t cq_heldout_workspace_size(int32_t n_boot, int32_t n_modules);
int32_t cq_heldout_compare(const double *pa, const double *pb, int64_t n_groups,
                           const int64_t *module_offsets, int32_t n_modules,
                           const int32_t *boot_idx, int32_t n_boot, double alpha,
                           int64_t *counts, double *effect, double *boot, double *ci,
                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * Measurement aid, not part of the method: the fp32 fma issue rate the vector units reach, the
 * ceiling against which the full-grid search's issue rate (and its fraction of the published
 * 157.3 TFLOP/s fp32 peak: 256 CUs x 128 fma lanes x 2 flop x 2.4 GHz) is read.
 *   iters          >= 1: fmas per chain; each thread of `blocks` workgroups of 256 threads runs
 *                  8 independent chains, so the launch issues blocks x 4 waves x 8 x iters
 *                  fma wave instructions (2 flop per lane each).
 *   mode           0: the chains as x = fma(x, c, y) with c, y in vector registers (the
 *                  three-operand encoding, v_fma_f32); 1: as x = fma(y, c, x) (the accumulate
 *                  encoding, v_fmac_f32, which the full-grid search's environment sums use);
 *                  2: as x = fma(x, a, b) with a, b scalar kernel arguments (v_fma_f32 with a
 *                  scalar-register operand).  The forms issue at different rates.
 *   out            device float [blocks * 256]: the chains' sums (kept so nothing is dead code).
 *   clocks         device uint64 [2 * blocks]: per workgroup, the shader clock cycles and the
 *                  constant-rate wall clock ticks between its thread 0's start and end.
 *   wall_clock_hz  HOST double, out: the wall clock's rate (cycles / ticks x this = the clock).
 * Returns CQ_EINVAL for iters < 1, blocks < 1, another mode or a null pointer.
 */
int32_t cq_probe_valu_fma(int32_t iters, int32_t blocks, int32_t mode, float *out, uint64_t *clocks,
                          double *wall_clock_hz, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* CQ_H */
