/*
 * fp8w_moe — mixture-of-experts operators and the int8 and 4-bit linear layers for
 * AMD MI355X (gfx950), next to the FP8 weight-only linear layer of fp8w.h.
 *
 * C ABI of libfp8w_moe.so. The conventions are those of fp8w.h: dense row-major
 * tensors, device pointers owned by the caller, no allocation by the library,
 * work enqueued on `stream` (0 = the null stream) in stream order, arguments
 * validated before anything is enqueued, status codes and dtypes of fp8w.h. The
 * thread's current device is the buffers' and the stream's. Every call is
 * asynchronous and can be captured into a HIP graph, but for fp8w_quantize_int8 and
 * fp8w_quantize_fp4, which synchronize. A call's results depend on its arguments alone (no order of
 * atomics enters them). Inputs may be read by whole aligned dwords, that is with
 * up to three bytes beside their first and last. Sizes up to 2^31 - 1 unless
 * stated; a call whose products or sums would need a launch of 2^32 threads or
 * more (above 3e10 outputs) is invalid.
 */
#ifndef FP8W_MOE_H
#define FP8W_MOE_H

#include "fp8w.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The router: each token's top_k experts, their weights, and the token slots
 * ordered by expert.
 *   logits   [t, e] of dtype (BF16, FP16 or FP32); 1 <= e <= 1024,
 *            1 <= top_k <= min(e, 64), t * top_k <= 2^31 - 1.
 *   weights  [t, top_k] fp32: exp(l_j - l_0) over the sum of the chosen experts'
 *            (renormalize != 0) or of all of the token's (the softmax's values).
 *   experts  [t, top_k] int32: the experts by falling logit, equal logits by
 *            the lower index. An expert with logit -inf is never taken; places
 *            that are left over hold -1 and weight 0 (all of them for a token
 *            whose logits are all -inf: a padding token). A NaN counts as above
 *            every number; a token with a NaN or +inf logit has NaN weights.
 *   offsets  [e + 1] int32: expert i has positions offsets[i] .. offsets[i+1]-1
 *            of slots; offsets[e] slots have an expert.
 *   slots    [t * top_k] int32: the slots token * top_k + j by expert, rising
 *            within an expert; slots without an expert from offsets[e] on.
 *   tokens   [t * top_k] int32: slots / top_k.
 *   workspace of fp8w_route_workspace_bytes bytes (0 for few tokens), 4-byte
 *            aligned.
 * No two buffers may overlap. t == 0 writes offsets (zeros).
 */
FP8W_API fp8w_status_t fp8w_route(const void* logits, fp8w_dtype_t dtype, int64_t t, int64_t e, int64_t top_k,
                                  int renormalize, float* weights, int32_t* experts, int32_t* offsets, int32_t* slots,
                                  int32_t* tokens, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes of fp8w_route; 0 for invalid sizes. */
FP8W_API size_t fp8w_route_workspace_bytes(int64_t t, int64_t e, int64_t top_k);

/*
 * Products grouped by expert, ragged sizes. For the positions p of expert i,
 * offsets[i] <= p < offsets[i + 1]:
 *   y[dst(p), c] = scale[i, c] * sum_k x[src(p), k] * value(q[i, c, k]) + bias[i, c]
 * in fp32, rounded once to act_dtype (BF16 or FP16).
 *   x        [x_count, k]; src(p) = x_rows[p], or p without x_rows (then
 *            x_count == m).
 *   q, scale [e, n, k] e4m3 codes and [e, n] fp32, an expert's as written by
 *            fp8w_quantize (one call on the [e * n, k] weights); 1 <= e <= 1024.
 *   bias     [e, n] of act_dtype, or NULL.
 *   offsets  [e + 1] int32 on the device, rising from 0 to at most m. Positions
 *            offsets[e] .. m - 1 belong to no expert: their rows are zeros.
 *   x_rows, y_rows  [m] int32 on the device, or NULL; dst(p) = y_rows[p], or p.
 *            y_rows must not name a row twice.
 *   y        [m, n] of act_dtype; must not overlap an input.
 *   workspace, workspace_bytes: not used, whatever they are (no plan needs one).
 * Device values are not validated, and nothing outside the buffers is touched
 * whatever they hold: offsets are clamped to 0 .. m, a position whose src is
 * outside x gives a row of NaN, one whose dst is outside y is not written.
 */
FP8W_API fp8w_status_t fp8w_linear_experts(const void* x, fp8w_dtype_t act_dtype, int64_t x_count, int64_t k,
                                           const uint8_t* q, const float* scale, const void* bias, int64_t e,
                                           int64_t n, const int32_t* offsets, int64_t m, const int32_t* x_rows,
                                           const int32_t* y_rows, void* y, void* workspace, size_t workspace_bytes,
                                           hipStream_t stream);

/* Workspace bytes fp8w_linear_experts uses: 0. */
FP8W_API size_t fp8w_linear_experts_workspace_bytes(int64_t m, int64_t e, int64_t n, int64_t k, const void* x,
                                                    const uint8_t* q);

/* Name of the kernel fp8w_linear_experts runs for an x of up to m rows, NULL for
 * invalid sizes and calls that run none. The string lives until the thread's next
 * call. */
FP8W_API const char* fp8w_linear_experts_kernel(int64_t m, int64_t e, int64_t n, int64_t k, const void* x,
                                                const uint8_t* q);

/*
 * A token's weighted sum over its slots:
 *   out[t, c] = sum_j weights[t, j] * y[t * top_k + j, c], j = 0 .. top_k - 1,
 * fp32 in the order of j, rounded once to act_dtype.
 *   y [t * top_k, n], weights [t, top_k] fp32, out [t, n]; out must not overlap
 *   an input; 0 <= top_k <= 64 (0: zeros).
 */
FP8W_API fp8w_status_t fp8w_combine(const void* y, fp8w_dtype_t act_dtype, const float* weights, int64_t t,
                                    int64_t top_k, int64_t n, void* out, hipStream_t stream);

/*
 * Build-time int8 quantizer: scale[r] = amax_k |w[r, k]| / 127 (fp32), codes
 * round(fl32(127 w) / amax) to the nearest integer, ties to even (-127 .. 127);
 * an all-zero row has scale 0 and codes 0. Arguments, synchronization and
 * FP8W_ERR_NONFINITE as in fp8w_quantize; k <= 131072.
 */
FP8W_API fp8w_status_t fp8w_quantize_int8(const void* w, fp8w_dtype_t w_dtype, int64_t n, int64_t k, int8_t* q,
                                          float* scale, hipStream_t stream);

/*
 * Per-token int8 quantization of activations x [m, k] (BF16 or FP16): the same
 * scale and codes (for these types the codes are the exact quotient's nearest
 * integers). A row with a NaN or an infinity gets a NaN scale and zero codes.
 */
FP8W_API fp8w_status_t fp8w_quantize_activations_int8(const void* x, fp8w_dtype_t act_dtype, int64_t m, int64_t k,
                                                      int8_t* qx, float* sx, hipStream_t stream);

/*
 * y[t, c] = (sum_k qx[t, k] * q[c, k]) * sx[t] * scale[c] + bias[c]: the sum in
 * 32-bit integers (exact for codes -128 .. 127: k <= 131072), the rest in fp32,
 * rounded once to out_dtype (BF16 or FP16). bias [n] of out_dtype, or NULL; y must not overlap
 * an input.
 */
FP8W_API fp8w_status_t fp8w_gemm_int8(const int8_t* qx, const float* sx, int64_t m, int64_t k, const int8_t* q,
                                      const float* scale, const void* bias, int64_t n, void* y,
                                      fp8w_dtype_t out_dtype, hipStream_t stream);

/*
 * The int8 layer on 16-bit activations: per-token quantization of x and
 * fp8w_gemm_int8, y of act_dtype. workspace of fp8w_linear_int8_workspace_bytes
 * bytes, 16-byte aligned (FP8W_ERR_WORKSPACE when short).
 */
FP8W_API fp8w_status_t fp8w_linear_int8(const void* x, fp8w_dtype_t act_dtype, int64_t m, int64_t k, const int8_t* q,
                                        const float* scale, const void* bias, int64_t n, void* y, void* workspace,
                                        size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes of fp8w_linear_int8 for these sizes and pointers (NULL:
 * aligned); 0 for invalid sizes. */
FP8W_API size_t fp8w_linear_int8_workspace_bytes(int64_t m, int64_t n, int64_t k, const void* x, const int8_t* q);

/* Names of the kernels fp8w_linear_int8 runs; NULL as for experts. */
FP8W_API const char* fp8w_linear_int8_kernel(int64_t m, int64_t n, int64_t k, const void* x, const int8_t* q);

/*
 * 4-bit weights: e2m1 codes (sign, two bits of exponent, one of mantissa: 0, 0.5,
 * 1, 1.5, 2, 3, 4, 6) with one e8m0 scale 2^(s - 127) for a block of 32 along k, the
 * OCP MX format of that element type.
 *   q      [n, (k + 1) / 2] bytes: an even k's code in the low four bits, the next
 *          one's in the high four (those of an odd row's last byte are ignored).
 *   scale  [n, (k + 31) / 32] bytes s; the last block of a row may be shorter. 255
 *          makes the block's weights NaN.
 * A weight enters a product as its value in the activation type: exact in BF16 for
 * every scale; in FP16 exact for scales 2^-23 .. 2^13, beyond them rounded as FP16
 * rounds (to its subnormals, or to infinity above 65504).
 */

/*
 * Build-time quantizer of w [n, k] (BF16, FP16 or FP32): s = floor(log2(amax)) - 2 +
 * 127 of each block (0 for a block below 2^-124 or of zeros), codes the nearest
 * values of w / 2^(s - 127), ties to the even code, those beyond 6 the code of 6.
 * Synchronizes; FP8W_ERR_NONFINITE when a weight is NaN or infinite (its block then
 * has s == 255). k <= 2^31 - 1. No two buffers may overlap.
 */
FP8W_API fp8w_status_t fp8w_quantize_fp4(const void* w, fp8w_dtype_t w_dtype, int64_t n, int64_t k, uint8_t* q,
                                         uint8_t* scale, hipStream_t stream);

/* The weights [n, k] of codes and scales, rounded once to out_dtype (exact in FP32
 * and BF16). */
FP8W_API fp8w_status_t fp8w_dequantize_fp4(const uint8_t* q, const uint8_t* scale, int64_t n, int64_t k, void* out,
                                           fp8w_dtype_t out_dtype, hipStream_t stream);

/*
 * The linear layer on 4-bit weights:
 *   y[t, c] = sum_k x[t, k] * w[c, k] + bias[c]
 * in fp32, rounded once to act_dtype (BF16 or FP16). x [m, k], bias [n] of act_dtype
 * or NULL, y [m, n]; y must not overlap an input. workspace of
 * fp8w_linear_fp4_workspace_bytes bytes, 16-byte aligned (FP8W_ERR_WORKSPACE when
 * short), for the calls that split k over workgroups.
 */
FP8W_API fp8w_status_t fp8w_linear_fp4(const void* x, fp8w_dtype_t act_dtype, int64_t m, int64_t k, const uint8_t* q,
                                       const uint8_t* scale, const void* bias, int64_t n, void* y, void* workspace,
                                       size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes of fp8w_linear_fp4 for these sizes and pointers (NULL: aligned);
 * 0 for invalid sizes. */
FP8W_API size_t fp8w_linear_fp4_workspace_bytes(int64_t m, int64_t n, int64_t k, const void* x, const uint8_t* q,
                                                const uint8_t* scale);

/* Name of the kernel fp8w_linear_fp4 runs; NULL as for experts. */
FP8W_API const char* fp8w_linear_fp4_kernel(int64_t m, int64_t n, int64_t k, const void* x, const uint8_t* q,
                                            const uint8_t* scale);

/*
 * fp8w_linear_experts on 4-bit weights: q [e, n, (k + 1) / 2], scale [e, n, (k + 31) /
 * 32]; everything else as there. No workspace.
 */
FP8W_API fp8w_status_t fp8w_linear_experts_fp4(const void* x, fp8w_dtype_t act_dtype, int64_t x_count, int64_t k,
                                               const uint8_t* q, const uint8_t* scale, const void* bias, int64_t e,
                                               int64_t n, const int32_t* offsets, int64_t m, const int32_t* x_rows,
                                               const int32_t* y_rows, void* y, hipStream_t stream);

/* Name of its kernel, as fp8w_linear_experts_kernel. */
FP8W_API const char* fp8w_linear_experts_fp4_kernel(int64_t m, int64_t e, int64_t n, int64_t k, const void* x,
                                                    const uint8_t* q, const uint8_t* scale);

/* Formats of a layer's weights. */
typedef enum fp8w_weight_format {
    FP8W_WEIGHT_E4M3 = 0, /* q [.., n, k] e4m3 codes, scale [.., n] fp32 */
    FP8W_WEIGHT_FP4 = 1   /* q [.., n, (k + 1) / 2], scale [.., n, (k + 31) / 32] bytes */
} fp8w_weight_format_t;

/*
 * A whole mixture-of-experts layer for a few tokens, in two launches:
 *   choice and weights[t, j] of fp8w_route(logits, dtype, t, e, top_k, renormalize);
 *   gate, up = the expert's rows 0 .. inner - 1 and inner .. 2 inner - 1 of q_gate_up
 *              on x[t] (and their bias);
 *   h        = gate / (1 + exp(-gate)) * up, rounded to act_dtype (above 65504 in FP16:
 *              infinite, and with it the token's row, infinite or NaN);
 *   out[t]   = sum_j weights[t, j] * (the expert's q_down on h, and its bias),
 * sums, scales, biases and the activation in fp32, out rounded once to act_dtype
 * (BF16 or FP16). Places of the choice that are left over add nothing: a padding
 * token's row is zeros. A token with a NaN weight has a row of NaN.
 *   x, out     [t, hidden]; t <= 64 (more: fp8w_route, fp8w_linear_experts,
 *              fp8w_combine). logits [t, e] of logits_dtype.
 *   q_gate_up, scale_gate_up, bias_gate_up  [e, 2 inner, hidden] in `format`,
 *              bias [e, 2 inner] of act_dtype or NULL.
 *   q_down, scale_down, bias_down  [e, hidden, inner], [e, hidden].
 *   hidden, inner >= 1, up to 2^22; t * top_k * (inner + 64) < 2^27.
 *   workspace of fp8w_moe_layer_workspace_bytes bytes, 16-byte aligned.
 * out and workspace must not overlap an input or each other.
 */
FP8W_API fp8w_status_t fp8w_moe_layer(const void* x, fp8w_dtype_t act_dtype, int64_t t, int64_t hidden,
                                      const void* logits, fp8w_dtype_t logits_dtype, int64_t e, int64_t top_k,
                                      int renormalize, fp8w_weight_format_t format, const uint8_t* q_gate_up,
                                      const void* scale_gate_up, const void* bias_gate_up, int64_t inner,
                                      const uint8_t* q_down, const void* scale_down, const void* bias_down, void* out,
                                      void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes of fp8w_moe_layer; 0 for invalid sizes and for t == 0. */
FP8W_API size_t fp8w_moe_layer_workspace_bytes(int64_t t, int64_t e, int64_t top_k, int64_t hidden, int64_t inner);

/* The hipError_t behind this thread's last FP8W_ERR_HIP of this library. */
FP8W_API int fp8w_moe_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8W_MOE_H */
