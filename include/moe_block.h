/*
 * moe_block.h — C ABI of libmoe.so, second part: the operators around the MoE
 * layer of moe.h.  The residual addition and RMS norm in front of it with an
 * FP8 output, forward and backward; the whole layer for a few tokens; and the
 * global norm and clipping of its gradients.
 *
 * The conventions are those of moe.h: device pointers owned by the caller,
 * row-major layouts, 16-byte alignment of BF16 and byte matrices and 4-byte
 * alignment of FP32 and int32 arrays unless stated otherwise, nothing
 * allocated and nothing synchronised by the library, every call enqueued on
 * `stream` of the current device and returning after host-side validation and
 * launch, an error code with no work enqueued and moe_last_error() set.
 * All calls can be captured into a graph.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* moe_rmsnorm_quant — residual addition, RMS norm and FP8 quantisation of the
 * layer's input, in one pass over the rows.
 *   x         [T, d] BF16
 *   residual  [T, d] BF16, or NULL
 *   weight    [d] BF16
 *   eps       > 0
 *   sum       [T, d] BF16 out: x + residual (x itself without a residual), or
 *             NULL.  May be x's or residual's own memory.
 *   y         [T, d] BF16 out: the normed rows (the router's input), or NULL
 *   q, scale  [T, d] E4M3 and [T, d/128] FP32 out: y in 1x128 tiles, or both
 *             NULL
 *   rstd      [T] FP32 out, for the backward, or NULL
 * Per row: h = bf16(x + residual); rstd = fl32(1 / sqrt(sum(h^2) / d + eps)),
 * evaluated in FP64; y = bf16(fl32(fl32(h * rstd) * weight)).  (q, scale) are
 * bit for bit what fp8_quant_1x128 makes of y, whether y is stored or not.
 * No output may otherwise overlap an input or another output.
 * T = 0 is a no-op.  MOE_ERR_INVALID_ARG: d not a positive multiple of 128,
 * eps not positive and finite, q without scale or the reverse, no output at
 * all, outputs that overlap.  MOE_ERR_UNSUPPORTED: d > 16384. */
moe_status moe_rmsnorm_quant(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int T, int d,
                             float eps, uint16_t* sum, uint16_t* y, uint8_t* q, float* scale, float* rstd,
                             void* stream);

/* moe_rmsnorm_quant_pow2 — moe_rmsnorm_quant with the power-of-two scale rule
 * of fp8_quant_1x128_pow2. */
moe_status moe_rmsnorm_quant_pow2(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int T, int d,
                                  float eps, uint16_t* sum, uint16_t* y, uint8_t* q, float* scale, float* rstd,
                                  void* stream);

/* Bytes of device workspace moe_rmsnorm_backward needs (0 on bad sizes and for
 * T = 0). */
size_t moe_rmsnorm_backward_workspace_bytes(int T, int d);

/* moe_rmsnorm_backward — gradients of moe_rmsnorm_quant's norm and addition
 * (the quantisation passes gradients through).
 *   dy       [T, d] BF16: the gradient with respect to y
 *   h        [T, d] BF16: the forward's sum (x without a residual)
 *   weight   [d] BF16;  rstd [T] FP32 from the forward
 *   dres     [T, d] BF16: the gradient that reaches sum past the norm (through
 *            the residual stream), or NULL
 *   dh       [T, d] BF16 out: the gradient with respect to sum, which is that
 *            of x and of residual.  May be dres's own memory.
 *   dweight  [d] FP32 out (zeros for T = 0)
 *   workspace  at least moe_rmsnorm_backward_workspace_bytes(T, d) bytes,
 *            16-byte aligned; overwritten; calls that share it must not overlap
 * With xh = h * rstd, g = dy * weight, c = sum(g * xh) / d per row:
 * dh = bf16(rstd * (g - xh * c) + dres), dweight = sum over rows of dy * xh;
 * FP32 throughout, the last sum's second stage FP64.  Deterministic.
 * Errors as moe_rmsnorm_quant, and MOE_ERR_WORKSPACE. */
moe_status moe_rmsnorm_backward(const uint16_t* dy, const uint16_t* h, const uint16_t* weight, const float* rstd,
                                const uint16_t* dres, int T, int d, uint16_t* dh, float* dweight, void* workspace,
                                size_t workspace_bytes, void* stream);

/* Bytes of device workspace moe_layer_few needs (0 for sizes it refuses and for
 * T = 0). */
size_t moe_layer_few_workspace_bytes(int T, int d, int f, int E, int k);

/* moe_layer_few — the whole layer for T <= 16 tokens: moe_route,
 * fp8_quant_1x128, the grouped GEMMs and moe_combine in one call that streams
 * the chosen experts' weights.
 *   x         [T, d] BF16;  wg [E, d] BF16;  bias [E] FP32 or NULL; p as for
 *             moe_route
 *   w13, w13_s, w2, w2_s  the expert weights as for grouped_gemm_fp8_swiglu
 *             with n_groups = E + 1: [E + 1, 2f, d] and [E + 1, d, f] E4M3 with
 *             128x128 block scales, group E the shared expert
 *   residual  [T, d] BF16 added to the output, or NULL
 *   idx, w    [T, k] int32 / FP32 out: the selection and its gates, as
 *             moe_route writes them
 *   out       [T, d] BF16 out.  May be x's or residual's own memory.  No
 *             output may otherwise overlap an input or another output.
 *   workspace at least moe_layer_few_workspace_bytes(T, d, f, E, k) bytes,
 *             16-byte aligned; overwritten; calls that share it must not overlap
 * The layer's arithmetic (the activations and h in 1x128 FP8 tiles, FP32
 * promotion of every K block) with two steps kept in higher precision: the
 * selection ranks FP64 scores by all their bits, equal ones by the lower index
 * (moe_route's FP32 scores agree except within 1e-6 of a tie), and the experts'
 * outputs are summed in FP32 before the one rounding of out, without being
 * rounded to BF16 first.
 * T = 0 is a no-op.  Errors as moe_route and grouped_gemm_fp8_swiglu,
 * MOE_ERR_WORKSPACE, and MOE_ERR_UNSUPPORTED for T > 16, d > 8192 or f > 32768. */
moe_status moe_layer_few(const uint16_t* x, const uint16_t* wg, const float* bias, int T, int d, int f,
                         moe_route_params p, const uint8_t* w13, const float* w13_s, const uint8_t* w2,
                         const float* w2_s, const uint16_t* residual, int32_t* idx, float* w, uint16_t* out,
                         void* workspace, size_t workspace_bytes, void* stream);

/* moe_layer_few_pow2 — moe_layer_few with the power-of-two scale rule for x and
 * h (the weights' scales may be any, as fp8_quant_128x128_pow2 writes them in
 * that variant). */
moe_status moe_layer_few_pow2(const uint16_t* x, const uint16_t* wg, const float* bias, int T, int d, int f,
                              moe_route_params p, const uint8_t* w13, const float* w13_s, const uint8_t* w2,
                              const float* w2_s, const uint16_t* residual, int32_t* idx, float* w, uint16_t* out,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Element types of the gradient lists below. */
typedef enum {
  MOE_GRAD_FP32 = 0,
  MOE_GRAD_BF16 = 1
} moe_grad_type;

/* Bytes of device workspace moe_grad_norm needs for n_tensors tensors (0 for
 * n_tensors <= 0). */
size_t moe_grad_norm_workspace_bytes(int n_tensors);

/* moe_grad_norm — L2 norm of all elements of a list of tensors, and the factor
 * that clips them to max_norm.
 *   grads      [n_tensors] HOST array of device pointers, each aligned to its
 *              elements (4 or 2 bytes); NULL only for an empty tensor
 *   sizes      [n_tensors] HOST array of element counts (0 and counts above
 *              2^32 included)
 *   types      [n_tensors] HOST array of moe_grad_type
 *   max_norm   > 0 (infinity: the factor is 1 for every finite norm)
 *   norm       [1] FP32 out: sqrt of the sum of squares, summed in FP64
 *   coef       [1] FP32 out: 1 if norm <= max_norm, else max_norm / norm
 *              (0 for an infinite norm, NaN for a NaN)
 *   workspace  moe_grad_norm_workspace_bytes(n_tensors) bytes, 8-byte aligned
 *              (may be NULL when that is 0); overwritten; calls that share it
 *              must not overlap
 * norm, coef and the workspace share no memory with each other or a gradient.
 * The host arrays are read before the call returns.  Infinities and NaN in the
 * gradients are allowed and show in norm.  The same tensors give the same
 * bits.  n_tensors = 0: norm 0, coef 1. */
moe_status moe_grad_norm(const void* const* grads, const int64_t* sizes, const int* types, int n_tensors,
                         float max_norm, float* norm, float* coef, void* workspace, size_t workspace_bytes,
                         void* stream);

/* moe_grad_scale — outs[i] = grads[i] * coef[0] for every tensor, the FP32
 * product rounded to the tensor's type (round to nearest even).
 *   grads, outs, sizes, types  HOST arrays as for moe_grad_norm; outs[i] may be
 *              grads[i] (in place: with a coef of 1 nothing is then read or
 *              written), and must not overlap it otherwise, nor another output, another
 *              tensor's gradient or coef
 *   coef       [1] FP32 on the device (moe_grad_norm's) */
moe_status moe_grad_scale(const void* const* grads, void* const* outs, const int64_t* sizes, const int* types,
                          int n_tensors, const float* coef, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
