/*
 * moe_experts.h — C ABI of libmoe.so, third part: experts and projections
 * whose operands are not quantised.  Tokens sorted by expert and back with
 * their weights, forward and backward; grouped and dense matrix products in 16
 * bits with bias, activation and residual in the epilogue, and their gradients;
 * and dropout whose mask is recomputed instead of stored.
 *
 * The conventions are those of moe.h: device pointers owned by the caller,
 * row-major layouts, nothing allocated and nothing synchronised by the library,
 * every call enqueued on `stream` of the current device and returning after
 * host-side validation and launch, an error code with no work enqueued and
 * moe_last_error() set.  All calls can be captured into a graph.  Infinities
 * and NaN are allowed: they reach the outputs that depend on them, no others.
 * Tensors of a moe_dtype are 16-byte aligned, FP32 and int32 arrays 4-byte
 * aligned.  No output may overlap an input or another output unless stated
 * otherwise.  Sums are FP32; an output in fewer bits is rounded once, to
 * nearest even.  The same arguments give the same bits.
 */
#ifndef MOE_EXPERTS_H
#define MOE_EXPERTS_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_BF16 = 0,
  MOE_FP16 = 1,
  MOE_FP32 = 2   /* the token calls and dropout only */
} moe_dtype;

/* ---- Tokens sorted by expert, and back ----
 * T tokens have k slots each; slot s = t * k + j names an expert or none.  Row
 * pos[s] of the sorted order belongs to slot s; pos[s] < 0 (or >= rows): the
 * slot is dropped, has no row and counts for nothing, whatever its weight. */

/* Bytes of device workspace moe_sort needs (0 for sizes it refuses and for
 * T = 0). */
size_t moe_sort_workspace_bytes(int T, int k, int E);

/* moe_sort — the stable order of the slots by expert.  Unlike moe_permute it
 * takes dropped slots, an expert more than once for a token, and adds no
 * shared rows.
 *   idx       [T, k] int32: the slot's expert in [0, E); anything else drops it
 *   offsets   [E + 1] int32 out: expert e owns rows [offsets[e], offsets[e+1]);
 *             offsets[E] is the number of slots that are not dropped
 *   pos       [T, k] int32 out: the slot's row, -1 for a dropped one
 *   row_slot  [T * k] int32 out: the slot of every row, -1 from offsets[E] on
 *   workspace at least moe_sort_workspace_bytes(T, k, E) bytes, 4-byte aligned
 *             (may be NULL when that is 0); overwritten; calls that share it must not overlap
 * T = 0: offsets are zeros.  MOE_ERR_INVALID_ARG: T < 0, k < 1, E < 1.
 * MOE_ERR_UNSUPPORTED: k > 64, E > 1024, T * k > 2^30. */
moe_status moe_sort(const int32_t* idx, int T, int k, int E, int32_t* offsets, int32_t* pos, int32_t* row_slot,
                    void* workspace, size_t workspace_bytes, void* stream);

/* moe_dispatch — tokens to their rows: out[pos[s]] = w[s] * x[t].
 *   x     [T, d];  pos [T, k] int32, rows distinct;  w [T, k] FP32, or NULL for ones
 *   out   [rows, d] out; rows that no slot has are left as they were
 * Any d >= 1.  T = 0 is a no-op.  MOE_ERR_INVALID_ARG: T < 0, rows < 0, k < 1,
 * d < 1, an unknown type.  MOE_ERR_UNSUPPORTED: k > 64, T or rows * d > 2^40. */
moe_status moe_dispatch(moe_dtype type, const void* x, const int32_t* pos, const float* w, int T, int k, int d,
                        int rows, void* out, void* stream);

/* moe_dispatch_backward — gradients of moe_dispatch:
 *   dx[t] = sum_j w[s] * drows[pos[s]] (+ residual[t]),
 *   dw[s] = <x[t], drows[pos[s]]> (0 for a dropped slot)
 *   drows     [rows, d];  x [T, d] and dw [T, k] FP32 out, or both NULL
 *   residual  [T, d] added to dx (a gradient that reaches x another way), or NULL
 *   dx        [T, d] out; may be residual's own memory
 * Errors as moe_dispatch, and x without dw or the reverse. */
moe_status moe_dispatch_backward(moe_dtype type, const void* drows, const int32_t* pos, const float* w, const void* x,
                                 const void* residual, int T, int k, int d, int rows, void* dx, float* dw,
                                 void* stream);

/* moe_collect — rows back to their tokens:
 *   out[t] = sum_j w[s] * y[pos[s]] (+ residual[t]), in slot order, the residual last
 *   y [rows, d];  w [T, k] FP32, or NULL for ones;  residual [T, d] or NULL
 *   out [T, d] out; may be residual's own memory
 * Errors as moe_dispatch. */
moe_status moe_collect(moe_dtype type, const void* y, const int32_t* pos, const float* w, const void* residual, int T,
                       int k, int d, int rows, void* out, void* stream);

/* moe_collect_backward — gradients of moe_collect (that of the residual is dout):
 *   dy[pos[s]] = w[s] * dout[t],  dw[s] = <dout[t], y[pos[s]]> (0 for a dropped slot)
 *   dout [T, d];  y [rows, d] and dw [T, k] FP32 out, or both NULL
 *   dy   [rows, d] out; rows that no slot has are left as they were.  May be
 *        y's own memory (every row is read before it is written).
 * Errors as moe_dispatch, and y without dw or the reverse. */
moe_status moe_collect_backward(moe_dtype type, const void* dout, const int32_t* pos, const float* w, const void* y,
                                int T, int k, int d, int rows, void* dy, float* dw, void* stream);

/* ---- Matrix products in 16 bits ----
 * Rows [offsets[g], offsets[g+1]) of the operands belong to group g, as
 * moe_sort and moe_permute order them; with offsets NULL and n_groups = 1 all
 * rows do (a dense product).  offsets [n_groups + 1] int32 on the device,
 * non-decreasing, from 0 to at most rows; rows from offsets[n_groups] on belong
 * to no group: they are not read, and their outputs are left as they were. */

typedef enum {
  MOE_ACT_NONE = 0,
  MOE_ACT_RELU = 1,
  MOE_ACT_SILU = 2,     /* z / (1 + e^-z); 0 below z = -87.3, where it is at most 2^-119 */
  MOE_ACT_GELU = 3,     /* z / 2 (1 + erf(z / sqrt 2)) */
  MOE_ACT_SWIGLU = 4    /* N = 2f: silu(z[:, 0:f]) * z[:, f:2f], f columns out */
} moe_act;

/* Bytes of device workspace grouped_gemm16 needs (0 where it needs none, and
 * for sizes it refuses). */
size_t grouped_gemm16_workspace_bytes(int rows, int n_groups, int K, int N, moe_act act);

/* grouped_gemm16 — for every row r of group g
 *   z = b[g] a_r + bias[g] (FP32),  out_r = act(z) + residual_r
 *   a         [rows, K];  b [n_groups, N, K];  bias [n_groups, N] or NULL, all
 *             of `type`
 *   residual  [rows, No] or NULL;  No = f for MOE_ACT_SWIGLU, else N
 *   pre       [rows, N] out: z, for the activation's gradient, or NULL
 *   out       [rows, No] out; may be residual's own memory
 *   workspace at least grouped_gemm16_workspace_bytes(...) bytes, 16-byte
 *             aligned (may be NULL when that is 0); overwritten; calls that
 *             share it must not overlap
 * rows = 0 is a no-op.  MOE_ERR_INVALID_ARG: K or No not a positive multiple of
 * 8, n_groups < 1, offsets NULL with n_groups > 1, an unknown type or act.
 * MOE_ERR_UNSUPPORTED: n_groups > 1024, rows > 2^31 - 1024, K or N > 2^20,
 * MOE_FP32.
 * MOE_ERR_WORKSPACE: workspace missing, misaligned or short. */
moe_status grouped_gemm16(moe_dtype type, const void* a, const int32_t* offsets, int n_groups, int rows, int K, int N,
                          const void* b, const void* bias, moe_act act, const void* residual, void* pre, void* out,
                          void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace grouped_act_backward needs for dbias (0 for sizes
 * it refuses). */
size_t grouped_act_backward_workspace_bytes(int rows, int n_groups, int N);

/* grouped_act_backward — gradient of the epilogue: dz = dout * act'(pre) (for
 * MOE_ACT_SWIGLU [dg, du] of both halves), and dbias[g] = the sum of the
 * group's rows of dz before they are rounded.  relu'(0) = 0.
 *   dout [rows, No];  pre [rows, N] (may be NULL for MOE_ACT_NONE)
 *   dz     [rows, N] out, or NULL; may be pre's own memory, and dout's where No = N
 *   dbias  [n_groups, N] FP32 out (zeros for a group without rows), or NULL
 *   workspace  for dbias, as above
 * rows = 0: dbias is zeros.  Errors as grouped_gemm16, and neither dz nor dbias. */
moe_status grouped_act_backward(moe_dtype type, const void* dout, const void* pre, const int32_t* offsets, int n_groups,
                                int rows, int N, moe_act act, void* dz, float* dbias, void* workspace,
                                size_t workspace_bytes, void* stream);

/* Bytes of device workspace grouped_gemm16_dgrad and grouped_gemm16_wgrad need
 * (0 where they need none, and for sizes they refuse). */
size_t grouped_gemm16_backward_workspace_bytes(int rows, int n_groups, int K, int N);

/* grouped_gemm16_dgrad — gradient of the rows: da_r = dz_r b[g] (+ residual_r).
 *   dz [rows, N];  b [n_groups, N, K];  residual [rows, K] or NULL
 *   da [rows, K] out; may be residual's own memory
 * Workspace and errors as grouped_gemm16, N and K multiples of 8. */
moe_status grouped_gemm16_dgrad(moe_dtype type, const void* dz, const int32_t* offsets, int n_groups, int rows, int K,
                                int N, const void* b, const void* residual, void* da, void* workspace,
                                size_t workspace_bytes, void* stream);

/* grouped_gemm16_wgrad — gradient of the weights: db[g] = dz_g^T a_g over the
 * group's rows.
 *   dz [rows, N];  a [rows, K];  db [n_groups, N, K] FP32 out (zeros for a
 *   group without rows, and for rows = 0), 16-byte aligned
 * Workspace and errors as grouped_gemm16_dgrad. */
moe_status grouped_gemm16_wgrad(moe_dtype type, const void* dz, const void* a, const int32_t* offsets, int n_groups,
                                int rows, int K, int N, float* db, void* workspace, size_t workspace_bytes,
                                void* stream);

/* ---- Dropout ---- */

/* moe_dropout — out_i = residual_i + (keep_i ? x_i / q : 0) over n elements.
 * keep_i is the generator's value for element i below q 2^16, with the
 * probability of keeping q = round((1 - p) 2^16) / 2^16: the scale belongs to
 * the q that is used, so the expectation is exact.  The value is 16-bit half
 * i mod 8 (low half of word 0 first) of Philox4x32-10 (Salmon, Moraes, Dror and
 * Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) with the key
 * rng[0] (low word first) and the counter (i / 8, rng[1]), 64 bits each, low
 * words first.  x of a dropped element counts for nothing, NaN or not.
 *   x, residual  [n], residual may be NULL;  p in [0, 1]
 *   rng   [2] int64 on the DEVICE, 8-byte aligned: {seed, call}.  A program
 *         gives every call a number of its own; read when the kernel runs, so
 *         that a captured graph drops other elements once they were changed.
 *   out   [n] out; may be x's or residual's own memory
 * n = 0 is a no-op.  MOE_ERR_INVALID_ARG: n < 0, p outside [0, 1] or NaN.
 * MOE_ERR_UNSUPPORTED: n > 2^40. */
moe_status moe_dropout(moe_dtype type, const void* x, const void* residual, int64_t n, float p, const int64_t* rng,
                       void* out, void* stream);

/* moe_dropout_backward — the gradient of x: dx_i = keep_i ? dout_i / q : 0 with
 * the forward's p and rng (whose values have to be the forward's still); that
 * of the residual is dout.  dx may be dout's own memory. */
moe_status moe_dropout_backward(moe_dtype type, const void* dout, int64_t n, float p, const int64_t* rng, void* dx,
                                void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_H */
