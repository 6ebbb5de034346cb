// Launch functions of the gfx950 kernels (host side of each .hip file).  Every
// function enqueues on `stream` and returns hipGetLastError(); arguments are
// validated by the C ABI layer before any of these is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

hipError_t launch_quant_1x128(const uint16_t* x, long rows, int cols, uint8_t* q, float* scale,
                              bool pow2, hipStream_t stream);
hipError_t launch_quant_128x128(const uint16_t* w, int N, int K, uint8_t* q, float* scale,
                                bool pow2, hipStream_t stream);

hipError_t launch_route(const uint16_t* x, const uint16_t* wg, const float* bias, int T, int d,
                        int E, int G, int M, int k, float route_scale, int32_t* idx, float* w,
                        hipStream_t stream);
size_t route_workspace_bytes(int T, int E);
hipError_t launch_route_ws(const uint16_t* x, const uint16_t* wg, const float* bias, int T, int d, int E,
                           int G, int M, int k, float route_scale, int32_t* idx, float* w, float* logits,
                           hipStream_t stream);

size_t permute_workspace_bytes(int T, int E);
// Largest workspace the allocation-free permute holds in its static device
// array (per-block histograms: ceil(T/256) * E int32).
constexpr size_t kPermuteScratchBytes = size_t(1) << 20;
hipError_t launch_permute_noalloc(const int32_t* idx, int T, int k, int E, const uint8_t* xq,
                                  const float* xs, int d, int32_t* offsets, int32_t* pos,
                                  int32_t* row_token, uint8_t* xq_perm, float* xs_perm,
                                  hipStream_t stream);
hipError_t launch_permute(const int32_t* idx, int T, int k, int E, const uint8_t* xq,
                          const float* xs, int d, int32_t* offsets, int32_t* pos,
                          int32_t* row_token, uint8_t* xq_perm, float* xs_perm, void* ws,
                          hipStream_t stream);

hipError_t launch_gemm_up(const uint8_t* aq, const float* as, int a_rows, const int32_t* row_src,
                          const int32_t* offsets, int n_groups, int total_rows, int d, int f,
                          const uint8_t* w13, const float* w13_s, uint8_t* h, float* hs,
                          bool e8m0, hipStream_t stream, uint8_t* gu = nullptr, float* gus = nullptr);
hipError_t launch_gemm_down(const uint8_t* h, const float* hs, const int32_t* offsets, int n_groups,
                            int total_rows, int d, int f, const uint8_t* w2, const float* w2_s,
                            uint16_t* y, bool e8m0, hipStream_t stream);

// Variants of the two expert GEMMs for few rows per group (weight streaming;
// launch_gemm_up/down choose them when total_rows <= 16 * n_groups and K is at
// most kSmallMaxK, the activation rows they stage in LDS).
constexpr int kSmallMaxK = 7168;
hipError_t launch_gemm_up_small(const uint8_t* aq, const float* as, int a_rows,
                                const int32_t* row_src, const int32_t* offsets, int n_groups,
                                int total_rows, int d, int f, const uint8_t* w13,
                                const float* w13_s, uint8_t* h, float* hs, bool pow2,
                                hipStream_t stream);
hipError_t launch_gemm_down_small(const uint8_t* h, const float* hs, const int32_t* offsets,
                                  int n_groups, int total_rows, int d, int f, const uint8_t* w2,
                                  const float* w2_s, uint16_t* y, hipStream_t stream);

hipError_t launch_bias_update(const int32_t* offsets, int E, float gamma, float* bias,
                              hipStream_t stream);

// Backward around the expert GEMMs (backward.hip).
hipError_t launch_transpose_blocks(const uint8_t* w, const float* ws, int G, int N, int K, uint8_t* wt,
                                   float* wts, hipStream_t stream);
hipError_t launch_combine_backward(const uint16_t* dout, const uint16_t* y, const int32_t* pos,
                                   const float* w, int T, int k, int d, int shared_row0, uint16_t* dy,
                                   float* dw, uint8_t* dyq, float* dys, hipStream_t stream);
int wgrad_blocks_bound(int total_rows, int n_groups);
hipError_t launch_regroup_128x1(const uint8_t* xq, const float* xs, const uint16_t* xb,
                                const int32_t* row_src, const int32_t* offsets, int n_groups,
                                int total_rows, int C, int Kp, uint8_t* out, float* out_s,
                                hipStream_t stream);
hipError_t launch_swiglu_backward(const uint8_t* guq, const float* gus, const uint16_t* dh,
                                  const int32_t* offsets, int n_groups, int total_rows, int f, int Kp,
                                  uint8_t* dguq, float* dgus, uint8_t* dgut, float* dguts, uint8_t* ht,
                                  float* hts, hipStream_t stream);

hipError_t launch_wgrad(const uint8_t* A, const float* sA, const uint8_t* B, const float* sB,
                        const int32_t* offsets, int n_groups, int M, int N, int Kp, float* out,
                        hipStream_t stream);

hipError_t launch_combine(const uint16_t* y, const int32_t* pos, const float* w, int T, int k,
                          int d, int shared_row0, const uint16_t* residual, uint16_t* out,
                          hipStream_t stream);

// The last-level cache: data of calls that move more than this goes past it.
constexpr size_t kCacheBytes = size_t(256) << 20;

// Residual addition + RMS norm + 1x128 quantisation, and its backward
// (norm.hip).  kNormMaxD: the widest row a workgroup holds in registers.
constexpr int kNormMaxD = 16384;
hipError_t launch_rmsnorm_quant(const uint16_t* x, const uint16_t* res, const uint16_t* w, int T, int d, float eps,
                                uint16_t* sum, uint16_t* y, uint8_t* q, float* scale, float* rstd, bool pow2,
                                hipStream_t stream);
int rmsnorm_backward_groups(int T, int d);
hipError_t launch_rmsnorm_backward(const uint16_t* dy, const uint16_t* h, const uint16_t* w, const float* rstd,
                                   const uint16_t* dres, int T, int d, uint16_t* dh, float* dw, float* partial,
                                   hipStream_t stream);

// The whole layer for a few tokens (few.hip).
constexpr int kFewMaxT = 16;
constexpr int kFewMaxD = 8192;
constexpr int kFewMaxF = 32768;
size_t layer_few_workspace_bytes(int T, int d, int f, int E, int k);
hipError_t launch_layer_few(const uint16_t* x, const uint16_t* wg, const float* bias, int T, int d, int f, int E,
                            int G, int M, int k, float route_scale, const uint8_t* w13, const float* w13_s,
                            const uint8_t* w2, const float* w2_s, const uint16_t* residual, int32_t* idx, float* w,
                            uint16_t* out, void* workspace, bool pow2, hipStream_t stream);

// Global gradient norm and scaling over lists of tensors (grad.hip).
size_t grad_norm_workspace_bytes(int n_tensors);
hipError_t launch_grad_norm(const void* const* grads, const int64_t* sizes, const int* types, int n_tensors,
                            float max_norm, float* norm, float* coef, double* partial, hipStream_t stream);
hipError_t launch_grad_scale(const void* const* grads, void* const* outs, const int64_t* sizes, const int* types,
                             int n_tensors, const float* coef, hipStream_t stream);

// Tokens sorted by expert and back (tokens.hip).  type: moe_dtype.
constexpr int kSortMaxK = 64, kSortMaxE = 1024;
size_t sort_workspace_bytes(int T, int k, int E);
hipError_t launch_sort(const int32_t* idx, int T, int k, int E, int32_t* offsets, int32_t* pos, int32_t* row_slot,
                       int32_t* counts, hipStream_t stream);
// rows of a token's slots = w * token row, and the rows of y times the token's
hipError_t launch_spread(int type, const void* x, const int32_t* pos, const float* w, const void* y, int T, int k, int d,
                         int rows, void* out, float* dots, hipStream_t stream);
// token row = sum of w * rows + residual, and the rows times x's
hipError_t launch_sum(int type, const void* rows_in, const int32_t* pos, const float* w, const void* x,
                      const void* residual, int T, int k, int d, int rows, void* out, float* dots, hipStream_t stream);

// Matrix products in 16 bits (gemm16.hip) and their activation's gradient
// (act.hip).  act: moe_act; group count up to groups.h's kMaxGroups.
size_t gemm16_workspace_bytes(int rows, int n_groups, int K, int N, int act);
hipError_t launch_gemm16(int type, const void* a, const int32_t* offsets, int n_groups, int rows, int K, int N,
                         const void* b, const void* bias, int act, const void* residual, void* pre, void* out,
                         void* workspace, hipStream_t stream);
size_t gemm16_backward_workspace_bytes(int rows, int n_groups, int K, int N);
hipError_t launch_gemm16_dgrad(int type, const void* dz, const int32_t* offsets, int n_groups, int rows, int K, int N,
                               const void* b, const void* residual, void* da, void* workspace, hipStream_t stream);
hipError_t launch_gemm16_wgrad(int type, const void* dz, const void* a, const int32_t* offsets, int n_groups, int rows,
                               int K, int N, float* db, void* workspace, hipStream_t stream);
size_t act_backward_workspace_bytes(int rows, int n_groups, int N);
hipError_t launch_act_backward(int type, const void* dout, const void* pre, const int32_t* offsets, int n_groups,
                               int rows, int N, int act, void* dz, float* dbias, float* partial, hipStream_t stream);

// Dropout (dropout.hip).
hipError_t launch_dropout(int type, const void* x, const void* residual, int64_t n, float p, const int64_t* rng,
                          void* out, hipStream_t stream);

// Measured roofs (roofs.hip): FP8 MFMA issue rate and HBM read streaming.
hipError_t launch_roof_mfma(int workgroups, int iters, float* sink, hipStream_t stream);
hipError_t launch_roof_dma(const void* buf, size_t bytes, int K, int ahead, int workgroups, uint32_t* sink,
                           hipStream_t stream);
hipError_t launch_roof_chase(const uint32_t* next, size_t n, uint32_t start, int steps, uint32_t* sink,
                             hipStream_t stream);
hipError_t launch_roof_read(const void* buf, size_t bytes, int workgroups, uint32_t* sink,
                            hipStream_t stream);

}  // namespace moe
