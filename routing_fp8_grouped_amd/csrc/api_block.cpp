// C ABI of include/moe_block.h: host-side validation, then launches on the
// caller's stream, as api.cpp does for moe.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <utility>
#include <vector>

#include "check.h"
#include "kernels.h"
#include "moe_block.h"

namespace {

moe_status check_norm_shape(int T, int d) {
  REQUIRE(T >= 0, "T=%d is negative", T);
  REQUIRE(d >= 128 && d % 128 == 0, "d=%d must be a positive multiple of 128", d);
  if (d > moe::kNormMaxD) return fail(MOE_ERR_UNSUPPORTED, "d=%d > %d is not implemented", d, moe::kNormMaxD);
  return MOE_OK;
}

#define REQUIRE_ALIGNED_OR_NULL(p)                                                                          \
  do {                                                                                                      \
    if ((p) != nullptr && !aligned16(p)) return fail(MOE_ERR_INVALID_ARG, "%s is not 16-byte aligned", #p); \
  } while (0)

// An operand's memory; NULL: not given.
struct Span {
  const char* name;
  const void* p;
  size_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x != 0 && y != 0 && x < y + b.bytes && y < x + a.bytes;
}
// No output shares memory with an input (but for `same`, whose operand it may
// be as a whole) or with another output.
struct Out {
  Span span;
  std::initializer_list<const void*> same;
};
moe_status check_apart(std::initializer_list<Out> outs, std::initializer_list<Span> ins) {
  for (const Out* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins) {
      bool allowed = false;
      for (const void* s : o->same) allowed = allowed || (s == i.p && s == o->span.p);
      REQUIRE(allowed || !overlap(o->span, i), "%s must not share memory with %s", o->span.name, i.name);
    }
    for (const Out* b = outs.begin(); b != o; ++b)
      REQUIRE(!overlap(o->span, b->span), "%s must not share memory with %s", o->span.name, b->span.name);
  }
  return MOE_OK;
}

moe_status rmsnorm_impl(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int T, int d, float eps,
                        uint16_t* sum, uint16_t* y, uint8_t* q, float* scale, float* rstd, bool pow2, void* stream) {
  moe_status s = check_norm_shape(T, d);
  if (s != MOE_OK) return s;
  REQUIRE(std::isfinite(eps) && eps > 0.0f, "eps=%g must be positive and finite", (double)eps);
  REQUIRE((q == nullptr) == (scale == nullptr), "q and scale must be given together");
  if (T == 0) return MOE_OK;
  REQUIRE(sum != nullptr || y != nullptr || q != nullptr || rstd != nullptr, "no output is given");
  REQUIRE_PTR(x);
  REQUIRE_ALIGNED_OR_NULL(residual);
  REQUIRE_PTR(weight);
  REQUIRE_ALIGNED_OR_NULL(sum);
  REQUIRE_ALIGNED_OR_NULL(y);
  REQUIRE_ALIGNED_OR_NULL(q);
  REQUIRE_ALIGNED4_OR_NULL(scale);
  REQUIRE_ALIGNED4_OR_NULL(rstd);
  const size_t n = (size_t)T * d, row = (size_t)T * 4;
  s = check_apart({{{"sum", sum, 2 * n}, {x, residual}},
                   {{"y", y, 2 * n}, {}},
                   {{"q", q, n}, {}},
                   {{"scale", scale, n / 32}, {}},
                   {{"rstd", rstd, row}, {}}},
                  {{"x", x, 2 * n}, {"residual", residual, 2 * n}, {"weight", weight, (size_t)d * 2}});
  if (s != MOE_OK) return s;
  return hip_status(moe::launch_rmsnorm_quant(x, residual, weight, T, d, eps, sum, y, q, scale, rstd, pow2,
                                              static_cast<hipStream_t>(stream)),
                    pow2 ? "moe_rmsnorm_quant_pow2 launch" : "moe_rmsnorm_quant launch");
}

size_t rmsnorm_backward_bytes(int T, int d) {
  if (T <= 0 || d < 128 || d % 128 != 0 || d > moe::kNormMaxD) return 0;
  return (size_t)moe::rmsnorm_backward_groups(T, d) * d * sizeof(float);
}

moe_status check_few(int T, int d, int f, int E, int k) {
  REQUIRE(T >= 0, "T=%d is negative", T);
  REQUIRE(d >= 128 && d % 128 == 0, "d=%d must be a positive multiple of 128", d);
  REQUIRE(f >= 128 && f % 128 == 0, "f=%d must be a positive multiple of 128", f);
  REQUIRE(E >= 1 && E <= 256, "E=%d must be in [1, 256]", E);
  REQUIRE(k >= 1 && k <= 16 && k <= E, "k=%d must be in [1, min(16, E)]", k);
  if (T > moe::kFewMaxT) return fail(MOE_ERR_UNSUPPORTED, "T=%d > %d is not implemented", T, moe::kFewMaxT);
  if (d > moe::kFewMaxD) return fail(MOE_ERR_UNSUPPORTED, "d=%d > %d is not implemented", d, moe::kFewMaxD);
  if (f > moe::kFewMaxF) return fail(MOE_ERR_UNSUPPORTED, "f=%d > %d is not implemented", f, moe::kFewMaxF);
  return MOE_OK;
}

moe_status layer_few_impl(const uint16_t* x, const uint16_t* wg, const float* bias, int T, int d, int f,
                          moe_route_params p, const uint8_t* w13, const float* w13_s, const uint8_t* w2,
                          const float* w2_s, const uint16_t* residual, int32_t* idx, float* w, uint16_t* out,
                          void* workspace, size_t workspace_bytes, bool pow2, void* stream) {
  moe_status s = check_route_params(p);
  if (s == MOE_OK) s = check_few(T, d, f, p.n_experts, p.topk);
  if (s != MOE_OK || T == 0) return s;
  REQUIRE_PTR(x);
  REQUIRE_PTR(wg);
  REQUIRE_ALIGNED4_OR_NULL(bias);
  REQUIRE_PTR(w13);
  REQUIRE_PTR4(w13_s);
  REQUIRE_PTR(w2);
  REQUIRE_PTR4(w2_s);
  REQUIRE_ALIGNED_OR_NULL(residual);
  REQUIRE_PTR4(idx);
  REQUIRE_PTR4(w);
  REQUIRE_PTR(out);
  const size_t need = moe::layer_few_workspace_bytes(T, d, f, p.n_experts, p.topk);
  if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "workspace %p of %zu bytes: %zu bytes, 16-byte aligned, needed", workspace,
                workspace_bytes, need);
  const size_t n = (size_t)T * d * 2, sel = (size_t)T * p.topk * 4, E = p.n_experts, wn = (E + 1) * f * d;
  s = check_apart({{{"out", out, n}, {x, residual}},
                   {{"idx", idx, sel}, {}},
                   {{"w", w, sel}, {}},
                   {{"workspace", workspace, need}, {}}},
                  {{"x", x, n}, {"residual", residual, n}, {"wg", wg, E * d * 2}, {"bias", bias, E * 4},
                   {"w13", w13, 2 * wn}, {"w13_s", w13_s, wn / 2048}, {"w2", w2, wn}, {"w2_s", w2_s, wn / 4096}});
  if (s != MOE_OK) return s;
  return hip_status(moe::launch_layer_few(x, wg, bias, T, d, f, p.n_experts, p.n_groups, p.topk_groups, p.topk,
                                          p.route_scale, w13, w13_s, w2, w2_s, residual, idx, w, out, workspace,
                                          pow2, static_cast<hipStream_t>(stream)),
                    pow2 ? "moe_layer_few_pow2 launch" : "moe_layer_few launch");
}

moe_status check_grads(const void* const* grads, const int64_t* sizes, const int* types, int n_tensors) {
  REQUIRE(n_tensors >= 0, "n_tensors=%d is negative", n_tensors);
  if (n_tensors == 0) return MOE_OK;
  REQUIRE(grads != nullptr, "grads is NULL");
  REQUIRE(sizes != nullptr, "sizes is NULL");
  REQUIRE(types != nullptr, "types is NULL");
  for (int i = 0; i < n_tensors; ++i) {
    REQUIRE(sizes[i] >= 0 && sizes[i] <= (INT64_C(1) << 40), "sizes[%d]=%lld must be in [0, 2^40]", i,
            (long long)sizes[i]);
    REQUIRE(types[i] == MOE_GRAD_FP32 || types[i] == MOE_GRAD_BF16, "types[%d]=%d is not a moe_grad_type", i,
            types[i]);
    if (sizes[i] == 0) continue;
    REQUIRE(grads[i] != nullptr, "grads[%d] is NULL", i);
    REQUIRE(aligned(grads[i], types[i] == MOE_GRAD_FP32 ? 4 : 2), "grads[%d] is not aligned to its elements", i);
  }
  return MOE_OK;
}

size_t grad_bytes(const int64_t* sizes, const int* types, int i) {
  return (size_t)sizes[i] * (types[i] == MOE_GRAD_FP32 ? 4 : 2);
}

// No output shares memory with another output (a tensor listed twice would be
// scaled twice), with another tensor's gradient or with coef.
moe_status check_disjoint(const void* const* grads, void* const* outs, const int64_t* sizes, const int* types,
                          int n_tensors, const float* coef) {
  try {
    std::vector<std::pair<uintptr_t, uintptr_t>> at;
    at.reserve(n_tensors);
    auto bytes = [&](int i) { return grad_bytes(sizes, types, i); };
    for (int i = 0; i < n_tensors; ++i) {
      if (sizes[i] == 0) continue;
      const uintptr_t o = reinterpret_cast<uintptr_t>(outs[i]);
      at.emplace_back(o, o + bytes(i));
    }
    std::sort(at.begin(), at.end());
    for (size_t i = 1; i < at.size(); ++i) REQUIRE(at[i - 1].second <= at[i].first, "two outputs overlap");
    // the outputs being apart, the last one that starts before `end` tells
    auto touched = [&](uintptr_t begin, uintptr_t end) {
      const auto it = std::lower_bound(at.begin(), at.end(), std::make_pair(end, (uintptr_t)0));
      return it != at.begin() && (it - 1)->second > begin;
    };
    for (int i = 0; i < n_tensors; ++i) {
      const uintptr_t g = reinterpret_cast<uintptr_t>(grads[i]);
      if (sizes[i] != 0 && grads[i] != outs[i])   // in place: an output of its own, apart from the others
        REQUIRE(!touched(g, g + bytes(i)), "an output overlaps grads[%d] in part, or another tensor's", i);
    }
    const uintptr_t c = reinterpret_cast<uintptr_t>(coef);
    REQUIRE(!touched(c, c + sizeof(float)), "an output overlaps coef");
  } catch (...) {
    return fail(MOE_ERR_INVALID_ARG, "n_tensors=%d: out of host memory", n_tensors);
  }
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_rmsnorm_quant(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int T, int d,
                             float eps, uint16_t* sum, uint16_t* y, uint8_t* q, float* scale, float* rstd,
                             void* stream) {
  clear_error();
  return rmsnorm_impl(x, residual, weight, T, d, eps, sum, y, q, scale, rstd, false, stream);
}

moe_status moe_rmsnorm_quant_pow2(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int T, int d,
                                  float eps, uint16_t* sum, uint16_t* y, uint8_t* q, float* scale, float* rstd,
                                  void* stream) {
  clear_error();
  return rmsnorm_impl(x, residual, weight, T, d, eps, sum, y, q, scale, rstd, true, stream);
}

size_t moe_rmsnorm_backward_workspace_bytes(int T, int d) { return rmsnorm_backward_bytes(T, d); }

moe_status moe_rmsnorm_backward(const uint16_t* dy, const uint16_t* h, const uint16_t* weight, const float* rstd,
                                const uint16_t* dres, int T, int d, uint16_t* dh, float* dweight, void* workspace,
                                size_t workspace_bytes, void* stream) {
  clear_error();
  moe_status s = check_norm_shape(T, d);
  if (s != MOE_OK) return s;
  REQUIRE_PTR4(dweight);
  if (T > 0) {
    REQUIRE_PTR(dy);
    REQUIRE_PTR(h);
    REQUIRE_PTR(weight);
    REQUIRE_PTR4(rstd);
    REQUIRE_ALIGNED_OR_NULL(dres);
    REQUIRE_PTR(dh);
    const size_t need = rmsnorm_backward_bytes(T, d);
    if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < need)
      return fail(MOE_ERR_WORKSPACE, "workspace %p of %zu bytes: %zu bytes, 16-byte aligned, needed", workspace,
                  workspace_bytes, need);
    const size_t n = (size_t)T * d * 2;
    s = check_apart({{{"dh", dh, n}, {dres}},
                     {{"dweight", dweight, (size_t)d * 4}, {}},
                     {{"workspace", workspace, need}, {}}},
                    {{"dy", dy, n}, {"h", h, n}, {"weight", weight, (size_t)d * 2}, {"rstd", rstd, (size_t)T * 4},
                     {"dres", dres, n}});
    if (s != MOE_OK) return s;
  }
  return hip_status(moe::launch_rmsnorm_backward(dy, h, weight, rstd, dres, T, d, dh, dweight,
                                                 static_cast<float*>(workspace), static_cast<hipStream_t>(stream)),
                    "moe_rmsnorm_backward launch");
}

size_t moe_layer_few_workspace_bytes(int T, int d, int f, int E, int k) {
  if (T <= 0 || T > moe::kFewMaxT || d < 128 || d % 128 != 0 || d > moe::kFewMaxD || f < 128 || f % 128 != 0 ||
      f > moe::kFewMaxF || E < 1 || E > 256 || k < 1 || k > 16 || k > E)
    return 0;
  return moe::layer_few_workspace_bytes(T, d, f, E, k);
}

moe_status moe_layer_few(const uint16_t* x, const uint16_t* wg, const float* bias, int T, int d, int f,
                         moe_route_params p, const uint8_t* w13, const float* w13_s, const uint8_t* w2,
                         const float* w2_s, const uint16_t* residual, int32_t* idx, float* w, uint16_t* out,
                         void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  return layer_few_impl(x, wg, bias, T, d, f, p, w13, w13_s, w2, w2_s, residual, idx, w, out, workspace,
                        workspace_bytes, false, stream);
}

moe_status moe_layer_few_pow2(const uint16_t* x, const uint16_t* wg, const float* bias, int T, int d, int f,
                              moe_route_params p, const uint8_t* w13, const float* w13_s, const uint8_t* w2,
                              const float* w2_s, const uint16_t* residual, int32_t* idx, float* w, uint16_t* out,
                              void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  return layer_few_impl(x, wg, bias, T, d, f, p, w13, w13_s, w2, w2_s, residual, idx, w, out, workspace,
                        workspace_bytes, true, stream);
}

size_t moe_grad_norm_workspace_bytes(int n_tensors) {
  return n_tensors <= 0 ? 0 : moe::grad_norm_workspace_bytes(n_tensors);
}

moe_status moe_grad_norm(const void* const* grads, const int64_t* sizes, const int* types, int n_tensors,
                         float max_norm, float* norm, float* coef, void* workspace, size_t workspace_bytes,
                         void* stream) {
  clear_error();
  moe_status s = check_grads(grads, sizes, types, n_tensors);
  if (s != MOE_OK) return s;
  REQUIRE(max_norm > 0.0f, "max_norm=%g must be positive", (double)max_norm);
  REQUIRE_PTR4(norm);
  REQUIRE_PTR4(coef);
  const size_t need = moe_grad_norm_workspace_bytes(n_tensors);
  if (need > 0 && (workspace == nullptr || !aligned(workspace, 8) || workspace_bytes < need))
    return fail(MOE_ERR_WORKSPACE, "workspace %p of %zu bytes: %zu bytes, 8-byte aligned, needed", workspace,
                workspace_bytes, need);
  const Span outs[] = {{"norm", norm, 4}, {"coef", coef, 4}, {"workspace", workspace, need}};
  s = check_apart({{outs[0], {}}, {outs[1], {}}, {outs[2], {}}}, {});
  if (s != MOE_OK) return s;
  // partial sums and results are written while other workgroups still read
  for (const Span& o : outs)
    for (int i = 0; i < n_tensors; ++i)
      REQUIRE(sizes[i] == 0 || !overlap(o, {"", grads[i], grad_bytes(sizes, types, i)}),
              "%s must not share memory with grads[%d]", o.name, i);
  return hip_status(moe::launch_grad_norm(grads, sizes, types, n_tensors, max_norm, norm, coef,
                                          static_cast<double*>(workspace), static_cast<hipStream_t>(stream)),
                    "moe_grad_norm launch");
}

moe_status moe_grad_scale(const void* const* grads, void* const* outs, const int64_t* sizes, const int* types,
                          int n_tensors, const float* coef, void* stream) {
  clear_error();
  moe_status s = check_grads(grads, sizes, types, n_tensors);
  if (s != MOE_OK) return s;
  REQUIRE_PTR4(coef);
  if (n_tensors == 0) return MOE_OK;
  REQUIRE(outs != nullptr, "outs is NULL");
  for (int i = 0; i < n_tensors; ++i) {
    if (sizes[i] == 0) continue;
    REQUIRE(outs[i] != nullptr, "outs[%d] is NULL", i);
    REQUIRE(aligned(outs[i], types[i] == MOE_GRAD_FP32 ? 4 : 2), "outs[%d] is not aligned to its elements", i);
  }
  s = check_disjoint(grads, outs, sizes, types, n_tensors, coef);
  if (s != MOE_OK) return s;
  return hip_status(moe::launch_grad_scale(grads, outs, sizes, types, n_tensors, coef,
                                           static_cast<hipStream_t>(stream)),
                    "moe_grad_scale launch");
}

}  // extern "C"
