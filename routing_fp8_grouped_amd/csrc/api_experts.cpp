// C ABI of include/moe_experts.h: host-side validation, then launches on the
// caller's stream, as api.cpp does for moe.h.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "check.h"
#include "groups.h"
#include "kernels.h"
#include "moe_experts.h"

namespace {

constexpr int64_t kMaxElements = INT64_C(1) << 40;

size_t bytes_of(moe_dtype type) { return type == MOE_FP32 ? 4 : 2; }

moe_status check_type(moe_dtype type) {
  REQUIRE(type == MOE_BF16 || type == MOE_FP16 || type == MOE_FP32, "type=%d is not a moe_dtype", (int)type);
  return MOE_OK;
}

moe_status check_workspace(const void* workspace, size_t bytes, size_t need, uintptr_t align) {
  if (need > 0 && (workspace == nullptr || !aligned(workspace, align) || bytes < need))
    return fail(MOE_ERR_WORKSPACE, "workspace %p of %zu bytes: %zu bytes, %d-byte aligned, needed", workspace, bytes,
                need, (int)align);
  return MOE_OK;
}

moe_status check_sort(int T, int k, int E) {
  REQUIRE(T >= 0, "T=%d is negative", T);
  REQUIRE(k >= 1, "k=%d must be positive", k);
  REQUIRE(E >= 1, "E=%d must be positive", E);
  if (k > moe::kSortMaxK) return fail(MOE_ERR_UNSUPPORTED, "k=%d > %d is not implemented", k, moe::kSortMaxK);
  if (E > moe::kSortMaxE) return fail(MOE_ERR_UNSUPPORTED, "E=%d > %d is not implemented", E, moe::kSortMaxE);
  if ((int64_t)T * k > (1 << 30)) return fail(MOE_ERR_UNSUPPORTED, "T*k=%lld > 2^30", (long long)T * k);
  return MOE_OK;
}

moe_status check_copy(moe_dtype type, const int32_t* pos, const float* w, int T, int k, int d, int rows) {
  moe_status s = check_type(type);
  if (s != MOE_OK) return s;
  REQUIRE(T >= 0, "T=%d is negative", T);
  REQUIRE(rows >= 0, "rows=%d is negative", rows);
  REQUIRE(k >= 1, "k=%d must be positive", k);
  REQUIRE(d >= 1, "d=%d must be positive", d);
  if (k > moe::kSortMaxK) return fail(MOE_ERR_UNSUPPORTED, "k=%d > %d is not implemented", k, moe::kSortMaxK);
  if ((int64_t)T * d > kMaxElements || (int64_t)rows * d > kMaxElements)
    return fail(MOE_ERR_UNSUPPORTED, "T=%d or rows=%d times d=%d is above 2^40", T, rows, d);
  if (T == 0) return MOE_OK;
  REQUIRE_PTR4(pos);
  REQUIRE_ALIGNED4_OR_NULL(w);
  return MOE_OK;
}

struct CopySizes {
  size_t tokens, rows, slots;
  CopySizes(moe_dtype type, int T, int k, int d, int r)
      : tokens((size_t)T * d * bytes_of(type)), rows((size_t)r * d * bytes_of(type)), slots((size_t)T * k * 4) {}
};

moe_status spread(moe_dtype type, const void* x, const int32_t* pos, const float* w, const void* y, int T, int k, int d,
                  int rows, void* out, float* dw, const char* x_name, const char* out_name, const char* what,
                  void* stream) {
  moe_status s = check_copy(type, pos, w, T, k, d, rows);
  if (s != MOE_OK) return s;
  REQUIRE((y == nullptr) == (dw == nullptr) || rows == 0, "y and dw must be given together");
  if (T == 0) return MOE_OK;
  REQUIRE(x != nullptr && aligned16(x), "%s is NULL or not 16-byte aligned", x_name);
  REQUIRE(rows == 0 || (out != nullptr && aligned16(out)), "%s is NULL or not 16-byte aligned", out_name);
  REQUIRE_ALIGNED_OR_NULL(y);
  REQUIRE_ALIGNED4_OR_NULL(dw);
  const CopySizes n(type, T, k, d, rows);
  s = check_apart({{{out_name, out, n.rows}, {"y"}}, {{"dw", dw, n.slots}, {}}},
                  {{x_name, x, n.tokens}, {"pos", pos, n.slots}, {"w", w, n.slots}, {"y", y, n.rows}});
  if (s != MOE_OK) return s;
  return hip_status(moe::launch_spread(type, x, pos, w, y, T, k, d, rows, out, dw, static_cast<hipStream_t>(stream)), what);
}

moe_status sum(moe_dtype type, const void* in, const int32_t* pos, const float* w, const void* x, const void* residual,
               int T, int k, int d, int rows, void* out, float* dw, const char* in_name, const char* out_name,
               const char* what, void* stream) {
  moe_status s = check_copy(type, pos, w, T, k, d, rows);
  if (s != MOE_OK) return s;
  REQUIRE((x == nullptr) == (dw == nullptr), "x and dw must be given together");
  if (T == 0) return MOE_OK;
  REQUIRE(rows == 0 || (in != nullptr && aligned16(in)), "%s is NULL or not 16-byte aligned", in_name);
  REQUIRE(out != nullptr && aligned16(out), "%s is NULL or not 16-byte aligned", out_name);
  REQUIRE_ALIGNED_OR_NULL(x);
  REQUIRE_ALIGNED_OR_NULL(residual);
  REQUIRE_ALIGNED4_OR_NULL(dw);
  const CopySizes n(type, T, k, d, rows);
  s = check_apart({{{out_name, out, n.tokens}, {"residual"}}, {{"dw", dw, n.slots}, {}}},
                  {{in_name, in, n.rows}, {"pos", pos, n.slots}, {"w", w, n.slots}, {"x", x, n.tokens},
                   {"residual", residual, n.tokens}});
  if (s != MOE_OK) return s;
  return hip_status(moe::launch_sum(type, in, pos, w, x, residual, T, k, d, rows, out, dw,
                                    static_cast<hipStream_t>(stream)), what);
}

// ---- products ----

// Sizes that every product shares; glu: N's halves have to be whole 16-byte chunks.
moe_status check_product(int n_groups, int rows, int K, int N, bool glu) {
  REQUIRE(rows >= 0, "rows=%d is negative", rows);
  REQUIRE(n_groups >= 1, "n_groups=%d must be positive", n_groups);
  REQUIRE(K >= 8 && K % 8 == 0, "K=%d must be a positive multiple of 8", K);
  const int unit = glu ? 16 : 8;
  REQUIRE(N >= unit && N % unit == 0, "N=%d must be a positive multiple of %d", N, unit);
  if (n_groups > moe::kMaxGroups)
    return fail(MOE_ERR_UNSUPPORTED, "n_groups=%d > %d is not implemented", n_groups, moe::kMaxGroups);
  if (rows > moe::kMaxRows) return fail(MOE_ERR_UNSUPPORTED, "rows=%d > %d is not implemented", rows, moe::kMaxRows);
  if (K > (1 << 20) || N > (1 << 20)) return fail(MOE_ERR_UNSUPPORTED, "K=%d or N=%d is above 2^20", K, N);
  return MOE_OK;
}
moe_status check_type16(moe_dtype type) {
  moe_status s = check_type(type);
  if (s == MOE_OK && type == MOE_FP32) s = fail(MOE_ERR_UNSUPPORTED, "MOE_FP32 operands are not implemented");
  return s;
}
moe_status check_offsets(const int32_t* offsets, int n_groups) {
  REQUIRE(offsets != nullptr || n_groups == 1, "offsets is NULL with n_groups=%d", n_groups);
  REQUIRE_ALIGNED4_OR_NULL(offsets);
  return MOE_OK;
}
moe_status check_act(moe_act act) {
  REQUIRE(act >= MOE_ACT_NONE && act <= MOE_ACT_SWIGLU, "act=%d is not a moe_act", (int)act);
  return MOE_OK;
}
size_t offsets_bytes(int n_groups) { return ((size_t)n_groups + 1) * 4; }

}  // namespace

extern "C" {

size_t moe_sort_workspace_bytes(int T, int k, int E) {
  if (T <= 0 || k < 1 || k > moe::kSortMaxK || E < 1 || E > moe::kSortMaxE || (int64_t)T * k > (1 << 30)) return 0;
  return moe::sort_workspace_bytes(T, k, E);
}

moe_status moe_sort(const int32_t* idx, int T, int k, int E, int32_t* offsets, int32_t* pos, int32_t* row_slot,
                    void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  moe_status s = check_sort(T, k, E);
  if (s != MOE_OK) return s;
  REQUIRE_PTR4(offsets);
  const size_t need = moe_sort_workspace_bytes(T, k, E), n = (size_t)T * k * 4;
  if (T > 0) {
    REQUIRE_PTR4(idx);
    REQUIRE_PTR4(pos);
    REQUIRE_PTR4(row_slot);
    s = check_workspace(workspace, workspace_bytes, need, 4);
    if (s == MOE_OK)
      s = check_apart({{{"offsets", offsets, offsets_bytes(E)}, {}}, {{"pos", pos, n}, {}}, {{"row_slot", row_slot, n}, {}},
                       {{"workspace", need ? workspace : nullptr, need}, {}}}, {{"idx", idx, n}});
    if (s != MOE_OK) return s;
  }
  return hip_status(moe::launch_sort(idx, T, k, E, offsets, pos, row_slot, static_cast<int32_t*>(workspace),
                                     static_cast<hipStream_t>(stream)), "moe_sort launch");
}

moe_status moe_dispatch(moe_dtype type, const void* x, const int32_t* pos, const float* w, int T, int k, int d, int rows,
                        void* out, void* stream) {
  clear_error();
  return spread(type, x, pos, w, nullptr, T, k, d, rows, out, nullptr, "x", "out", "moe_dispatch launch", stream);
}

moe_status moe_dispatch_backward(moe_dtype type, const void* drows, const int32_t* pos, const float* w, const void* x,
                                 const void* residual, int T, int k, int d, int rows, void* dx, float* dw,
                                 void* stream) {
  clear_error();
  return sum(type, drows, pos, w, x, residual, T, k, d, rows, dx, dw, "drows", "dx", "moe_dispatch_backward launch",
             stream);
}

moe_status moe_collect(moe_dtype type, const void* y, const int32_t* pos, const float* w, const void* residual, int T,
                       int k, int d, int rows, void* out, void* stream) {
  clear_error();
  return sum(type, y, pos, w, nullptr, residual, T, k, d, rows, out, nullptr, "y", "out", "moe_collect launch", stream);
}

moe_status moe_collect_backward(moe_dtype type, const void* dout, const int32_t* pos, const float* w, const void* y,
                                int T, int k, int d, int rows, void* dy, float* dw, void* stream) {
  clear_error();
  return spread(type, dout, pos, w, y, T, k, d, rows, dy, dw, "dout", "dy", "moe_collect_backward launch", stream);
}

size_t grouped_gemm16_workspace_bytes(int rows, int n_groups, int K, int N, moe_act act) {
  clear_error();
  if (check_act(act) != MOE_OK || check_product(n_groups, rows, K, N, act == MOE_ACT_SWIGLU) != MOE_OK || rows == 0) {
    clear_error();
    return 0;
  }
  return moe::gemm16_workspace_bytes(rows, n_groups, K, N, act);
}

moe_status grouped_gemm16(moe_dtype type, const void* a, const int32_t* offsets, int n_groups, int rows, int K, int N,
                          const void* b, const void* bias, moe_act act, const void* residual, void* pre, void* out,
                          void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  moe_status s = check_type16(type);
  if (s == MOE_OK) s = check_act(act);
  if (s == MOE_OK) s = check_product(n_groups, rows, K, N, act == MOE_ACT_SWIGLU);
  if (s == MOE_OK) s = check_offsets(offsets, n_groups);
  if (s != MOE_OK || rows == 0) return s;
  REQUIRE_PTR(a);
  REQUIRE_PTR(b);
  REQUIRE_ALIGNED_OR_NULL(bias);
  REQUIRE_ALIGNED_OR_NULL(residual);
  REQUIRE_ALIGNED_OR_NULL(pre);
  REQUIRE_PTR(out);
  const size_t need = moe::gemm16_workspace_bytes(rows, n_groups, K, N, act);
  s = check_workspace(workspace, workspace_bytes, need, 16);
  if (s != MOE_OK) return s;
  const size_t R = rows, G = n_groups, No = act == MOE_ACT_SWIGLU ? N / 2 : N;
  s = check_apart({{{"out", out, 2 * R * No}, {"residual"}}, {{"pre", pre, 2 * R * N}, {}},
                   {{"workspace", need ? workspace : nullptr, need}, {}}},
                  {{"a", a, 2 * R * K}, {"b", b, 2 * G * N * K}, {"bias", bias, 2 * G * N},
                   {"residual", residual, 2 * R * No}, {"offsets", offsets, offsets_bytes(n_groups)}});
  if (s != MOE_OK) return s;
  return hip_status(moe::launch_gemm16(type, a, offsets, n_groups, rows, K, N, b, bias, act, residual, pre, out,
                                       workspace, static_cast<hipStream_t>(stream)), "grouped_gemm16 launch");
}

size_t grouped_act_backward_workspace_bytes(int rows, int n_groups, int N) {
  clear_error();
  if (check_product(n_groups, rows, 8, N, false) != MOE_OK) {
    clear_error();
    return 0;
  }
  return moe::act_backward_workspace_bytes(rows, n_groups, N);
}

moe_status grouped_act_backward(moe_dtype type, const void* dout, const void* pre, const int32_t* offsets, int n_groups,
                                int rows, int N, moe_act act, void* dz, float* dbias, void* workspace,
                                size_t workspace_bytes, void* stream) {
  clear_error();
  moe_status s = check_type16(type);
  if (s == MOE_OK) s = check_act(act);
  if (s == MOE_OK) s = check_product(n_groups, rows, 8, N, act == MOE_ACT_SWIGLU);
  if (s == MOE_OK) s = check_offsets(offsets, n_groups);
  if (s != MOE_OK) return s;
  REQUIRE(dz != nullptr || dbias != nullptr, "no output is given");
  REQUIRE_ALIGNED4_OR_NULL(dbias);
  const size_t need = dbias ? moe::act_backward_workspace_bytes(rows, n_groups, N) : 0;
  if (rows > 0) {
    REQUIRE_PTR(dout);
    if (act != MOE_ACT_NONE) REQUIRE_PTR(pre);
    REQUIRE_ALIGNED_OR_NULL(dz);
    s = check_workspace(workspace, workspace_bytes, need, 4);
    if (s != MOE_OK) return s;
    const size_t R = rows, G = n_groups, No = act == MOE_ACT_SWIGLU ? N / 2 : N;
    const void* used = act == MOE_ACT_NONE ? nullptr : pre;
    s = check_apart({{{"dz", dz, 2 * R * N}, {"pre", "dout"}}, {{"dbias", dbias, 4 * G * N}, {}},
                     {{"workspace", need ? workspace : nullptr, need}, {}}},
                    {{"dout", dout, 2 * R * No}, {"pre", used, 2 * R * N},
                     {"offsets", offsets, offsets_bytes(n_groups)}});
    if (s != MOE_OK) return s;
  }
  return hip_status(moe::launch_act_backward(type, dout, pre, offsets, n_groups, rows, N, act, dz, dbias,
                                             static_cast<float*>(workspace), static_cast<hipStream_t>(stream)),
                    "grouped_act_backward launch");
}

size_t grouped_gemm16_backward_workspace_bytes(int rows, int n_groups, int K, int N) {
  clear_error();
  if (check_product(n_groups, rows, K, N, false) != MOE_OK || rows == 0) {
    clear_error();
    return 0;
  }
  return moe::gemm16_backward_workspace_bytes(rows, n_groups, K, N);
}

moe_status grouped_gemm16_dgrad(moe_dtype type, const void* dz, const int32_t* offsets, int n_groups, int rows, int K,
                                int N, const void* b, const void* residual, void* da, void* workspace,
                                size_t workspace_bytes, void* stream) {
  clear_error();
  moe_status s = check_type16(type);
  if (s == MOE_OK) s = check_product(n_groups, rows, K, N, false);
  if (s == MOE_OK) s = check_offsets(offsets, n_groups);
  if (s != MOE_OK || rows == 0) return s;
  REQUIRE_PTR(dz);
  REQUIRE_PTR(b);
  REQUIRE_ALIGNED_OR_NULL(residual);
  REQUIRE_PTR(da);
  const size_t need = moe::gemm16_backward_workspace_bytes(rows, n_groups, K, N);
  s = check_workspace(workspace, workspace_bytes, need, 16);
  if (s != MOE_OK) return s;
  const size_t R = rows, G = n_groups;
  s = check_apart({{{"da", da, 2 * R * K}, {"residual"}}, {{"workspace", need ? workspace : nullptr, need}, {}}},
                  {{"dz", dz, 2 * R * N}, {"b", b, 2 * G * N * K}, {"residual", residual, 2 * R * K},
                   {"offsets", offsets, offsets_bytes(n_groups)}});
  if (s != MOE_OK) return s;
  return hip_status(moe::launch_gemm16_dgrad(type, dz, offsets, n_groups, rows, K, N, b, residual, da, workspace,
                                             static_cast<hipStream_t>(stream)), "grouped_gemm16_dgrad launch");
}

moe_status grouped_gemm16_wgrad(moe_dtype type, const void* dz, const void* a, const int32_t* offsets, int n_groups,
                                int rows, int K, int N, float* db, void* workspace, size_t workspace_bytes,
                                void* stream) {
  clear_error();
  moe_status s = check_type16(type);
  if (s == MOE_OK) s = check_product(n_groups, rows, K, N, false);
  if (s == MOE_OK) s = check_offsets(offsets, n_groups);
  if (s != MOE_OK) return s;
  REQUIRE_PTR(db);
  const size_t need = rows > 0 ? moe::gemm16_backward_workspace_bytes(rows, n_groups, K, N) : 0;
  if (rows > 0) {
    REQUIRE_PTR(dz);
    REQUIRE_PTR(a);
    s = check_workspace(workspace, workspace_bytes, need, 16);
    if (s != MOE_OK) return s;
  }
  const size_t R = rows, G = n_groups;
  s = check_apart({{{"db", db, 4 * G * N * K}, {}}, {{"workspace", need ? workspace : nullptr, need}, {}}},
                  {{"dz", dz, 2 * R * N}, {"a", a, 2 * R * K}, {"offsets", offsets, offsets_bytes(n_groups)}});
  if (s != MOE_OK) return s;
  return hip_status(moe::launch_gemm16_wgrad(type, dz, a, offsets, n_groups, rows, K, N, db, workspace,
                                             static_cast<hipStream_t>(stream)), "grouped_gemm16_wgrad launch");
}

static moe_status dropout(moe_dtype type, const void* x, const void* residual, int64_t n, float p, const int64_t* rng,
                          void* out, const char* x_name, const char* out_name, const char* what, void* stream) {
  moe_status s = check_type(type);
  if (s != MOE_OK) return s;
  REQUIRE(n >= 0, "n=%lld is negative", (long long)n);
  REQUIRE(p >= 0.0f && p <= 1.0f, "p=%g must be in [0, 1]", (double)p);
  if (n > kMaxElements) return fail(MOE_ERR_UNSUPPORTED, "n=%lld is above 2^40", (long long)n);
  if (n == 0) return MOE_OK;
  REQUIRE(x != nullptr && aligned16(x), "%s is NULL or not 16-byte aligned", x_name);
  REQUIRE_ALIGNED_OR_NULL(residual);
  REQUIRE_PTR_A(rng, 8);
  REQUIRE(out != nullptr && aligned16(out), "%s is NULL or not 16-byte aligned", out_name);
  const size_t bytes = (size_t)n * bytes_of(type);
  s = check_apart({{{out_name, out, bytes}, {x_name, "residual"}}},
                  {{x_name, x, bytes}, {"residual", residual, bytes}, {"rng", rng, 16}});
  if (s != MOE_OK) return s;
  return hip_status(moe::launch_dropout(type, x, residual, n, p, rng, out, static_cast<hipStream_t>(stream)), what);
}

moe_status moe_dropout(moe_dtype type, const void* x, const void* residual, int64_t n, float p, const int64_t* rng,
                       void* out, void* stream) {
  clear_error();
  return dropout(type, x, residual, n, p, rng, out, "x", "out", "moe_dropout launch", stream);
}

moe_status moe_dropout_backward(moe_dtype type, const void* dout, int64_t n, float p, const int64_t* rng, void* dx,
                                void* stream) {
  clear_error();
  return dropout(type, dout, nullptr, n, p, rng, dx, "dout", "dx", "moe_dropout_backward launch", stream);
}

}  // extern "C"
