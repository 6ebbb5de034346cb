// Argument checks and the error state shared by the C ABI's translation units:
// an entry point clears the thread's message, checks on the host, and returns
// a code with the message set where a check fails.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "moe.h"

namespace moe {
extern thread_local char g_err[512];   // api.cpp; read by moe_last_error
}

namespace {

inline moe_status fail(moe_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(moe::g_err, sizeof moe::g_err, fmt, ap);
  va_end(ap);
  return s;
}

inline void clear_error() { moe::g_err[0] = '\0'; }

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }

inline moe_status hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return MOE_OK;
  return fail(MOE_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

#define REQUIRE(cond, ...)                                 \
  do {                                                     \
    if (!(cond)) return fail(MOE_ERR_INVALID_ARG, __VA_ARGS__); \
  } while (0)

// Byte and BF16 matrices are accessed with 16-byte vector loads/stores; FP32
// and int32 arrays element by element.
#define REQUIRE_PTR_A(p, a)                                                   \
  do {                                                                        \
    if ((p) == nullptr) return fail(MOE_ERR_INVALID_ARG, "%s is NULL", #p);   \
    if (!aligned((p), (a)))                                                   \
      return fail(MOE_ERR_INVALID_ARG, "%s is not %d-byte aligned", #p, (int)(a)); \
  } while (0)
#define REQUIRE_PTR(p) REQUIRE_PTR_A(p, 16)
#define REQUIRE_PTR4(p) REQUIRE_PTR_A(p, 4)

#define REQUIRE_ALIGNED4_OR_NULL(p)                                           \
  do {                                                                        \
    if ((p) != nullptr && !aligned((p), 4))                                   \
      return fail(MOE_ERR_INVALID_ARG, "%s is not 4-byte aligned", #p);       \
  } while (0)

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
inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x != 0 && y != 0 && x < y + b.bytes && y < x + a.bytes;
}
// No output shares memory with an input (but for those named in `same`, which
// it may be as a whole; NULL names none) or with another output.  An input that
// is not named is refused at a named one's address, too.
struct Out {
  Span span;
  std::initializer_list<const char*> same;
};
inline moe_status check_apart(std::initializer_list<Out> outs, std::initializer_list<Span> ins) {
  for (const Out* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins) {
      bool allowed = false;
      for (const char* s : o->same)
        allowed = allowed || (s && i.p == o->span.p && i.bytes == o->span.bytes && std::strcmp(s, i.name) == 0);
      REQUIRE(allowed || !overlap(o->span, i), "%s must not share memory with %s", o->span.name, i.name);
    }
    for (const Out* b = outs.begin(); b != o; ++b)
      REQUIRE(!overlap(o->span, b->span), "%s must not share memory with %s", o->span.name, b->span.name);
  }
  return MOE_OK;
}

inline moe_status check_route_params(const moe_route_params& p) {
  REQUIRE(p.n_experts >= 1 && p.n_experts <= 256, "n_experts=%d must be in [1, 256]", p.n_experts);
  REQUIRE(p.n_groups >= 1 && p.n_groups <= 64, "n_groups=%d must be in [1, 64]", p.n_groups);
  REQUIRE(p.n_experts % p.n_groups == 0, "n_experts=%d is not a multiple of n_groups=%d",
          p.n_experts, p.n_groups);
  REQUIRE(p.topk_groups >= 1 && p.topk_groups <= p.n_groups, "topk_groups=%d must be in [1, %d]",
          p.topk_groups, p.n_groups);
  REQUIRE(p.topk >= 1, "topk=%d must be >= 1", p.topk);
  REQUIRE(p.topk % p.topk_groups == 0, "topk=%d is not a multiple of topk_groups=%d", p.topk,
          p.topk_groups);
  const int per = p.n_experts / p.n_groups;
  REQUIRE(p.topk / p.topk_groups <= per, "topk/topk_groups=%d exceeds the %d experts of a group",
          p.topk / p.topk_groups, per);
  REQUIRE(p.topk <= p.topk_groups * per, "topk=%d exceeds the %d experts of the kept groups",
          p.topk, p.topk_groups * per);
  REQUIRE(std::isfinite(p.route_scale), "route_scale is not finite");
  if (p.topk > 16) return fail(MOE_ERR_UNSUPPORTED, "topk=%d > 16 is not implemented", p.topk);
  return MOE_OK;
}

}  // namespace
