// What the kernels of the 16-bit matrix products share (gemm16.hip,
// gemm16_slim.hip).
#pragma once

#include "activation.h"
#include "groups.h"
#include "kernels.h"
#include "types16.h"

namespace moe {

struct Gemm16Args {
  const uint16_t* p;     // m-side operand
  const uint16_t* q;     // n-side operand
  Groups groups;
  int M, N, K;           // M: wgrad only (the others' m are the groups' rows); K: forward and dgrad only
  const uint16_t* bias;      // [n_groups, N] or NULL
  const uint16_t* residual;  // or NULL
  uint16_t* pre;             // or NULL
  void* out;
  int act;
  int parts;                 // of k, where the result is their FP32 sums in a workspace
};

template <int N>
__device__ __forceinline__ void activate(int act, float (&z)[N]) {
  auto each = [&](auto f) {
#pragma unroll
    for (int e = 0; e < N; ++e) z[e] = f(z[e]);
  };
  if (act == kActRelu) each([](float v) { return act_value<kActRelu>(v); });
  else if (act == kActSilu) each([](float v) { return act_value<kActSilu>(v); });
  else if (act == kActGelu) each([](float v) { return act_value<kActGelu>(v); });
}

// The forward's product by gemm16_slim.hip, and about how many us it takes
// besides its launch (infinity where it cannot).
double gemm16_slim_time(const Gemm16Args& p);
hipError_t launch_gemm16_slim(int type, const Gemm16Args& p, hipStream_t stream);

}  // namespace moe
