// Dropout whose mask is recomputed (include/moe_experts.h): out = residual +
// (keep ? x / q : 0), keep from Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011).  One counter makes 128
// bits, which are the 16-bit values of eight consecutive elements: what a
// thread loads and stores as one 16-byte chunk of a 16-bit type.  A value of
// 16 bits makes the probability a multiple of 2^-16 (the scale is that of the
// probability used) and halves the 32-bit multiplications per element, which
// would otherwise cost as much time as the memory does.
#include <cmath>

#include "kernels.h"
#include "types16.h"

namespace moe {

namespace {

struct Philox {
  uint32_t k0, k1, c2, c3;
  __device__ __forceinline__ explicit Philox(const int64_t* rng) {
    const uint64_t seed = (uint64_t)rng[0], call = (uint64_t)rng[1];
    k0 = (uint32_t)seed;
    k1 = (uint32_t)(seed >> 32);
    c2 = (uint32_t)call;
    c3 = (uint32_t)(call >> 32);
  }
  __device__ __forceinline__ u32x4 operator()(uint64_t i) const {
    uint32_t a = (uint32_t)i, b = (uint32_t)(i >> 32), c = c2, d = c3, x = k0, y = k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      const uint64_t p = (uint64_t)0xD2511F53u * a, q = (uint64_t)0xCD9E8D57u * c;
      a = (uint32_t)(q >> 32) ^ b ^ x;
      b = (uint32_t)q;
      c = (uint32_t)(p >> 32) ^ d ^ y;
      d = (uint32_t)p;
      x += 0x9E3779B9u;
      y += 0xBB67AE85u;
    }
    return u32x4{a, b, c, d};
  }
};

constexpr int kThreads = 256;

// Eight elements a thread.  x, residual and out may be one memory: each element
// is read by the thread that writes it, before it does.  One turn a thread: a
// grid of 4096 workgroups that loop took 137 us for 16384 x 7168 (BF16, 705 MB)
// where this takes 119, 5.9 TB/s.
template <class E, bool RES>
__global__ __launch_bounds__(kThreads) void dropout_kernel(const typename E::storage* x,
                                                           const typename E::storage* residual, int64_t n,
                                                           uint32_t kept, float scale, const int64_t* rng,
                                                           typename E::storage* out) {
  constexpr int V = E::kWidth, C = 8 / V;
  using Val = Values<E, true>;
  const Philox philox(rng);
  const int64_t i = workgroup() * kThreads + threadIdx.x;
  if (i < n / 8) {
    u32x4 xr[C], rr[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      xr[c] = load_chunk(x + i * 8 + c * V);
      if (RES) rr[c] = load_chunk(residual + i * 8 + c * V);
    }
    const u32x4 u = philox((uint64_t)i);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const Val v(xr[c]);
      Val o;
      if (RES) o = Val(rr[c]);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int h = c * V + e;
        const uint32_t word = u[h / 2], value = (h & 1) ? word >> 16 : word & 0xFFFFu;
        o.v[e] = value < kept ? (RES ? fmaf(v.v[e], scale, o.v[e]) : v.v[e] * scale) : o.v[e];
      }
      o.put(out + i * 8 + c * V);
    }
  } else if (i == n / 8) {   // the last, cut off
    const u32x4 u = philox((uint64_t)i);
    for (int h = 0; i * 8 + h < n; ++h) {
      const uint32_t word = h < 2 ? u[0] : h < 4 ? u[1] : h < 6 ? u[2] : u[3];
      const uint32_t value = (h & 1) ? word >> 16 : word & 0xFFFFu;
      const float v = E::load(x[i * 8 + h]), r = RES ? E::load(residual[i * 8 + h]) : 0.0f;
      out[i * 8 + h] = E::store(value < kept ? (RES ? fmaf(v, scale, r) : v * scale) : r);
    }
  }
}

template <class E>
void run(const void* x, const void* residual, int64_t n, uint32_t kept, float scale, const int64_t* rng, void* out,
         hipStream_t stream) {
  using S = typename E::storage;
  const int64_t groups = n / 8 + 1;
  const dim3 grid = grid_of((groups + kThreads - 1) / kThreads);
  if (residual)
    hipLaunchKernelGGL((dropout_kernel<E, true>), grid, dim3(kThreads), 0, stream, static_cast<const S*>(x),
                       static_cast<const S*>(residual), n, kept, scale, rng, static_cast<S*>(out));
  else
    hipLaunchKernelGGL((dropout_kernel<E, false>), grid, dim3(kThreads), 0, stream, static_cast<const S*>(x),
                       static_cast<const S*>(nullptr), n, kept, scale, rng, static_cast<S*>(out));
}

}  // namespace

hipError_t launch_dropout(int type, const void* x, const void* residual, int64_t n, float p, const int64_t* rng,
                          void* out, hipStream_t stream) {
  // q in FP64: 1 - p of a float is exact there
  const uint32_t kept = (uint32_t)std::nearbyint((1.0 - (double)p) * 65536.0);
  const float scale = kept ? (float)(65536.0 / kept) : 0.0f;
  if (type == 0) run<Bf16>(x, residual, n, kept, scale, rng, out, stream);
  else if (type == 1) run<Fp16>(x, residual, n, kept, scale, rng, out, stream);
  else run<Fp32>(x, residual, n, kept, scale, rng, out, stream);
  return hipGetLastError();
}

}  // namespace moe
