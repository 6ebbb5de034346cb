// Global gradient norm over a list of tensors, and the scaling that clips them.
//
//   N = sqrt(sum over tensors and elements of g^2)   FP64, rounded once to FP32
//   c = 1 if N <= max_norm, else max_norm / N        FP64, rounded once to FP32
//   out = g c                                        FP32 product, rounded to g's type
//
// An FP32 square has 48 bits and so is exact in FP64; the sum runs there too:
// squares neither overflow nor vanish, and 10^10 of them lose nothing that the
// FP32 result would show.  The FP64 units take 32 elements per clock and CU
// (a conversion and a multiply-add each), ten times what memory delivers.
//
// Tensor addresses and sizes travel in the kernel arguments, kGradBatch tensors
// per launch, so a call needs no table in device memory and can be captured.
// The tensors of a launch are cut into chunks of kGradChunk elements dealt to
// the workgroups in turn; a workgroup's partial sum depends only on the sizes
// and addresses' alignment, and the partials are added in a fixed order, so
// equal inputs give equal bits.
//
// Bound by HBM: 5.8 GB of FP32 gradients are squared in 0.85 ms (6.8 TB/s) and
// scaled in 2.1 ms (11.6 GB read and written, 5.5 TB/s; a large copy makes
// 4.8), other lists' passes in between.  The same list over and over is scaled in
// 1.84 to 1.91 ms in place and 1.81 to 1.89 out of place, norm and scaling
// together in 2.75 to 2.82 and 2.71 to 2.79; in place with a factor of 1 the
// scaling takes 0.07 ms, in which its workgroups find that out.  A few megabytes are bound by the three launches and the host's work
// per tensor: 13 MB take 5 + 2 + 5 us on the device.
#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kGradBatch = 64;            // tensors per launch
constexpr int kGradChunk = 8192;          // elements per chunk: 8 loads of 16 bytes a thread (FP32)
constexpr int kGradGroups = 2048;         // most workgroups of a squares launch: its partial sums
constexpr int kScaleGroups = 32768;       // most of a scaling launch (5.8 GB: 4096 take 1.3% longer)
constexpr int kGradThreads = 256;
constexpr int kAhead = 4;                 // 16-byte loads in flight per thread

struct GradList {
  const void* g[kGradBatch];
  void* out[kGradBatch];
  int64_t n[kGradBatch];
  int64_t chunk0[kGradBatch + 1];         // first chunk of each tensor
  uint64_t bf16;                          // bit i: tensor i is BF16
  int count;
};

__device__ __forceinline__ int tensor_of(const GradList& L, int64_t chunk) {
  int a = 0, b = L.count - 1;
  while (a < b) {
    const int mid = (a + b + 1) >> 1;
    if (L.chunk0[mid] <= chunk) a = mid; else b = mid - 1;
  }
  return a;
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename V>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4;   // elements of 16 bytes
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
  static __device__ __forceinline__ void unpack(const u32x4& u, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(u[i]);
  }
  static __device__ __forceinline__ u32x4 scale(const u32x4& u, float c) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(__uint_as_float(u[i]) * c);
    return r;
  }
};
// Round to nearest even, keeping NaN a NaN and infinities (gradients may hold
// either; the caller reads them off the norm).
__device__ __forceinline__ uint16_t grad_bf16(float f) {
  return f != f ? (uint16_t)0x7FC0 : f32_to_bf16(f);
}
template <>
struct Elem<uint16_t> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float get(uint16_t v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ uint16_t put(float v) { return grad_bf16(v); }
  static __device__ __forceinline__ void unpack(const u32x4& u, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ u32x4 scale(const u32x4& u, float c) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = (uint32_t)grad_bf16(__uint_as_float(u[i] << 16) * c) |
             ((uint32_t)grad_bf16(__uint_as_float(u[i] & 0xFFFF0000u) * c) << 16);
    return r;
  }
};

template <bool STREAM>
__device__ __forceinline__ u32x4 load16(const u32x4* p) {
  return STREAM ? __builtin_nontemporal_load(p) : *p;
}
template <bool STREAM>
__device__ __forceinline__ void store16(u32x4* p, const u32x4& v) {
  if (STREAM) __builtin_nontemporal_store(v, p);
  else *p = v;
}

// Elements before the first 16-byte boundary of p (at most n).
template <typename V>
__device__ __forceinline__ int head_of(const V* p, int n) {
  return min((int)(((16u - ((uint32_t)(uintptr_t)p & 15u)) & 15u) / sizeof(V)), n);
}

// Sum of squares of chunk elements [0, n): a scalar head up to a 16-byte
// boundary, 16-byte loads, a scalar tail.
template <bool STREAM, typename V>
__device__ __forceinline__ double chunk_squares(const V* __restrict__ p, int n) {
  constexpr int kVec = Elem<V>::kVec;
  double s = 0.0;
  const int head = head_of(p, n);
  if ((int)threadIdx.x < head) {
    const double v = Elem<V>::get(p[threadIdx.x]);
    s = v * v;
  }
  const int nv = (n - head) / kVec;
  const u32x4* vp = reinterpret_cast<const u32x4*>(p + head);
  for (int i = threadIdx.x; i < nv; i += kAhead * kGradThreads) {
    u32x4 u[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i + k * kGradThreads < nv) u[k] = load16<STREAM>(vp + i + k * kGradThreads);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (i + k * kGradThreads < nv) {
        float v[kVec];
        Elem<V>::unpack(u[k], v);
#pragma unroll
        for (int j = 0; j < kVec; ++j) s = fma((double)v[j], (double)v[j], s);
      }
    }
  }
  for (int i = head + nv * kVec + threadIdx.x; i < n; i += kGradThreads) {
    const double v = Elem<V>::get(p[i]);
    s = fma(v, v, s);
  }
  return s;
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[kGradThreads / 64];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = red[0];
#pragma unroll
  for (int i = 1; i < kGradThreads / 64; ++i) s += red[i];
  return s;
}

template <bool STREAM>
__global__ __launch_bounds__(kGradThreads) void grad_squares_kernel(const GradList L, double* __restrict__ partial) {
  double s = 0.0;
  const int64_t total = L.chunk0[L.count];
  for (int64_t c = blockIdx.x; c < total; c += gridDim.x) {
    const int t = tensor_of(L, c);
    const int64_t e0 = (c - L.chunk0[t]) * kGradChunk;
    const int n = (int)min((int64_t)kGradChunk, L.n[t] - e0);
    if ((L.bf16 >> t) & 1)
      s += chunk_squares<STREAM>(static_cast<const uint16_t*>(L.g[t]) + e0, n);
    else
      s += chunk_squares<STREAM>(static_cast<const float*>(L.g[t]) + e0, n);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ __launch_bounds__(kGradThreads) void grad_norm_kernel(const double* __restrict__ partial, int n,
                                                                 float max_norm, float* __restrict__ norm,
                                                                 float* __restrict__ coef) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kGradThreads) s += partial[i];
  s = block_sum(s);
  if (threadIdx.x == 0) {
    const double r = sqrt(s);
    *norm = (float)r;
    *coef = r <= (double)max_norm ? 1.0f : (float)((double)max_norm / r);
  }
}

// out = g c over a chunk.  The 16-byte form needs g and out equally far from a
// boundary; otherwise element by element.
template <bool STREAM, typename V>
__device__ __forceinline__ void chunk_scale(const V* g, V* out, int n, float c) {
  constexpr int kVec = Elem<V>::kVec;
  const bool together = (((uintptr_t)g ^ (uintptr_t)out) & 15u) == 0;
  const int head = together ? head_of(g, n) : n;
  for (int i = threadIdx.x; i < head; i += kGradThreads) out[i] = Elem<V>::put(Elem<V>::get(g[i]) * c);
  const int nv = (n - head) / kVec;
  const u32x4* gp = reinterpret_cast<const u32x4*>(g + head);
  u32x4* op = reinterpret_cast<u32x4*>(out + head);
  // the loads ahead of their stores (out may be g: a thread writes only what it has read)
  for (int i = threadIdx.x; i < nv; i += kAhead * kGradThreads) {
    u32x4 u[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i + j * kGradThreads < nv) u[j] = load16<STREAM>(gp + i + j * kGradThreads);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i + j * kGradThreads < nv) store16<STREAM>(op + i + j * kGradThreads, Elem<V>::scale(u[j], c));
  }
  for (int i = head + nv * kVec + threadIdx.x; i < n; i += kGradThreads) out[i] = Elem<V>::put(Elem<V>::get(g[i]) * c);
}

template <bool STREAM>
__global__ __launch_bounds__(kGradThreads) void grad_scale_kernel(const GradList L, const float* __restrict__ coef) {
  const float c = *coef;
  const int64_t total = L.chunk0[L.count];
  for (int64_t k = blockIdx.x; k < total; k += gridDim.x) {
    const int t = tensor_of(L, k);
    if (c == 1.0f && L.g[t] == L.out[t]) continue;   // in place and below the limit: nothing changes
    const int64_t e0 = (k - L.chunk0[t]) * kGradChunk;
    const int n = (int)min((int64_t)kGradChunk, L.n[t] - e0);
    if ((L.bf16 >> t) & 1)
      chunk_scale<STREAM>(static_cast<const uint16_t*>(L.g[t]) + e0, static_cast<uint16_t*>(L.out[t]) + e0, n, c);
    else
      chunk_scale<STREAM>(static_cast<const float*>(L.g[t]) + e0, static_cast<float*>(L.out[t]) + e0, n, c);
  }
}

// Fills L with the next non-empty tensors from i on; returns the first index
// not taken.
int fill_list(GradList& L, const void* const* grads, void* const* outs, const int64_t* sizes, const int* types,
              int n_tensors, int i) {
  L.count = 0;
  L.bf16 = 0;
  L.chunk0[0] = 0;
  for (; i < n_tensors && L.count < kGradBatch; ++i) {
    if (sizes[i] == 0) continue;
    const int k = L.count++;
    L.g[k] = grads[i];
    L.out[k] = outs ? outs[i] : nullptr;
    L.n[k] = sizes[i];
    L.chunk0[k + 1] = L.chunk0[k] + (sizes[i] + kGradChunk - 1) / kGradChunk;
    if (types[i] == 1) L.bf16 |= 1ull << k;
  }
  return i;
}

// Bytes of a list.  Lists beyond the last-level cache are read and written past
// the caches (5.8 GB: squares 1.01 -> 0.88 ms, scaling 2.24 -> 2.19); smaller
// ones stay in them from the norm to the scaling (24 MB: scaling 8.1 us, past
// the caches 10.7).
size_t list_bytes(const int64_t* sizes, const int* types, int n_tensors) {
  size_t b = 0;
  for (int i = 0; i < n_tensors; ++i) b += (size_t)sizes[i] * (types[i] == 1 ? 2 : 4);
  return b;
}

}  // namespace

size_t grad_norm_workspace_bytes(int n_tensors) {
  return (size_t)((n_tensors + kGradBatch - 1) / kGradBatch) * kGradGroups * sizeof(double);
}

hipError_t launch_grad_norm(const void* const* grads, const int64_t* sizes, const int* types, int n_tensors,
                            float max_norm, float* norm, float* coef, double* partial, hipStream_t stream) {
  GradList L;
  const bool past_caches = list_bytes(sizes, types, n_tensors) > kCacheBytes;
  int used = 0;
  for (int i = 0; i < n_tensors;) {
    i = fill_list(L, grads, nullptr, sizes, types, n_tensors, i);
    if (L.count == 0) break;
    const int groups = (int)std::min<int64_t>(kGradGroups, L.chunk0[L.count]);
    if (past_caches) hipLaunchKernelGGL(grad_squares_kernel<true>, dim3(groups), dim3(kGradThreads), 0, stream, L, partial + used);
    else hipLaunchKernelGGL(grad_squares_kernel<false>, dim3(groups), dim3(kGradThreads), 0, stream, L, partial + used);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    used += groups;
  }
  hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kGradThreads), 0, stream, partial, used, max_norm, norm, coef);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const void* const* grads, void* const* outs, const int64_t* sizes, const int* types,
                             int n_tensors, const float* coef, hipStream_t stream) {
  GradList L;
  const bool past_caches = list_bytes(sizes, types, n_tensors) > kCacheBytes;
  for (int i = 0; i < n_tensors;) {
    i = fill_list(L, grads, outs, sizes, types, n_tensors, i);
    if (L.count == 0) break;
    const int groups = (int)std::min<int64_t>(kScaleGroups, L.chunk0[L.count]);
    if (past_caches) hipLaunchKernelGGL(grad_scale_kernel<true>, dim3(groups), dim3(kGradThreads), 0, stream, L, coef);
    else hipLaunchKernelGGL(grad_scale_kernel<false>, dim3(groups), dim3(kGradThreads), 0, stream, L, coef);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipGetLastError();
}

}  // namespace moe
