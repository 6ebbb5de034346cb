// Gradient of the products' activation and bias (include/moe_experts.h):
// dz = dout act'(pre), dbias[g] = column sums of the group's rows of dz.
//
// One pass over dout and pre.  A workgroup takes a chunk of a group's rows and
// 512 columns; its four waves share the rows, a lane owns eight neighbouring
// columns and keeps their sums in registers.  The chunks' sums go to the
// workspace (beside a pass that writes dz a 64th to a 96th of its bytes with
// chunks of 64 rows, an eighth to a twelfth with eight) and a second kernel adds
// them per group in order: no atomics, the same bits every time.  Bound by HBM:
// 8192 rows of SwiGLU over N 4096 in 32 groups take 43 us, 41 of them the pass
// (168 MB at 4.1 TB/s).
#include <algorithm>

#include "activation.h"
#include "groups.h"
#include "kernels.h"
#include "types16.h"

namespace moe {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64, kCols = 512;
constexpr int U = 4;   // rows in flight a wave

// Rows of a chunk: 64, fewer while the launch would not fill the chip, more
// where its chunks would be 2^32 threads (a launch's dimension takes fewer and
// cuts the others off without an error).
int chunk_rows(int rows, int n_groups, int N) {
  int r = 64;
  while (r > 8 && (long)(rows / r + 1) * ((N + kCols - 1) / kCols) < 1024) r /= 2;
  while (((int64_t)rows / r + n_groups) * kThreads >= int64_t(1) << 32) r *= 2;
  return r;
}

struct ActArgs {
  const uint16_t* dout;
  const uint16_t* pre;
  Groups groups;
  int N, R;
  uint16_t* dz;      // or NULL
  float* partial;    // [chunks][N], or NULL
};

template <class E, int ACT>
__global__ __launch_bounds__(kThreads) void act_backward_kernel(ActArgs p) {
  using Val = Values<E, true>;
  constexpr bool GLU = ACT == kActSwiglu;
  __shared__ int first[kMaxGroups + 1];
  __shared__ float sums[kWaves][GLU ? 2 : 1][kCols];
  list_tiles(p.groups, p.R, first);
  const int chunk = blockIdx.x;
  if (chunk >= first[p.groups.n]) return;
  const int g = tile_group(first, p.groups.n, chunk);
  const int r0 = p.groups.at(g) + (chunk - first[g]) * p.R, r1 = min(r0 + p.R, p.groups.at(g + 1));
  const int width = GLU ? p.N / 2 : p.N;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.y * kCols + lane * 8;
  Val sg, su;
  if (col < width) {
    // U rows' loads before the first is used; rows past the chunk's end repeat its last one and are dropped
    for (int r = r0 + wave; r < r1; r += U * kWaves) {
      u32x4 dr[U], zr[U], ur[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const size_t m = min(r + k * kWaves, r1 - 1);
        dr[k] = load_chunk(p.dout + m * width + col);
        if (ACT != kActNone) zr[k] = load_chunk(p.pre + m * p.N + col);
        if (GLU) ur[k] = load_chunk(p.pre + m * p.N + width + col);
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int m = r + k * kWaves;
        if (m >= r1) break;
        const Val d(dr[k]);
        Val og, ou, z, u;
        if (ACT != kActNone) z = Val(zr[k]);
        if (GLU) u = Val(ur[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if constexpr (GLU) {
            const float e = sigmoid_f32(z.v[i]), v = z.v[i] * e;
            og.v[i] = d.v[i] * u.v[i] * fmaf(v, 1.0f - e, e);
            ou.v[i] = d.v[i] * v;
            su.v[i] += ou.v[i];
          } else if constexpr (ACT == kActRelu) {
            og.v[i] = z.v[i] > 0.0f ? d.v[i] : 0.0f;
          } else {
            og.v[i] = d.v[i] * act_slope<ACT>(z.v[i]);
          }
          sg.v[i] += og.v[i];
        }
        if (p.dz) {
          og.put(p.dz + (size_t)m * p.N + col);
          if (GLU) ou.put(p.dz + (size_t)m * p.N + width + col);
        }
      }
    }
  }
  if (!p.partial) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sums[wave][0][lane * 8 + i] = sg.v[i];
    if (GLU) sums[wave][GLU ? 1 : 0][lane * 8 + i] = su.v[i];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < kCols; c += kThreads) {
    const int at = blockIdx.y * kCols + c;
    if (at >= width) break;
#pragma unroll
    for (int h = 0; h < (GLU ? 2 : 1); ++h) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += sums[w][h][c];
      p.partial[(size_t)chunk * p.N + h * width + at] = v;
    }
  }
}

// dbias[g][c] = sum of the group's chunks, 64 columns a workgroup, its waves
// sharing the chunks.
__global__ __launch_bounds__(kThreads) void act_sums_kernel(Groups groups, int R, int N, const float* __restrict__ partial,
                                                            float* __restrict__ dbias) {
  __shared__ int first[kMaxGroups + 1];
  __shared__ float sums[kWaves][64];
  list_tiles(groups, R, first);
  const int g = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.y * 64 + lane;
  float v = 0.0f;
  if (col < N)
#pragma unroll 4
    for (int c = first[g] + wave; c < first[g + 1]; c += kWaves) v += partial[(size_t)c * N + col];
  sums[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && col < N) {
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += sums[w][lane];
    dbias[(size_t)g * N + col] = v;
  }
}

template <class E>
void run(int act, const ActArgs& p, dim3 grid, hipStream_t stream) {
  switch (act) {
    case kActRelu: hipLaunchKernelGGL((act_backward_kernel<E, kActRelu>), grid, dim3(kThreads), 0, stream, p); break;
    case kActSilu: hipLaunchKernelGGL((act_backward_kernel<E, kActSilu>), grid, dim3(kThreads), 0, stream, p); break;
    case kActGelu: hipLaunchKernelGGL((act_backward_kernel<E, kActGelu>), grid, dim3(kThreads), 0, stream, p); break;
    case kActSwiglu: hipLaunchKernelGGL((act_backward_kernel<E, kActSwiglu>), grid, dim3(kThreads), 0, stream, p); break;
    default: hipLaunchKernelGGL((act_backward_kernel<E, kActNone>), grid, dim3(kThreads), 0, stream, p); break;
  }
}

}  // namespace

size_t act_backward_workspace_bytes(int rows, int n_groups, int N) {
  return rows == 0 ? 0 : ((size_t)rows / chunk_rows(rows, n_groups, N) + n_groups) * N * sizeof(float);
}

hipError_t launch_act_backward(int type, const void* dout, const void* pre, const int32_t* offsets, int n_groups,
                               int rows, int N, int act, void* dz, float* dbias, float* partial, hipStream_t stream) {
  const Groups groups{offsets, n_groups, rows};
  const int R = chunk_rows(rows, n_groups, N);
  if (rows > 0) {
    const int width = act == kActSwiglu ? N / 2 : N;
    const ActArgs p{static_cast<const uint16_t*>(dout), static_cast<const uint16_t*>(pre), groups, N, R,
                    static_cast<uint16_t*>(dz), dbias ? partial : nullptr};
    const dim3 grid(rows / R + n_groups, (width + kCols - 1) / kCols);
    if (type == 0) run<Bf16>(act, p, grid, stream);
    else run<Fp16>(act, p, grid, stream);
  }
  if (dbias)
    hipLaunchKernelGGL(act_sums_kernel, dim3(n_groups, (N + 63) / 64), dim3(kThreads), 0, stream, groups, R, N, partial,
                       dbias);
  return hipGetLastError();
}

}  // namespace moe
