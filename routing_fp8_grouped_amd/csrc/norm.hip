// Residual addition, RMS norm and FP8 quantisation in front of the layer, and
// the norm's backward.
//
// Forward, per row of d elements (all rounding steps in this order):
//   h    = bf16(x + r)                 (h = x without a residual)
//   rstd = fl32(1 / sqrt(sum h^2 / d + eps))   sum, quotient and root in FP64
//   y    = bf16(fl32(fl32(h * rstd) * w))
//   s, q = the 1x128 tiles of y, as fp8_quant_1x128 makes them
// A BF16 square is exact in FP64, and no term goes through more than 38
// additions (16 of its thread, 6 over the lanes, 16 over the waves), so the
// sum's error is below 38 x 2^-53 < 2^-47 relative: rstd, and with it every
// output, does not depend on how a row is split over threads (up to a sum within
// that distance of an FP32 rounding border).
// The FP64 work, one conversion and one multiply-add per element, hides behind
// the memory traffic: 9 bytes per element with a residual.
//
// Backward, with xh = h rstd, g = dy w:
//   c  = sum(g xh) / d
//   dh = bf16(rstd (g - xh c) + dres),  dw = sum over rows of dy xh
// in FP32 products; c and the rows' sums are FP32 trees, dw's partial sums per
// workgroup FP32 and their total FP64.  8 bytes per element with dres.
//
// Both are HBM-bound.  A row belongs to a team of threads, each holding NC
// 16-byte chunks in registers between the sum and the second use, so every
// operand is read once.  At 16384 x 7168 the forward with a residual and all
// outputs moves 1.06 GB in 182 us (5.8 TB/s), the backward with dres 0.94 GB in
// 161 us (5.8 TB/s) and 5 us for dw; a large copy makes 4.8 TB/s, a plain read
// 7.05.  At tens of rows a call waits on the host (7 to 8 us); the kernel alone
// takes 3.7 us for 37 x 384 and 6.1 for 64 x 7168 (0.9 us of bytes, on 64 of
// the 256 CUs), launched from a graph 3.1 and 5.3.
//
// Two chunks per thread for wide rows: one chunk (896 threads for a 7168 row)
// took 214 us, four (256 threads) 224.  The next row's loads ahead of the
// backward's sums gained nothing (other workgroups' loads fill that time).
#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int NORM_THREADS = 256;   // wave teams: four rows per workgroup

// ---- team reductions: a wave, or a whole workgroup through LDS ----

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Sum over the workgroup's waves in wave order; `buf` alternates between two
// halves from call to call, so one barrier per call is enough: a wave writes a
// half again only after the barrier of the call in between, which every wave
// reaches after it has read that half.
template <typename V>
__device__ __forceinline__ V group_sum(V v, V* buf, int waves) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  V s = 0;
  for (int i = 0; i < waves; ++i) s += buf[i];
  return s;
}

// Row data; STREAM: past the caches.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <bool STREAM>
__device__ __forceinline__ uint4 load16(const uint16_t* p) {
  const u32x4* v = reinterpret_cast<const u32x4*>(p);
  const u32x4 u = STREAM ? __builtin_nontemporal_load(v) : *v;
  return make_uint4(u[0], u[1], u[2], u[3]);
}
template <bool STREAM>
__device__ __forceinline__ void store16(uint16_t* p, const uint4& v) {
  const u32x4 u = {v.x, v.y, v.z, v.w};
  if (STREAM) __builtin_nontemporal_store(u, reinterpret_cast<u32x4*>(p));
  else *reinterpret_cast<u32x4*>(p) = u;
}

// Largest of the 16 lanes of a DPP row, by rotations within it.
__device__ __forceinline__ float row_max(float v) {
#define MOE_ROW_MAX(N)                                                                                              \
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + (N), 0xF, 0xF, true)))
  MOE_ROW_MAX(8);
  MOE_ROW_MAX(4);
  MOE_ROW_MAX(2);
  MOE_ROW_MAX(1);
#undef MOE_ROW_MAX
  return v;
}

__device__ __forceinline__ void unpack8(const uint4& raw, float (&v)[8]) {
  const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = (uint32_t)f32_to_bf16(v[2 * i]) | ((uint32_t)f32_to_bf16(v[2 * i + 1]) << 16);
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// Codes of eight elements of a tile with scale s: the correctly rounded
// quotients, as fp8_quant_1x128 divides.  A power-of-two scale divides by its
// exact inverse.  Otherwise Divider, whose quotient is correctly rounded while
// its reciprocal and remainders are normal numbers: with s >= 2^-60 a
// remainder is too small for that only where the quotient lies below 2^-40,
// whose code is a zero either way.  Smaller scales, and the infinite one of a
// tile that holds an infinity, take the plain division.
template <bool POW2>
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float s) {
  float t[8];
  if (POW2) {
    const float r = 1.0f / s;
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = v[i] * r;
  } else if (s >= 0x1p-60f && s <= 0x1p126f) {
    const Divider div(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = div(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = v[i] / s;
  }
  return make_uint2(f32x4_to_e4m3(t[0], t[1], t[2], t[3]), f32x4_to_e4m3(t[4], t[5], t[6], t[7]));
}

// x and res are read and sum is written at the same places by the same thread,
// the loads first, so sum may be x's or res's own memory: none is restrict.
template <int NC, bool WAVE_ROW, bool POW2, bool STREAM>
__global__ __launch_bounds__(WAVE_ROW ? NORM_THREADS : 1024) void rmsnorm_quant_kernel(
    const uint16_t* x, const uint16_t* res, const uint16_t* __restrict__ w, int T, int d, float eps, uint16_t* sum,
    uint16_t* __restrict__ y, uint8_t* __restrict__ q, float* __restrict__ scale, float* __restrict__ rstd) {
  __shared__ double red[2][16];
  const int team = WAVE_ROW ? 64 : blockDim.x;
  const int tl = WAVE_ROW ? (threadIdx.x & 63) : threadIdx.x;
  const int per = WAVE_ROW ? NORM_THREADS / 64 : 1;   // rows per workgroup and step
  const int chunks = d / 8;
  int half = 0;
  for (long row = (long)blockIdx.x * per + (WAVE_ROW ? (threadIdx.x >> 6) : 0); row < T;
       row += (long)gridDim.x * per) {
    const size_t base = (size_t)row * d;
    uint4 h[NC];
    double part = 0.0;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = tl + i * team;
      if (c < chunks) h[i] = load16<STREAM>(x + base + c * 8);
    }
    if (res) {
      uint4 r[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = tl + i * team;
        if (c < chunks) r[i] = load16<STREAM>(res + base + c * 8);
      }
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = tl + i * team;
        if (c < chunks) {
          float a[8], b[8];
          unpack8(h[i], a);
          unpack8(r[i], b);
#pragma unroll
          for (int j = 0; j < 8; ++j) a[j] += b[j];
          h[i] = pack8(a);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = tl + i * team;
      if (c < chunks) {
        if (sum) store16<STREAM>(sum + base + c * 8, h[i]);
        float a[8];
        unpack8(h[i], a);
#pragma unroll
        for (int j = 0; j < 8; ++j) part = fma((double)a[j], (double)a[j], part);
      }
    }
    const double ss = WAVE_ROW ? wave_sum(part) : group_sum(part, red[half], team >> 6);
    half ^= 1;
    const float rs = (float)(1.0 / sqrt(ss / d + (double)eps));
    if (rstd && tl == 0) rstd[row] = rs;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = tl + i * team;
      if (c < chunks) {   // a 128-wide tile's 16 lanes are all in or all out
        float a[8], g[8];
        unpack8(h[i], a);
        unpack8(*reinterpret_cast<const uint4*>(w + c * 8), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = (a[j] * rs) * g[j];
        const uint4 o = pack8(a);
        if (y) store16<STREAM>(y + base + c * 8, o);
        if (q) {
          float v[8], amax = 0.0f;
          unpack8(o, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
          const float s = tile_scale<POW2>(row_max(amax));
          *reinterpret_cast<uint2*>(q + base + c * 8) = codes8<POW2>(v, s);
          if ((c & 15) == 0) scale[(size_t)row * (d / 128) + (c >> 4)] = s;
        }
      }
    }
  }
}

// Rows are dealt to the teams in turn; every thread keeps the dw partial sums
// of its columns over its team's rows.  Workgroup b writes partial[b][0..d).
template <int NC, int THREADS, bool WAVE_ROW, bool STREAM>
__global__ __launch_bounds__(THREADS) void rmsnorm_backward_kernel(
    const uint16_t* __restrict__ dy, const uint16_t* __restrict__ h, const uint16_t* __restrict__ w,
    const float* __restrict__ rstd, const uint16_t* dres, int T, int d, uint16_t* dh, float* __restrict__ partial) {
  __shared__ float red[2][16];
  __shared__ float comb[WAVE_ROW ? NORM_THREADS / 64 : 1][WAVE_ROW ? NC * 512 : 1];
  const int team = WAVE_ROW ? 64 : blockDim.x;
  const int tl = WAVE_ROW ? (threadIdx.x & 63) : threadIdx.x;
  const int per = WAVE_ROW ? NORM_THREADS / 64 : 1;
  const int chunks = d / 8;
  const float inv_d = 1.0f / d;
  float acc[NC][8];
  uint4 wr[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = tl + i * team;
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
    wr[i] = c < chunks ? *reinterpret_cast<const uint4*>(w + c * 8) : make_uint4(0, 0, 0, 0);
  }
  int half = 0;
  for (long row = (long)blockIdx.x * per + (WAVE_ROW ? (threadIdx.x >> 6) : 0); row < T;
       row += (long)gridDim.x * per) {
    const size_t base = (size_t)row * d;
    const float rs = rstd[row];
    uint4 a[NC], b[NC], e[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = tl + i * team;
      a[i] = b[i] = e[i] = make_uint4(0, 0, 0, 0);
      if (c < chunks) {
        a[i] = load16<STREAM>(dy + base + c * 8);
        b[i] = load16<STREAM>(h + base + c * 8);
        if (dres) e[i] = load16<STREAM>(dres + base + c * 8);
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float gy[8], hv[8], wv[8];
      unpack8(a[i], gy);
      unpack8(b[i], hv);
      unpack8(wr[i], wv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float p = gy[j] * (hv[j] * rs);
        acc[i][j] += p;
        dot = fmaf(p, wv[j], dot);
      }
    }
    const float c1 = (WAVE_ROW ? wave_sum(dot) : group_sum(dot, red[half], team >> 6)) * inv_d;
    half ^= 1;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = tl + i * team;
      if (c < chunks) {
        float gy[8], hv[8], wv[8], r[8];
        unpack8(a[i], gy);
        unpack8(b[i], hv);
        unpack8(wr[i], wv);
        unpack8(e[i], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = fmaf(rs, fmaf(-(hv[j] * rs), c1, gy[j] * wv[j]), r[j]);
        store16<STREAM>(dh + base + c * 8, pack8(r));
      }
    }
  }
  float* out = partial + (size_t)blockIdx.x * d;
  if (WAVE_ROW) {
    float* mine = comb[threadIdx.x >> 6];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) mine[(tl + i * 64) * 8 + j] = acc[i][j];
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += NORM_THREADS) {
      float s = comb[0][c];
#pragma unroll
      for (int v = 1; v < NORM_THREADS / 64; ++v) s += comb[v][c];
      out[c] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = tl + i * team;
      if (c < chunks) {
        *reinterpret_cast<float4*>(out + c * 8) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        *reinterpret_cast<float4*>(out + c * 8 + 4) = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
      }
    }
  }
}

// dw[c] = sum over n partial rows, FP64, in a fixed order: 32 threads share a
// column's rows (row r to thread r % 32, eight loads in flight), their sums
// joined in LDS.
__global__ __launch_bounds__(1024) void rmsnorm_dw_kernel(const float* __restrict__ partial, int n, int d,
                                                          float* __restrict__ dw) {
  __shared__ double s[32][33];
  const int x = threadIdx.x & 31, part = threadIdx.x >> 5, col = blockIdx.x * 32 + x;
  double a = 0.0;
  int r = part;
  for (; r + 7 * 32 < n; r += 8 * 32) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = partial[(size_t)(r + 32 * i) * d + col];
#pragma unroll
    for (int i = 0; i < 8; ++i) a += v[i];
  }
  for (; r < n; r += 32) a += partial[(size_t)r * d + col];
  s[part][x] = a;
  __syncthreads();
  if (part == 0) {
#pragma unroll
    for (int i = 1; i < 32; ++i) a += s[i][x];
    dw[col] = (float)a;
  }
}

// Up to these widths a wave owns a row, beyond them a workgroup does (2 chunks
// per thread).  Forward: one chunk per lane; with four, up to 2048, 64 rows of
// that width took 6.8 us against the workgroup's 4.8 and 16384 rows 65 against
// 61.  Backward: up to four chunks per lane, since the waves share their dw
// sums: 16384 rows of 1152 take 35 us against the workgroup's 57, of 2048 55
// against 64 (64 rows: 6.5 against 5.9).
constexpr int kForwardWaveD = 512;
constexpr int kBackwardWaveD = 2048;

// Calls that move more than this go past the caches; below it what they write
// is still there for the kernel that reads it next.  Forward and the router
// and two readers of its outputs after it, 7168 wide, us through the caches and
// past them: 2048 rows (132 MB) 104.5 and 106.8, 4096 rows (264 MB) 149 and
// 146, 16384 rows 420 and 413.  Backward between a writer of dy and a reader of
// dh: 1024 rows (59 MB) 31 and 32, 2048 rows (117 MB) 51.7 and 49.1.
constexpr size_t kForwardCached = size_t(192) << 20;
constexpr size_t kBackwardCached = size_t(96) << 20;

int group_threads(int d) { return ((d / 16) + 63) / 64 * 64; }

}  // namespace

hipError_t launch_rmsnorm_quant(const uint16_t* x, const uint16_t* res, const uint16_t* w, int T, int d, float eps,
                                uint16_t* sum, uint16_t* y, uint8_t* q, float* scale, float* rstd, bool pow2,
                                hipStream_t stream) {
  const bool past_caches = (size_t)T * d * 9 > kForwardCached;
#define MOE_NORM_ONE(NC, WR, THREADS, POW2, STREAM)                                                                 \
  hipLaunchKernelGGL((rmsnorm_quant_kernel<NC, WR, POW2, STREAM>), grid, dim3(THREADS), 0, stream, x, res, w, T, d, \
                     eps, sum, y, q, scale, rstd)
#define MOE_NORM(NC, WR, THREADS, ROWS)                                                                             \
  do {                                                                                                              \
    const dim3 grid((unsigned)std::min((long)(1 << 20), ((long)T + (ROWS)-1) / (ROWS)));                            \
    if (pow2 && past_caches) MOE_NORM_ONE(NC, WR, THREADS, true, true);                                             \
    else if (pow2) MOE_NORM_ONE(NC, WR, THREADS, true, false);                                                      \
    else if (past_caches) MOE_NORM_ONE(NC, WR, THREADS, false, true);                                               \
    else MOE_NORM_ONE(NC, WR, THREADS, false, false);                                                               \
  } while (0)
  if (d <= kForwardWaveD) MOE_NORM(1, true, NORM_THREADS, NORM_THREADS / 64);
  else MOE_NORM(2, false, group_threads(d), 1);
#undef MOE_NORM
#undef MOE_NORM_ONE
  return hipGetLastError();
}

// Workgroups of the backward's first kernel: enough to fill the chip.  Each
// writes a row of dw partial sums that the second kernel reads, 4096 d bytes of
// traffic with 512 of them.  Of rows over 2048 wide that is an eighth of the
// operands' 8 T d at T = 4096 (49 us, 4.8 TB/s of operands at d 7168), half of
// them at 1024 (18 us, 3.2) and as much again up to 512, where every row has its
// own (15 us, 2.0).  At 16384 rows 256 and 1024 workgroups took 189 and 170 us against 164;
// fewer ones for fewer rows have not been measured.
int rmsnorm_backward_groups(int T, int d) {
  const int rows = d <= kBackwardWaveD ? NORM_THREADS / 64 : 1;
  return (int)std::min((long)512, ((long)T + rows - 1) / rows);
}

hipError_t launch_rmsnorm_backward(const uint16_t* dy, const uint16_t* h, const uint16_t* w, const float* rstd,
                                   const uint16_t* dres, int T, int d, uint16_t* dh, float* dw, float* partial,
                                   hipStream_t stream) {
  const int n = T > 0 ? rmsnorm_backward_groups(T, d) : 0;   // no rows: dw = 0 alone
  const bool stream_rows = (size_t)T * d * 8 > kBackwardCached;
#define MOE_NORM_BWD(NC, MAX, WR, THREADS)                                                                           \
  do {                                                                                                               \
    if (stream_rows)                                                                                                 \
      hipLaunchKernelGGL((rmsnorm_backward_kernel<NC, MAX, WR, true>), dim3(n), dim3(THREADS), 0, stream, dy, h, w, rstd, \
                         dres, T, d, dh, partial);                                                                   \
    else                                                                                                             \
      hipLaunchKernelGGL((rmsnorm_backward_kernel<NC, MAX, WR, false>), dim3(n), dim3(THREADS), 0, stream, dy, h, w,      \
                         rstd, dres, T, d, dh, partial);                                                             \
  } while (0)
  if (n > 0) {
    if (d <= 512) MOE_NORM_BWD(1, NORM_THREADS, true, NORM_THREADS);
    else if (d <= kBackwardWaveD) MOE_NORM_BWD(4, NORM_THREADS, true, NORM_THREADS);
    else if (d <= 8192) MOE_NORM_BWD(2, 512, false, group_threads(d));
    else MOE_NORM_BWD(2, 1024, false, group_threads(d));
  }
#undef MOE_NORM_BWD
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(rmsnorm_dw_kernel, dim3(d / 32), dim3(1024), 0, stream, partial, n, d, dw);
  return hipGetLastError();
}

}  // namespace moe
