// The whole MoE layer for a few tokens (T <= 16): router, quantisation, SwiGLU
// experts, combine and residual, as the layer's separate calls compute them,
// with two differences of precision: the selection ranks FP64 scores, and the
// experts' outputs are combined in FP32 without a BF16 rounding in between.
//
//   s = sigmoid(x . wg) in FP64, z = s + b; group-limited top-k of z (ties to
//   the lower index); gates route_scale s / sum s
//   xq = 1x128 tiles of x;  G, U = blocked FP8 products with W1, W3
//   h  = 1x128 tiles of SiLU(G) U;  out = bf16(sum_j w_j W2 h_j + W2 h_shared + residual)
//
// A step at this size is a read of the active experts' weights (44 MB each at
// d 7168, f 2048; at most T k + 1 of them) and little else, so the kernels
// stream weights and keep everything else off that path:
//   * All T <= 16 tokens are the 16 columns of the MFMA, whatever their
//     experts: an expert's weight rows are multiplied by every token and the
//     columns of tokens that did not choose it are dropped.  No gather, no
//     permutation, no row counts; the activations of the K blocks a wave owns
//     stay in its registers for the whole kernel.
//   * The eight waves of a workgroup split K, so a work item is only 16 weight
//     rows: 8 gate and the 8 matching up rows (fragment rows 0..7 and 8..15),
//     or 16 rows of W2 of every active expert in turn.  With 9 experts there
//     are still several items per CU, and all waves of the chip stream.
//   * The second product walks all active experts for its 16 output columns,
//     so the gated sum over experts is its accumulator and the combine, in
//     registers: expert outputs never reach memory.
#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int FW_T = kFewMaxT;          // tokens: the MFMA's columns
constexpr int FW_THREADS = 512;
constexpr int FW_WAVES = FW_THREADS / 64;
constexpr int FW_MAX_E = 256;
constexpr int FW_MAX_K = 16;
constexpr int FW_RING = 6;              // steps of W2 loads in flight per wave

// Device workspace (byte offsets; every part 256-byte aligned).
struct FewLayout {
  size_t sig, xq, xs, h, hq, hsg, plan, total;
};

struct FewPlan {                        // written by the first product's workgroup 0
  int n_active;                         // experts with a token, then the shared one
  int pad[3];
  int expert[FW_MAX_E + 1];
  float gate[FW_T * (FW_MAX_K + 1)];    // of row t (k + 1) + slot
  uint8_t slot[FW_MAX_E + 1][FW_T];     // slot of token t in active expert a, or 255
};

FewLayout few_layout(int T, int d, int f, int E, int k) {
  FewLayout L;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  const size_t rows = (size_t)T * (k + 1);
  L.sig = take((size_t)T * E * sizeof(double));
  L.xq = take((size_t)T * d);
  L.xs = take((size_t)T * (d / 128) * sizeof(float));
  L.h = take(rows * f * sizeof(float));
  L.hq = take(rows * f);
  L.hsg = take(rows * (f / 128) * sizeof(float));
  L.plan = take(sizeof(FewPlan));
  L.total = at;
  return L;
}

struct FewArgs {
  int T, d, f, E, G, M, k;
  double route_scale;
  const uint16_t* x;
  const uint16_t* wg;
  const float* bias;
  const uint8_t* w13;
  const float* w13_s;
  const uint8_t* w2;
  const float* w2_s;
  const uint16_t* residual;
  int32_t* idx;
  float* w;
  uint16_t* out;
  double* sig;      // [T, E]
  uint8_t* xq;      // [T, d]
  float* xs;        // [T, d/128]
  float* h;         // [T (k+1), f]
  uint8_t* hq;      // [T (k+1), f]
  float* hsg;       // [T (k+1), f/128]: scale times gate
  FewPlan* plan;
};

// Barrier that leaves this wave's loads in flight: waits for its LDS accesses
// only (vmcnt untouched).
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Weight fragment loads: 16 rows of 128 bytes as two whole-line loads (8 rows
// each), then two DPP moves per register give the MFMA's operand layout.  Lane
// (g, j) loads 16 bytes of chunk 2g + (j >= 8) from row j % 8 of each half;
// rotating each 16-lane row by 8 and taking half of its lanes leaves lane
// (g, j) with chunks 2g and 2g + 1 of fragment row j.
typedef int i32x4 __attribute__((ext_vector_type(4)));

struct Lines {
  i32x4 x, y;
};

__device__ __forceinline__ Lines load_weight(const uint8_t* x, const uint8_t* y) {
  return {__builtin_nontemporal_load(reinterpret_cast<const i32x4*>(x)),
          __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(y))};
}

__device__ __forceinline__ v8i weight_frag(const Lines& l) {
  constexpr int ROW_ROR8 = 0x128;
  v8i f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = __builtin_amdgcn_update_dpp(l.x[i], l.y[i], ROW_ROR8, 0xF, 0xC, false);
    f[4 + i] = __builtin_amdgcn_update_dpp(l.y[i], l.x[i], ROW_ROR8, 0xF, 0x3, false);
  }
  return f;
}

__device__ __forceinline__ v8i row_frag(const uint8_t* p) {
  const uint4 lo = *reinterpret_cast<const uint4*>(p);
  const uint4 hi = *reinterpret_cast<const uint4*>(p + 16);
  return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// ---- kernel 1: affinities (one workgroup per expert) and the tiles of x ----
template <bool POW2>
__global__ __launch_bounds__(256) void few_route_kernel(const FewArgs p) {
  __shared__ double red[4][FW_T];
  const int tid = threadIdx.x;
  if ((int)blockIdx.x >= p.E) {
    const int tile = ((int)blockIdx.x - p.E) * 16 + (tid >> 4);
    const int sub = tid & 15;
    if (tile >= p.T * (p.d / 128)) return;
    const uint4 raw = *reinterpret_cast<const uint4*>(p.x + (size_t)tile * 128 + sub * 8);
    const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
    float v[8], amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_to_f32((uint16_t)(u[i] & 0xFFFFu));
      v[2 * i + 1] = bf16_to_f32((uint16_t)(u[i] >> 16));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
    const float s = tile_scale<POW2>(amax);
    uint2 q;
    q.x = f32x4_to_e4m3(v[0] / s, v[1] / s, v[2] / s, v[3] / s);
    q.y = f32x4_to_e4m3(v[4] / s, v[5] / s, v[6] / s, v[7] / s);
    *reinterpret_cast<uint2*>(p.xq + (size_t)tile * 128 + sub * 8) = q;
    if (sub == 0) p.xs[tile] = s;
    return;
  }
  // a BF16 product is exact in FP32 and its sum runs in FP64, so the scores
  // that the selection compares are exact to 10^-15
  const int e = blockIdx.x;
  double acc[FW_T];
#pragma unroll
  for (int t = 0; t < FW_T; ++t) acc[t] = 0.0;
  for (int c = tid; c < p.d / 8; c += 256) {
    const uint4 raw = *reinterpret_cast<const uint4*>(p.wg + (size_t)e * p.d + c * 8);
    const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int t = 0; t < FW_T; ++t) {
      if (t < p.T) {
        const uint4 xr = *reinterpret_cast<const uint4*>(p.x + (size_t)t * p.d + c * 8);
        const uint32_t xu[4] = {xr.x, xr.y, xr.z, xr.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[t] += (double)(__uint_as_float(u[i] << 16) * __uint_as_float(xu[i] << 16));
          acc[t] += (double)(__uint_as_float(u[i] & 0xFFFF0000u) * __uint_as_float(xu[i] & 0xFFFF0000u));
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < FW_T; ++t) {
    if (t < p.T) {
      double v = acc[t];
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
      if ((tid & 63) == 0) red[tid >> 6][t] = v;
    }
  }
  __syncthreads();
  if (tid < p.T) {
    const double l = (red[0][tid] + red[1][tid]) + (red[2][tid] + red[3][tid]);
    p.sig[(size_t)tid * p.E + e] = 1.0 / (1.0 + exp(-l));
  }
}

// ---- selection: a wave per token ----
struct SelectLds {
  double z[FW_WAVES][FW_MAX_E];          // biased scores, later the group's best in order
  double best[FW_WAVES][FW_MAX_E];       // [group][rank]
  double group[FW_WAVES][64];
  double gate[FW_WAVES][FW_MAX_K];
  uint16_t id[FW_WAVES][FW_MAX_E];
  uint32_t mask[FW_WAVES][FW_MAX_E / 32];
  uint32_t active[FW_MAX_E / 32];        // experts any token chose
  int16_t chosen[FW_T][FW_MAX_K];
};

// Token t on this wave.  Ranks are counted, not sorted: an expert's rank in
// its group is the number of its better ones there; the best min(k, group
// size) of each group, in order, are all that the later steps read.  NaN
// scores rank last, so every index stays in range whatever the inputs.
__device__ void few_select_token(const FewArgs& p, SelectLds& S, FewPlan& P, int t, int wave, int lane,
                                 bool write_out) {
  const int per = p.E / p.G, n_top = p.k / p.M, keep = min(p.k, per);
  double* z = S.z[wave];
  const double* sig = p.sig + (size_t)t * p.E;
  for (int e = lane; e < p.E; e += 64) {
    const double v = sig[e] + (p.bias ? (double)p.bias[e] : 0.0);
    z[e] = v == v ? v : -__builtin_huge_val();
  }
  if (lane < FW_MAX_E / 32) S.mask[wave][lane] = 0;
  wave_lds_fence();
  for (int e = lane; e < p.E; e += 64) {
    const int g = e / per;
    const double v = z[e];
    int r = 0;
    for (int o = g * per; o < (g + 1) * per; ++o) r += (z[o] > v || (z[o] == v && o < e)) ? 1 : 0;
    if (r < keep) {
      S.best[wave][g * keep + r] = v;
      S.id[wave][g * keep + r] = (uint16_t)e;
    }
  }
  wave_lds_fence();
  double gs = 0.0;
  if (lane < p.G) {
    for (int r = 0; r < n_top; ++r) gs += S.best[wave][lane * keep + r];
    S.group[wave][lane] = gs;
  }
  wave_lds_fence();
  int gr = 0;
  if (lane < p.G)
    for (int o = 0; o < p.G; ++o) {
      const double og = S.group[wave][o];
      gr += (og > gs || (og == gs && o < lane)) ? 1 : 0;
    }
  const uint64_t kept = __ballot(lane < p.G && gr < p.M);
  for (int c = lane; c < p.G * keep; c += 64) {
    if (!((kept >> (c / keep)) & 1)) continue;
    const double v = S.best[wave][c];
    const int e = S.id[wave][c];
    int r = 0;
    for (int g = 0; g < p.G; ++g) {
      if (!((kept >> g) & 1)) continue;
      for (int o = g * keep; o < (g + 1) * keep; ++o) {
        const double ov = S.best[wave][o];
        r += (ov > v || (ov == v && S.id[wave][o] < e)) ? 1 : 0;
      }
    }
    if (r < p.k) {
      atomicOr(&S.mask[wave][e >> 5], 1u << (e & 31));
      atomicOr(&S.active[e >> 5], 1u << (e & 31));
    }
  }
  wave_lds_fence();
  // ascending ids: lane w < 8 lists word w's experts after the lower words'
  if (lane < FW_MAX_E / 32) {
    int j = 0;
    for (int i = 0; i < lane; ++i) j += __popc(S.mask[wave][i]);
    for (uint32_t m = S.mask[wave][lane]; m; m &= m - 1) {
      const int e = lane * 32 + __ffs(m) - 1;
      S.chosen[t][j] = (int16_t)e;
      S.gate[wave][j] = sig[e];
      ++j;
    }
  }
  wave_lds_fence();
  double total = 0.0;
  for (int j = 0; j < p.k; ++j) total += S.gate[wave][j];
  if (lane <= p.k) {
    const float w = lane < p.k ? (float)(p.route_scale * S.gate[wave][lane] / total) : 1.0f;
    P.gate[t * (p.k + 1) + lane] = w;
    if (write_out && lane < p.k) {
      p.w[(size_t)t * p.k + lane] = w;
      p.idx[(size_t)t * p.k + lane] = S.chosen[t][lane];
    }
  }
  wave_lds_fence();
}

// The plan of the batch in LDS, by the whole workgroup.
__device__ void few_select(const FewArgs& p, SelectLds& S, FewPlan& P, bool write_out) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  if (tid < FW_MAX_E / 32) S.active[tid] = 0;
  for (int i = tid; i < (FW_MAX_E + 1) * FW_T / 4; i += FW_THREADS) reinterpret_cast<uint32_t*>(P.slot)[i] = ~0u;
  __syncthreads();
  for (int t = wave; t < p.T; t += FW_WAVES) few_select_token(p, S, P, t, wave, lane, write_out);
  __syncthreads();
  auto place = [&](int e) {   // position of expert e in the ascending list
    int a = __popc(S.active[e >> 5] & ((1u << (e & 31)) - 1u));
    for (int i = 0; i < (e >> 5); ++i) a += __popc(S.active[i]);
    return a;
  };
  int n = 0;
#pragma unroll
  for (int i = 0; i < FW_MAX_E / 32; ++i) n += __popc(S.active[i]);
  for (int i = tid; i < p.T * p.k; i += FW_THREADS) {
    const int t = i / p.k, j = i - t * p.k, e = S.chosen[t][j], a = place(e);
    P.expert[a] = e;
    P.slot[a][t] = (uint8_t)j;
  }
  if (tid < p.T) P.slot[n][tid] = (uint8_t)p.k;
  if (tid == 0) {
    P.n_active = n + 1;
    P.expert[n] = p.E;
  }
  __syncthreads();
}

// ---- kernel 2: selection, then h = SiLU(G) U in FP32 ----
// Item i: active expert i / (f/8), h columns 8 (i % (f/8)) .. +7.  Wave w owns
// the K blocks w, w + 8, ... (NB of them at most): their activations and
// scales stay in registers, and as each block's weights are consumed the next
// item's are loaded into their place.
template <int NB>
__global__ __launch_bounds__(FW_THREADS, 1) void few_up_kernel(const FewArgs p) {
  __shared__ SelectLds S;
  __shared__ FewPlan P;
  __shared__ __attribute__((aligned(16))) v4f red[2][FW_WAVES][64];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int g16 = lane >> 4, r16 = lane & 15;
  const int KB = p.d / 128, FB = p.f / 128;

  few_select(p, S, P, blockIdx.x == 0);
  if (blockIdx.x == 0)
    for (int i = tid; i < (int)(sizeof(FewPlan) / 4); i += FW_THREADS)
      reinterpret_cast<uint32_t*>(p.plan)[i] = reinterpret_cast<const uint32_t*>(&P)[i];

  v8i xf[NB];
  float xs[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int kb = wave + 8 * j;
    xf[j] = v8i{0, 0, 0, 0, 0, 0, 0, 0};
    xs[j] = 0.0f;
    if (kb < KB && r16 < p.T) {
      xf[j] = row_frag(p.xq + (size_t)r16 * p.d + kb * 128 + g16 * 32);
      xs[j] = p.xs[r16 * KB + kb];
    }
  }
  const int per = p.f / 8, total = P.n_active * per;
  const size_t lane_off = (size_t)(r16 & 7) * p.d + (2 * g16 + (r16 >> 3)) * 16 + wave * 128;
  Lines b[NB];
  float sw[NB];
  auto bases = [&](int item, const uint8_t*& wp, const float*& sp) {
    const int a = item / per, n8 = item - a * per, e = __builtin_amdgcn_readfirstlane(P.expert[a]);
    wp = p.w13 + ((size_t)e * 2 * p.f + n8 * 8) * p.d + lane_off;
    sp = p.w13_s + ((size_t)e * 2 * FB + (g16 < 2 ? 0 : FB) + n8 / 16) * KB + wave;
  };
  const size_t up = (size_t)p.f * p.d;   // from a gate row to its up row
  int item = blockIdx.x;
  if (item < total) {
    const uint8_t* wp;
    const float* sp;
    bases(item, wp, sp);
#pragma unroll
    for (int j = 0; j < NB; ++j)
      if (wave + 8 * j < KB) {
        b[j] = load_weight(wp + j * 1024, wp + up + j * 1024);
        sw[j] = sp[8 * j];
      }
  }
  for (int n = 0; item < total; ++n) {
    const int next = item + gridDim.x;
    const uint8_t* wp = nullptr;
    const float* sp = nullptr;
    if (next < total) bases(next, wp, sp);
    v4f acc = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      if (wave + 8 * j < KB) {
        const v4f q = mfma_fp8_16x16x128(weight_frag(b[j]), xf[j], v4f{0.f, 0.f, 0.f, 0.f});
        const float s = sw[j] * xs[j];
        if (next < total) {
          b[j] = load_weight(wp + j * 1024, wp + up + j * 1024);
          sw[j] = sp[8 * j];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(q[i], s, acc[i]);
      }
    }
    // The waves' partial sums through LDS, in two halves in turn: one barrier
    // per item, since a half is written again only after the next item's
    // barrier, which the wave that reads it reaches afterwards.
    red[n & 1][wave][lane] = acc;
    lds_barrier();
    if (wave == (n & 7)) {
      v4f s = red[n & 1][0][lane];
#pragma unroll
      for (int v = 1; v < FW_WAVES; ++v) s += red[n & 1][v][lane];
      // lanes 0..31 hold G (columns 4 g16 .. +3), lanes 32..63 U
      v4f u;
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = __shfl_xor(s[i], 32);
      const int a = item / per, n8 = item - a * per;
      const int slot = P.slot[a][r16];
      if (g16 < 2 && slot != 255) {
        float4 h;
        h.x = swiglu_f32(s[0], u[0]);
        h.y = swiglu_f32(s[1], u[1]);
        h.z = swiglu_f32(s[2], u[2]);
        h.w = swiglu_f32(s[3], u[3]);
        *reinterpret_cast<float4*>(p.h + (size_t)(r16 * (p.k + 1) + slot) * p.f + n8 * 8 + g16 * 4) = h;
      }
    }
    item = next;
  }
}

// ---- kernel 3: the 1x128 tiles of h (one per 16 lanes) ----
template <bool POW2>
__global__ __launch_bounds__(256) void few_quant_kernel(const FewArgs p) {
  const int FB = p.f / 128;
  const int tile = blockIdx.x * 16 + (threadIdx.x >> 4), sub = threadIdx.x & 15;
  if (tile >= p.T * (p.k + 1) * FB) return;
  const float4 lo = *reinterpret_cast<const float4*>(p.h + (size_t)tile * 128 + sub * 8);
  const float4 hi = *reinterpret_cast<const float4*>(p.h + (size_t)tile * 128 + sub * 8 + 4);
  const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
  const float s = tile_scale<POW2>(amax);
  uint2 q;
  q.x = f32x4_to_e4m3(v[0] / s, v[1] / s, v[2] / s, v[3] / s);
  q.y = f32x4_to_e4m3(v[4] / s, v[5] / s, v[6] / s, v[7] / s);
  *reinterpret_cast<uint2*>(p.hq + (size_t)tile * 128 + sub * 8) = q;
  if (sub == 0) p.hsg[tile] = s * p.plan->gate[tile / FB];
}

// ---- kernel 4: out = sum over active experts of gate W2 h, + residual ----
// Item i: output columns 16 i .. +15.  The steps (active expert, K block) are
// dealt to the waves in turn; each keeps FW_RING steps of loads in flight.
__global__ __launch_bounds__(FW_THREADS, 1) void few_down_kernel(const FewArgs p) {
  __shared__ FewPlan P;
  __shared__ __attribute__((aligned(16))) v4f red[FW_WAVES][64];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int g16 = lane >> 4, r16 = lane & 15;
  const int FB = p.f / 128;
  for (int i = tid; i < (int)(sizeof(FewPlan) / 4); i += FW_THREADS)
    reinterpret_cast<uint32_t*>(&P)[i] = reinterpret_cast<const uint32_t*>(p.plan)[i];
  __syncthreads();
  const int steps = P.n_active * FB;
  const size_t lane_off = (size_t)(r16 & 7) * p.f + (2 * g16 + (r16 >> 3)) * 16;

  for (int item = blockIdx.x; item < p.d / 16; item += gridDim.x) {
    struct Step {
      Lines b;
      v8i hf;
      float s;
      bool live;      // this lane's token chose the expert
    } ring[FW_RING];
    const uint8_t* wbase = p.w2 + (size_t)item * 16 * p.f + lane_off;
    auto load = [&](Step& st, int step) {
      const int a = step / FB, kb = step - a * FB;
      const int e = __builtin_amdgcn_readfirstlane(P.expert[a]);
      const uint8_t* wp = wbase + (size_t)e * p.d * p.f + kb * 128;
      st.b = load_weight(wp, wp + (size_t)8 * p.f);
      const int slot = P.slot[a][r16];
      st.hf = v8i{0, 0, 0, 0, 0, 0, 0, 0};
      st.s = 0.0f;
      st.live = slot != 255;
      if (st.live) {
        const int row = r16 * (p.k + 1) + slot;
        st.hf = row_frag(p.hq + (size_t)row * p.f + kb * 128 + g16 * 32);
        st.s = p.hsg[row * FB + kb] * p.w2_s[((size_t)e * (p.d / 128) + item / 8) * FB + kb];
      }
    };
    v4f acc = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < FW_RING; ++r)
      if (wave + 8 * r < steps) load(ring[r], wave + 8 * r);
    for (int s0 = wave; s0 < steps; s0 += 8 * FW_RING) {
#pragma unroll
      for (int r = 0; r < FW_RING; ++r) {
        const int step = s0 + 8 * r;
        if (step < steps) {
          const v4f q = mfma_fp8_16x16x128(weight_frag(ring[r].b), ring[r].hf, v4f{0.f, 0.f, 0.f, 0.f});
          const float s = ring[r].s;
          const bool live = ring[r].live;   // other tokens take nothing, not even a NaN weight's product with 0
          if (step + 8 * FW_RING < steps) load(ring[r], step + 8 * FW_RING);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = live ? fmaf(q[i], s, acc[i]) : acc[i];
        }
      }
    }
    red[wave][lane] = acc;
    __syncthreads();
    if (wave == 0 && r16 < p.T) {
      v4f s = red[0][lane];
#pragma unroll
      for (int v = 1; v < FW_WAVES; ++v) s += red[v][lane];
      const size_t at = (size_t)r16 * p.d + item * 16 + g16 * 4;
      if (p.residual) {
        const uint2 r = *reinterpret_cast<const uint2*>(p.residual + at);
        s[0] += __uint_as_float(r.x << 16);
        s[1] += __uint_as_float(r.x & 0xFFFF0000u);
        s[2] += __uint_as_float(r.y << 16);
        s[3] += __uint_as_float(r.y & 0xFFFF0000u);
      }
      uint2 o;
      o.x = (uint32_t)f32_to_bf16(s[0]) | ((uint32_t)f32_to_bf16(s[1]) << 16);
      o.y = (uint32_t)f32_to_bf16(s[2]) | ((uint32_t)f32_to_bf16(s[3]) << 16);
      *reinterpret_cast<uint2*>(p.out + at) = o;
    }
    __syncthreads();
  }
}

}  // namespace

size_t layer_few_workspace_bytes(int T, int d, int f, int E, int k) { return few_layout(T, d, f, E, k).total; }

hipError_t launch_layer_few(const uint16_t* x, const uint16_t* wg, const float* bias, int T, int d, int f, int E,
                            int G, int M, int k, float route_scale, const uint8_t* w13, const float* w13_s,
                            const uint8_t* w2, const float* w2_s, const uint16_t* residual, int32_t* idx, float* w,
                            uint16_t* out, void* workspace, bool pow2, hipStream_t stream) {
  const FewLayout L = few_layout(T, d, f, E, k);
  char* ws = static_cast<char*>(workspace);
  FewArgs p{T, d, f, E, G, M, k, (double)route_scale, x, wg, bias, w13, w13_s, w2, w2_s, residual, idx, w, out,
            reinterpret_cast<double*>(ws + L.sig), reinterpret_cast<uint8_t*>(ws + L.xq),
            reinterpret_cast<float*>(ws + L.xs), reinterpret_cast<float*>(ws + L.h),
            reinterpret_cast<uint8_t*>(ws + L.hq), reinterpret_cast<float*>(ws + L.hsg),
            reinterpret_cast<FewPlan*>(ws + L.plan)};
  const int KB = d / 128, FB = f / 128;
  const dim3 g1(E + (T * KB + 15) / 16), g3((T * (k + 1) * FB + 15) / 16);
  if (pow2) hipLaunchKernelGGL(few_route_kernel<true>, g1, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL(few_route_kernel<false>, g1, dim3(256), 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // no more workgroups than items (each active expert has f/8)
  const dim3 g2(std::min(256, std::min(E, T * k) * (f / 8) + f / 8));
  if (KB <= 8) hipLaunchKernelGGL(few_up_kernel<1>, g2, dim3(FW_THREADS), 0, stream, p);
  else if (KB <= 16) hipLaunchKernelGGL(few_up_kernel<2>, g2, dim3(FW_THREADS), 0, stream, p);
  else if (KB <= 32) hipLaunchKernelGGL(few_up_kernel<4>, g2, dim3(FW_THREADS), 0, stream, p);
  else hipLaunchKernelGGL(few_up_kernel<8>, g2, dim3(FW_THREADS), 0, stream, p);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (pow2) hipLaunchKernelGGL(few_quant_kernel<true>, g3, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL(few_quant_kernel<false>, g3, dim3(256), 0, stream, p);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(few_down_kernel, dim3(std::min(256, d / 16)), dim3(FW_THREADS), 0, stream, p);
  return hipGetLastError();
}

}  // namespace moe
