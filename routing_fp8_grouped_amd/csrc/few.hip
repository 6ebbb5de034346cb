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
#include <type_traits>

#include "common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int FW_T = kFewMaxT;          // tokens: the MFMA's columns
constexpr int FW_THREADS = 512;
constexpr int FW_WAVES = FW_THREADS / 64;
constexpr int FW_MAX_E = 256;
constexpr int FW_MAX_K = 16;
constexpr int FR_THREADS = 512;         // router
constexpr int FR_WAVES = FR_THREADS / 64;
constexpr int FR_RING = 4;              // 32-element chunks in flight per wave
constexpr int FR_MAX_SPLITS = 8;

// Device workspace (byte offsets; every part 256-byte aligned).
struct FewLayout {
  size_t part, xq, xs, h, hq, hsg, plan, total;
};

struct FewPlan {                        // written by the first product's workgroup 0
  int n_active;                         // the shared expert, then those with a token, ascending
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
  L.part = take((size_t)FR_MAX_SPLITS * T * E * sizeof(double));
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
  int splits;       // parts of d in the logits' partial sums: 8, 4 or 2
  int e_log2;       // experts and candidates of a token, rounded up to powers of two
  int c_log2;
  double* part;     // [splits, T, E] partial logits
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

// ---- kernel 1: partial logits and the tiles of x ----
// A workgroup takes 16 experts and one of `splits` parts of d, so that the
// 3.7 MB of V3's router come through 128 CUs; the next kernel adds the parts.
// A BF16 MFMA multiplies 16 experts by 16 tokens over 32 elements, and those
// partial sums, good to 2^-24 of their largest product, add up in FP64: a
// logit is exact to 10^-8, ranked as FP64.  (The FP64 MFMA is exact but takes
// 64 clocks for 4 elements.)
typedef double v4d __attribute__((ext_vector_type(4)));

union Bf16x8 {
  uint4 u;
  v8bf v;
};

template <bool POW2>
__global__ __launch_bounds__(FR_THREADS) void few_route_kernel(const FewArgs p) {
  __shared__ v4d red[FR_WAVES][64];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int router = (p.E + 15) / 16 * p.splits;
  if ((int)blockIdx.x >= router) {
    const int tile = ((int)blockIdx.x - router) * (FR_THREADS / 16) + (tid >> 4);
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
  const int e0 = (int)blockIdx.x / p.splits * 16, split = (int)blockIdx.x % p.splits;
  const int r16 = lane & 15, g16 = lane >> 4;
  // rows past the last expert or token repeat it; their results are not stored
  const uint16_t* wr = p.wg + (size_t)min(e0 + r16, p.E - 1) * p.d + g16 * 8;
  const uint16_t* xr = p.x + (size_t)min(r16, p.T - 1) * p.d + g16 * 8;
  const int chunks = p.d / 32;
  v4d acc = v4d{0.0, 0.0, 0.0, 0.0};
  const int stride = FR_WAVES * p.splits;   // the parts interleave
  for (int c0 = split * FR_WAVES + wave; c0 < chunks; c0 += stride * FR_RING) {
    Bf16x8 a[FR_RING], b[FR_RING];
#pragma unroll
    for (int r = 0; r < FR_RING; ++r) {
      const int c = min(c0 + r * stride, chunks - 1);
      a[r].u = *reinterpret_cast<const uint4*>(wr + c * 32);
      b[r].u = *reinterpret_cast<const uint4*>(xr + c * 32);
    }
#pragma unroll
    for (int r = 0; r < FR_RING; ++r) {
      const v4f q = mfma_bf16_16x16x32(a[r].v, b[r].v, v4f{0.f, 0.f, 0.f, 0.f});
      if (c0 + r * stride < chunks) {   // uniform over the wave
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += (double)q[i];
      }
    }
  }
  red[wave][lane] = acc;
  __syncthreads();
  // lane l holds rows (experts) 4 (l / 16) + i, column (token) l % 16
  if (tid < 256) {
    const int i = tid >> 6, e = e0 + 4 * g16 + i;
    double l = red[0][lane][i];
#pragma unroll
    for (int v = 1; v < FR_WAVES; ++v) l += red[v][lane][i];
    if (r16 < p.T && e < p.E) p.part[((size_t)split * p.T + r16) * p.E + e] = l;
  }
}

// ---- selection, by a whole workgroup, (token, expert) pairs over its threads ----
struct SelectLds {
  uint64_t key[FW_T][FW_MAX_E];          // score order, then lower index: larger is better
  uint64_t best[FW_T][FW_MAX_E];         // [group][rank]: keys of each group's best, in order
  double z[FW_T][FW_MAX_E];              // biased scores
  double sig[FW_T][FW_MAX_E];            // affinities
  double group[FW_T][64];
  double gate[FW_T][FW_MAX_K];
  uint64_t kept[FW_T];                   // groups kept
  uint32_t mask[FW_T][FW_MAX_E / 32];    // experts chosen
  uint32_t active[FW_MAX_E / 32];        // experts any token chose
  int16_t chosen[FW_T][FW_MAX_K];        // ascending
};

// The partial logits of this thread's (token, expert) pairs: pair tid + 512 i
// of the tokens' rows of 2^e_log2.  `splits` parts of 16 / splits pairs each
// way are 16 loads, issued before the first weights (behind which they would
// queue for 4 us) and added up after.
struct PartialLogits {
  double v[16];

  template <int SPLITS>
  __device__ __forceinline__ void load_as(const FewArgs& p) {
#pragma unroll
    for (int i = 0; i < 16 / SPLITS; ++i) {
      const int at = threadIdx.x + FW_THREADS * i, t = min(at >> p.e_log2, p.T - 1);
      const int e = min(at & ((1 << p.e_log2) - 1), p.E - 1);
#pragma unroll
      for (int s = 0; s < SPLITS; ++s) v[i * SPLITS + s] = p.part[((size_t)s * p.T + t) * p.E + e];
    }
  }
  __device__ __forceinline__ void load(const FewArgs& p) {
    if (p.splits == 8) load_as<8>(p);
    else if (p.splits == 4) load_as<4>(p);
    else load_as<2>(p);
  }
  // l[i]: the logit of pair i (i < 16 / splits)
  template <int SPLITS>
  __device__ __forceinline__ void sum_as(double (&l)[8]) const {
#pragma unroll
    for (int i = 0; i < 16 / SPLITS; ++i) {
      l[i] = v[i * SPLITS];
#pragma unroll
      for (int s = 1; s < SPLITS; ++s) l[i] += v[i * SPLITS + s];
    }
  }
  __device__ __forceinline__ void sum(int splits, double (&l)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) l[i] = 0.0;
    if (splits == 8) sum_as<8>(l);
    else if (splits == 4) sum_as<4>(l);
    else sum_as<2>(l);
  }
};

// Doubles in an unsigned order, the low byte giving way to 255 - e: keys are
// distinct, equal scores rank by the lower index, and a score moves by at most
// 2^-44 of itself, far below the logits' own error.  NaN scores rank last, so
// every index below stays in range whatever the inputs.
__device__ __forceinline__ uint64_t score_key(double z, int e) {
  if (!(z == z)) z = -__builtin_huge_val();
  uint64_t u = (uint64_t)__double_as_longlong(z + 0.0);   // -0 as +0
  u = (u >> 63) ? ~u : u | 0x8000000000000000ull;
  return (u & ~255ull) | (uint32_t)(255 - e);
}
__device__ __forceinline__ int key_expert(uint64_t k) { return 255 - (int)(k & 255); }

// Entries of list[0..n) above k.
__device__ __forceinline__ int count_above(const uint64_t* list, int n, uint64_t k) {
  int r = 0;
#pragma unroll 8
  for (int i = 0; i < n; ++i) r += list[i] > k ? 1 : 0;
  return r;
}

// The batch's plan in LDS.  Ranks are counted, not sorted: an expert's rank in
// its group is the number of better ones there; the best min(k, group size) of
// each group, in order, are all that the later steps read.
__device__ void few_select(const FewArgs& p, SelectLds& S, FewPlan& P, const PartialLogits& part, bool write_out) {
  const int tid = threadIdx.x;
  const int per = p.E / p.G, n_top = p.k / p.M, keep = min(p.k, per), cand = p.G * keep;
  // i / per and i / keep for i < 256 by 16-bit reciprocals (exact: the error 255 / 65536 is below 1 / 256)
  const uint32_t inv_per = (65536 + per - 1) / per, inv_keep = (65536 + keep - 1) / keep;
  const int e_mask = (1 << p.e_log2) - 1, c_mask = (1 << p.c_log2) - 1;
  const int pairs = p.T << p.e_log2, cands = p.T << p.c_log2;
  {
    double l[8];
    part.sum(p.splits, l);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = tid + FW_THREADS * i, t = at >> p.e_log2, e = at & e_mask;
      if (at >= pairs) break;
      if (e < p.E) {
        const double s = 1.0 / (1.0 + exp(-l[i])), z = s + (p.bias ? (double)p.bias[e] : 0.0);
        S.sig[t][e] = s;
        S.z[t][e] = z;
        S.key[t][e] = score_key(z, e);
      }
    }
  }
  if (tid < FW_MAX_E / 32) S.active[tid] = 0;
  if (tid < FW_T) S.kept[tid] = 0;
  if (tid < FW_T * FW_MAX_E / 32) S.mask[0][tid] = 0;
  for (int i = tid; i < (FW_MAX_E + 1) * FW_T / 4; i += FW_THREADS) reinterpret_cast<uint32_t*>(P.slot)[i] = ~0u;
  lds_barrier();
  for (int at = tid; at < pairs; at += FW_THREADS) {
    const int t = at >> p.e_log2, e = at & e_mask, g = (int)(e * inv_per >> 16);
    if (e >= p.E) continue;
    const uint64_t k = S.key[t][e];
    const int r = count_above(&S.key[t][g * per], per, k);
    if (r < keep) S.best[t][g * keep + r] = k;
  }
  lds_barrier();
  for (int at = tid; at < p.T * 64; at += FW_THREADS) {
    const int t = at >> 6, g = at & 63;
    if (g >= p.G) continue;
    double s = 0.0;
    for (int r = 0; r < n_top; ++r) s += S.z[t][key_expert(S.best[t][g * keep + r])];
    S.group[t][g] = s;
  }
  lds_barrier();
  for (int at = tid; at < p.T * 64; at += FW_THREADS) {
    const int t = at >> 6, g = at & 63;
    if (g >= p.G) continue;
    const double s = S.group[t][g];
    int r = 0;
#pragma unroll 8
    for (int o = 0; o < p.G; ++o) {
      const double os = S.group[t][o];
      // a NaN sum ranks last, among its like by index
      r += (os > s || (s != s && os == os) || ((os == s || (s != s && os != os)) && o < g)) ? 1 : 0;
    }
    if (r < p.M) atomicOr(reinterpret_cast<unsigned long long*>(&S.kept[t]), 1ull << g);
  }
  lds_barrier();
  for (int at = tid; at < cands; at += FW_THREADS) {
    const int t = at >> p.c_log2, c = at & c_mask, g = (int)(c * inv_keep >> 16);
    const uint64_t kept = S.kept[t];
    if (c >= cand || !((kept >> g) & 1)) continue;
    const uint64_t k = S.best[t][c];
    int r = c - g * keep;
    for (uint64_t m = kept & ~(1ull << g); m; m &= m - 1)
      r += count_above(&S.best[t][(__ffsll((unsigned long long)m) - 1) * keep], keep, k);
    if (r < p.k) {
      const int e = key_expert(k);
      atomicOr(&S.mask[t][e >> 5], 1u << (e & 31));
      atomicOr(&S.active[e >> 5], 1u << (e & 31));
    }
  }
  lds_barrier();
  // position of expert e among a bit mask's, ascending
  auto place = [](const uint32_t* mask, int e) {
    int a = __popc(mask[e >> 5] & ((1u << (e & 31)) - 1u));
#pragma unroll
    for (int i = 0; i < FW_MAX_E / 32; ++i) a += i < (e >> 5) ? __popc(mask[i]) : 0;
    return a;
  };
  // a chosen expert is one of its group's best, so the candidates hold them all
  for (int at = tid; at < cands; at += FW_THREADS) {
    const int t = at >> p.c_log2, c = at & c_mask, g = (int)(c * inv_keep >> 16);
    if (c >= cand || !((S.kept[t] >> g) & 1)) continue;
    const int e = key_expert(S.best[t][c]);
    if (!((S.mask[t][e >> 5] >> (e & 31)) & 1)) continue;
    const int j = place(S.mask[t], e), a = 1 + place(S.active, e);
    S.chosen[t][j] = (int16_t)e;
    S.gate[t][j] = S.sig[t][e];
    P.expert[a] = e;
    P.slot[a][t] = (uint8_t)j;
  }
  if (tid < p.T) P.slot[0][tid] = (uint8_t)p.k;
  if (tid == FW_THREADS - 1) {
    int n = 1;
#pragma unroll
    for (int i = 0; i < FW_MAX_E / 32; ++i) n += __popc(S.active[i]);
    P.n_active = n;
    P.expert[0] = p.E;
  }
  lds_barrier();
  // only workgroup 0's gates are read: by the later kernels, and by the caller
  if (write_out) {
    for (int at = tid; at < p.T * 32; at += FW_THREADS) {
      const int t = at >> 5, j = at & 31;
      if (j > p.k) continue;
      float w = 1.0f;
      if (j < p.k) {
        double total = 0.0;
        for (int o = 0; o < p.k; ++o) total += S.gate[t][o];
        w = (float)(p.route_scale * S.gate[t][j] / total);
        p.w[t * p.k + j] = w;
        p.idx[t * p.k + j] = S.chosen[t][j];
      }
      P.gate[t * (p.k + 1) + j] = w;
    }
    lds_barrier();
  }
}

// ---- kernel 2: selection, then h = SiLU(G) U in FP32 ----
// Item i: active expert i / (f/8), h columns 8 (i % (f/8)) .. +7.  Wave w owns
// the K blocks w, w + 8, ... (NB = ceil(d/1024) of them): their activations
// and scales stay in registers, and as each block's weights are consumed the
// next item's are loaded into their place.  Nothing in that loop branches
// around a load: the compiler counts outstanding loads along straight-line
// code only, and a load that may or may not have been issued makes it wait for
// all of them (measured: 3.8 TB/s with such branches).  So a wave's missing
// last block repeats a present one with a scale of 0, and the last item has
// code of its own.
//
// The products run as BF16 MFMAs on weights widened in registers (E4M3 values
// are exact in BF16): the FP8 MFMA's sums of 128 products carry an error of
// 2.0e-6 RMS of sum|a b|, which moves one h in some hundreds across a rounding
// midpoint of E4M3; the BF16 MFMA's carry 1.3e-9 (both measured over 131072
// sums).  The conversions hide behind the weight stream.
__device__ __forceinline__ v8bf widen8(int lo, int hi) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <int NB>
__global__ __launch_bounds__(FW_THREADS, 1) void few_up_kernel(const FewArgs p) {
  __shared__ __attribute__((aligned(16))) SelectLds S;
  __shared__ FewPlan P;
  // the waves' sums, where the selection's keys were (16 of their 32 KB)
  v4f (*const red)[FW_WAVES][64] = reinterpret_cast<v4f(*)[FW_WAVES][64]>(&S.key);
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int g16 = lane >> 4, r16 = lane & 15;
  const int KB = p.d / 128, FB = p.f / 128;

  const int per = p.f / 8;
  PartialLogits part;
  part.load(p);
  // activations of this wave's blocks; tokens past T repeat the last
  v8i xq[NB];
  float xs[NB];
  int kb[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const bool mine = wave + 8 * j < KB;
    kb[j] = mine ? wave + 8 * j : KB - 1;
    const int t = min(r16, p.T - 1);
    xq[j] = row_frag(p.xq + (size_t)t * p.d + kb[j] * 128 + g16 * 32);
    xs[j] = p.xs[t * KB + kb[j]];
    if (!mine) xs[j] = 0.0f;
  }
  const size_t up = (size_t)p.f * p.d;   // from a gate row to its up row
  const uint8_t* lane_w = p.w13 + (size_t)(r16 & 7) * p.d + (2 * g16 + (r16 >> 3)) * 16;
  const float* lane_s = p.w13_s + (size_t)(g16 < 2 ? 0 : FB) * KB;
  Lines b[NB];
  float sw[NB];
  auto bases = [&](int e, int n8, const uint8_t*& wp, const float*& sp) {
    wp = lane_w + ((size_t)e * 2 * p.f + n8 * 8) * p.d;
    sp = lane_s + ((size_t)e * 2 * FB + n8 / 16) * KB;
  };
  auto load = [&](int j, const uint8_t* wp, const float* sp) {
    b[j] = load_weight(wp + kb[j] * 128, wp + up + kb[j] * 128);
    sw[j] = sp[kb[j]];
  };
  // the first `per` items are the shared expert's, known before the selection:
  // their loads run beneath it
  int item = blockIdx.x, n = 0;
  const uint8_t* wp;
  const float* sp;
  if (item < per) {
    bases(p.E, item, wp, sp);
#pragma unroll
    for (int j = 0; j < NB; ++j) load(j, wp, sp);
  }
  v8bf xb[NB][4];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) xb[j][q] = widen8(xq[j][2 * q], xq[j][2 * q + 1]);
  few_select(p, S, P, part, blockIdx.x == 0);
  if (blockIdx.x == 0)
    for (int i = tid; i < (int)(sizeof(FewPlan) / 4); i += FW_THREADS)
      reinterpret_cast<uint32_t*>(p.plan)[i] = reinterpret_cast<const uint32_t*>(&P)[i];
  const int total = __builtin_amdgcn_readfirstlane(P.n_active) * per;
  if (item >= total) return;
  if (item >= per) {
    const int a = item / per;
    bases(__builtin_amdgcn_readfirstlane(P.expert[a]), item - a * per, wp, sp);
#pragma unroll
    for (int j = 0; j < NB; ++j) load(j, wp, sp);
  }
  auto run = [&](auto more) {           // one item; `more`: another follows
    const int next = item + gridDim.x;
    if (more) {
      const int a = next / per;
      bases(__builtin_amdgcn_readfirstlane(P.expert[a]), next - a * per, wp, sp);
    }
    v4f acc = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const v8i w = weight_frag(b[j]);
      const float s = sw[j] * xs[j];
      if (more) load(j, wp, sp);
      v4f q = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) q = mfma_bf16_16x16x32(widen8(w[2 * i], w[2 * i + 1]), xb[j][i], q);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(q[i], s, acc[i]);
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
    ++n;
  };
  while (item + (int)gridDim.x < total) run(std::true_type{});
  run(std::false_type{});
}

// ---- a 1x128 tile of h: 16 lanes, 8 elements each ----
struct HTile {
  float v[8];

  __device__ __forceinline__ void load(const float* h) {
    const float4 lo = *reinterpret_cast<const float4*>(h);
    const float4 hi = *reinterpret_cast<const float4*>(h + 4);
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
    v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
  }
  // Codes into q; returns the scale.  The quotients are correctly rounded, as
  // fp8_quant_1x128's (by Divider, whose reciprocal and remainders are normal
  // numbers for s >= 2^-60; smaller scales take the plain division).
  template <bool POW2>
  __device__ __forceinline__ float quantise(uint2& q) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
    const float s = tile_scale<POW2>(amax);
    if (s >= 0x1p-60f) {
      const Divider div(s);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = div(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] / s;
    }
    q.x = f32x4_to_e4m3(v[0], v[1], v[2], v[3]);
    q.y = f32x4_to_e4m3(v[4], v[5], v[6], v[7]);
    return s;
  }
};

// ---- kernel 3, for batches whose h few_down_kernel does not stage ----
template <bool POW2>
__global__ __launch_bounds__(256) void few_quant_kernel(const FewArgs p) {
  const int FB = p.f / 128;
  const int tile = blockIdx.x * 16 + (threadIdx.x >> 4), sub = threadIdx.x & 15;
  if (tile >= p.T * (p.k + 1) * FB) return;
  HTile h;
  h.load(p.h + (size_t)tile * 128 + sub * 8);
  uint2 q;
  const float s = h.template quantise<POW2>(q);
  *reinterpret_cast<uint2*>(p.hq + (size_t)tile * 128 + sub * 8) = q;
  if (sub == 0) p.hsg[tile] = s * p.plan->gate[tile / FB];
}

// ---- kernel 4: out = sum over active experts of gate W2 h, + residual ----
// Workgroup b owns an even share of the output columns, in units of 4, and
// takes them 16 at a time (the last time what is left, its missing fragment
// rows repeating the last).  A pass's steps (active expert, U adjacent K
// blocks) are dealt to the waves in turn, `per` to each (steps past the last
// repeat it and add nothing).  The passes follow each other as one stream of
// steps with RING of them in flight per wave; loads are free of branches
// except in the stream's last steps, for the reason above.
//
// STAGE: the workgroup quantises h itself, into LDS, beneath its first weight
// loads; otherwise the tiles come from few_quant_kernel through memory.
constexpr int FW_STAGE_BYTES = 96 * 1024;

template <int U, bool STAGE>
struct DownStep {
  Lines b[U];
  float sw[U];
  v8i hf[STAGE ? 1 : U];
  float sh[STAGE ? 1 : U];
  int hrow;       // row of h for this lane's token
  int kb;
  bool live;      // this lane's token chose the expert, and the step is no repeat
};

template <int U, int RING, bool STAGE, bool POW2>
__global__ __launch_bounds__(FW_THREADS, 1) void few_down_kernel(const FewArgs p) {
  __shared__ FewPlan P;
  __shared__ __attribute__((aligned(16))) v4f red[2][FW_WAVES][64];
  __shared__ __attribute__((aligned(16))) uint8_t stage[STAGE ? FW_STAGE_BYTES : 16];
  constexpr int EARLY = 5;              // tiles of h a thread loads before the weights (9 rows of f 2048)
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int g16 = lane >> 4, r16 = lane & 15;
  const int FB = p.f / 128, FU = FB / U;
  const int tiles = p.T * (p.k + 1) * FB;
  for (int i = tid; i < (int)(sizeof(FewPlan) / 4); i += FW_THREADS)
    reinterpret_cast<uint32_t*>(&P)[i] = reinterpret_cast<const uint32_t*>(p.plan)[i];
  HTile early[STAGE ? EARLY : 1];
  if (STAGE) {
#pragma unroll
    for (int i = 0; i < EARLY; ++i)
      early[i].load(p.h + (size_t)min((tid >> 4) + i * (FW_THREADS / 16), tiles - 1) * 128 + (tid & 15) * 8);
  }
  lds_barrier();
  const int steps = __builtin_amdgcn_readfirstlane(P.n_active) * FU, per = (steps + 7) / 8;
  const int units = p.d / 4;
  const int c_begin = 4 * (int)((long)units * blockIdx.x / gridDim.x);
  const int c_end = 4 * (int)((long)units * (blockIdx.x + 1) / gridDim.x);
  const int count = (c_end - c_begin + 15) / 16 * per;   // steps of this wave's stream
  // a step's expert: step / FU by a rounded-up reciprocal, exact for step * FU < 2^32
  const uint32_t inv = (uint32_t)((0x100000000ull + FU - 1) / FU);
  const uint8_t* lane_w = p.w2 + (2 * g16 + (r16 >> 3)) * 16;
  const int hstride = p.f + 16;         // staged rows, 16 bytes apart in the banks
  float* const stage_s = reinterpret_cast<float*>(stage + p.T * (p.k + 1) * hstride);

  DownStep<U, STAGE> ring[RING];
  int lc = c_begin, lk = 0;             // the next load's first column and step within the pass
  auto load = [&](DownStep<U, STAGE>& st) {
    const int raw = wave + 8 * lk, step = min(raw, steps - 1);
    const int a = FU == 1 ? step : (int)__umulhi((uint32_t)step, inv), kb = (step - a * FU) * U;
    const int e = __builtin_amdgcn_readfirstlane(P.expert[a]);
    const int r0 = min(lc + (r16 & 7), c_end - 1), r1 = min(lc + 8 + (r16 & 7), c_end - 1);
    const uint8_t* wp = lane_w + (size_t)e * p.d * p.f + kb * 128;
    const float* sp = p.w2_s + ((size_t)e * (p.d / 128) + min(lc + 4 * g16, c_end - 1) / 128) * FB + kb;
    const uint8_t* w0 = wp + (size_t)r0 * p.f;
    const uint8_t* w1 = wp + (size_t)r1 * p.f;
#pragma unroll
    for (int q = 0; q < U; ++q) {
      st.b[q] = load_weight(w0 + q * 128, w1 + q * 128);
      st.sw[q] = sp[q];
    }
    const int slot = P.slot[a][r16];
    st.live = slot != 255 && raw < steps;
    // lanes without a token of this expert all read one row, so that they add one line to the load
    st.hrow = slot != 255 ? r16 * (p.k + 1) + slot : p.k;
    st.kb = kb;
    if (!STAGE) {
#pragma unroll
      for (int q = 0; q < U; ++q) {
        st.hf[q] = row_frag(p.hq + (size_t)st.hrow * p.f + (kb + q) * 128 + g16 * 32);
        st.sh[q] = p.hsg[st.hrow * FB + kb + q];
      }
    }
    if (++lk == per) {
      lk = 0;
      lc += 16;
    }
  };
  v4f acc = v4f{0.f, 0.f, 0.f, 0.f};
  int col = c_begin, k = 0, n = 0;      // the next consumed step's
  auto finish = [&]() {
    red[n & 1][wave][lane] = acc;
    lds_barrier();                      // halves in turn: see few_up_kernel
    if (wave == (n & 7) && r16 < p.T && col + 4 * g16 < c_end) {
      v4f s = red[n & 1][0][lane];
#pragma unroll
      for (int v = 1; v < FW_WAVES; ++v) s += red[n & 1][v][lane];
      const size_t at = (size_t)r16 * p.d + col + g16 * 4;
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
    acc = v4f{0.f, 0.f, 0.f, 0.f};
    k = 0;
    col += 16;
    ++n;
  };
  auto use = [&](const DownStep<U, STAGE>& st, auto&& refill) {
    v4f q[U];
    float s[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const v8i h = STAGE ? row_frag(stage + st.hrow * hstride + (st.kb + i) * 128 + g16 * 32) : st.hf[STAGE ? 0 : i];
      s[i] = (STAGE ? stage_s[st.hrow * FB + st.kb + i] : st.sh[STAGE ? 0 : i]) * st.sw[i];
      q[i] = mfma_fp8_16x16x128(weight_frag(st.b[i]), h, v4f{0.f, 0.f, 0.f, 0.f});
    }
    const bool live = st.live;   // other tokens take nothing, not even a NaN weight's product with 0
    refill();
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = live ? fmaf(q[i][j], s[i], acc[j]) : acc[j];
    if (++k == per) finish();
  };
#pragma unroll
  for (int r = 0; r < RING; ++r)
    if (r < count) load(ring[r]);
  if (STAGE) {
    auto put = [&](int tile, HTile& h) {
      const int row = tile / FB;
      uint2 q;
      const float s = h.template quantise<POW2>(q);
      *reinterpret_cast<uint2*>(stage + row * hstride + (tile - row * FB) * 128 + (tid & 15) * 8) = q;
      if ((tid & 15) == 0) stage_s[tile] = s * P.gate[row];
    };
#pragma unroll
    for (int i = 0; i < EARLY; ++i) {
      const int tile = (tid >> 4) + i * (FW_THREADS / 16);
      if (tile < tiles) put(tile, early[i]);
    }
    for (int tile = (tid >> 4) + EARLY * (FW_THREADS / 16); tile < tiles; tile += FW_THREADS / 16) {
      HTile h;
      h.load(p.h + (size_t)tile * 128 + (tid & 15) * 8);
      put(tile, h);
    }
    lds_barrier();
  }
  int u = 0;
  for (; u + 2 * RING <= count; u += RING) {
#pragma unroll
    for (int r = 0; r < RING; ++r) use(ring[r], [&] { load(ring[r]); });
  }
  for (; u < count; u += RING) {
#pragma unroll
    for (int r = 0; r < RING; ++r)
      if (u + r < count) use(ring[r], [&] {
        if (u + r + RING < count) load(ring[r]);
      });
  }
}

}  // namespace

size_t layer_few_workspace_bytes(int T, int d, int f, int E, int k) { return few_layout(T, d, f, E, k).total; }

hipError_t launch_layer_few(const uint16_t* x, const uint16_t* wg, const float* bias, int T, int d, int f, int E,
                            int G, int M, int k, float route_scale, const uint8_t* w13, const float* w13_s,
                            const uint8_t* w2, const float* w2_s, const uint16_t* residual, int32_t* idx, float* w,
                            uint16_t* out, void* workspace, bool pow2, hipStream_t stream) {
  const FewLayout L = few_layout(T, d, f, E, k);
  const int keep = std::min(k, E / G);
  int e_log2 = 0, c_log2 = 0;
  while ((1 << e_log2) < E) ++e_log2;
  while ((1 << c_log2) < G * keep) ++c_log2;
  // parts of d: as many as let a thread of the next kernel load all parts of its pairs by 16 loads
  const int pairs = ((T << e_log2) + FW_THREADS - 1) / FW_THREADS;
  const int splits = pairs <= 2 ? 8 : pairs <= 4 ? 4 : 2;
  char* ws = static_cast<char*>(workspace);
  FewArgs p{T, d, f, E, G, M, k, (double)route_scale, x, wg, bias, w13, w13_s, w2, w2_s, residual, idx, w, out,
            splits, e_log2, c_log2, reinterpret_cast<double*>(ws + L.part), reinterpret_cast<uint8_t*>(ws + L.xq),
            reinterpret_cast<float*>(ws + L.xs), reinterpret_cast<float*>(ws + L.h),
            reinterpret_cast<uint8_t*>(ws + L.hq), reinterpret_cast<float*>(ws + L.hsg),
            reinterpret_cast<FewPlan*>(ws + L.plan)};
  const int KB = d / 128, FB = f / 128;
  const dim3 g1((E + 15) / 16 * splits + (T * KB + FR_THREADS / 16 - 1) / (FR_THREADS / 16)), g3((T * (k + 1) * FB + 15) / 16);
  if (pow2) hipLaunchKernelGGL(few_route_kernel<true>, g1, dim3(FR_THREADS), 0, stream, p);
  else hipLaunchKernelGGL(few_route_kernel<false>, g1, dim3(FR_THREADS), 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // no more workgroups than items (each active expert has f/8)
  const dim3 g2(std::min(256, std::min(E, T * k) * (f / 8) + f / 8));
  switch ((KB + 7) / 8) {
    case 1: hipLaunchKernelGGL(few_up_kernel<1>, g2, dim3(FW_THREADS), 0, stream, p); break;
    case 2: hipLaunchKernelGGL(few_up_kernel<2>, g2, dim3(FW_THREADS), 0, stream, p); break;
    case 3: hipLaunchKernelGGL(few_up_kernel<3>, g2, dim3(FW_THREADS), 0, stream, p); break;
    case 4: hipLaunchKernelGGL(few_up_kernel<4>, g2, dim3(FW_THREADS), 0, stream, p); break;
    case 5: hipLaunchKernelGGL(few_up_kernel<5>, g2, dim3(FW_THREADS), 0, stream, p); break;
    case 6: hipLaunchKernelGGL(few_up_kernel<6>, g2, dim3(FW_THREADS), 0, stream, p); break;
    case 7: hipLaunchKernelGGL(few_up_kernel<7>, g2, dim3(FW_THREADS), 0, stream, p); break;
    default: hipLaunchKernelGGL(few_up_kernel<8>, g2, dim3(FW_THREADS), 0, stream, p); break;
  }
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int rows = T * (k + 1);
  const bool stage = (long)rows * (f + 16 + FB * 4) <= FW_STAGE_BYTES;
  if (!stage) {
    if (pow2) hipLaunchKernelGGL(few_quant_kernel<true>, g3, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL(few_quant_kernel<false>, g3, dim3(256), 0, stream, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 g4(std::min(256, d / 4));
#define MOE_FEW_DOWN(U, RING, STAGE, POW2) \
  hipLaunchKernelGGL((few_down_kernel<U, RING, STAGE, POW2>), g4, dim3(FW_THREADS), 0, stream, p)
  if (FB % 2 == 0) {
    if (!stage) MOE_FEW_DOWN(2, 4, false, false);
    else if (pow2) MOE_FEW_DOWN(2, 6, true, true);
    else MOE_FEW_DOWN(2, 6, true, false);
  } else {
    if (!stage) MOE_FEW_DOWN(1, 8, false, false);
    else if (pow2) MOE_FEW_DOWN(1, 12, true, true);
    else MOE_FEW_DOWN(1, 12, true, false);
  }
#undef MOE_FEW_DOWN
  return hipGetLastError();
}

}  // namespace moe
