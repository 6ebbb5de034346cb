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
//     rows: 8 gate and the 8 matching up rows (fragment rows 0..7 and 8..15).
//     With 9 experts there are still nine items per CU, and all waves stream.
//   * A workgroup of the second product owns some output columns (28 at d
//     7168) and walks every active expert for them, so the gated sum over
//     experts is its accumulator and the combine, in registers: expert outputs
//     never reach memory.
//
// Bound by HBM reads from T = 4 on: at d 7168, f 2048, E 256, k 8 a call takes
// 215 to 233 us at T = 4 (29 to 33 active experts, 1.28 to 1.45 GB, 6.1 to 6.4
// TB/s) and 637 to 714 at T = 16 (89 to 105 of them, 3.9 to 4.6 GB, 6.3 to 6.5
// TB/s); a plain read of the card's memory makes 7.05.  At T = 1 it takes 75 to
// 79 us for 396 MB, 56 at that rate: the router's kernel is 5.8 of them, the rest
// of the difference the selection where the first weights do not cover it and the
// starts and ends of the two products (46 and 26 us).  Where a batch is small
// the kernels' code counts: its first fetch takes some 0.1 us per 128 bytes, so
// what runs once is kept short (loops rolled, divisions on the host).
#include <algorithm>
#include <cstddef>
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
  size_t part, xq, xs, h, hq, hsg, plan, sum, ticket, total;
};

struct FewPlan {                        // written by the first product's first two workgroups
  int n_active;                         // the shared expert, then those with a token, ascending
  int expert[FW_MAX_E + 1];
  int pad[2];
  uint8_t slot[FW_MAX_E + 1][FW_T];     // slot of token t in active expert a, or 255
  float gate[FW_T * (FW_MAX_K + 1)];    // of row t (k + 1) + slot
};
constexpr int kPlanLoads = sizeof(FewPlan) / 16;
constexpr int kPlan = offsetof(FewPlan, gate) / 16;    // of them without the gates
static_assert(kPlanLoads <= FW_THREADS && sizeof(FewPlan) % 16 == 0 && offsetof(FewPlan, gate) % 16 == 0,
              "a thread moves 16 bytes of the plan");

// Workgroups of the last kernel that share the steps of 16 output columns: as
// many as fill 256, with two steps or more for each wave (a token's k + 1
// experts have that many at least).  1: the columns are shared out instead.
// With 64 experts, k 8, f 2048, us a call shared against not, at T = 16: d 512
// 67, 104; d 1024 81, 111; d 2048 132, 154; at T = 1 26.5, 28.7; 27.8, 30.1;
// 35.4, 36.3.  With 320 to 512 workgroups it was 85 to 93 at d 1024, and at d
// 2560, where 256 are not reached without (160 of them), 193 against 188.
constexpr int FW_MAX_SPLITS = 16;
int few_splits(int d, int f, int k) {
  return std::max(1, std::min({FW_MAX_SPLITS, 256 / (d / 16), (k + 1) * (f / 128) / (2 * FW_WAVES)}));
}

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
  const int splits = few_splits(d, f, k);
  L.sum = take(splits > 1 ? (size_t)splits * d * FW_T * sizeof(float) : 0);
  L.ticket = take(splits > 1 ? (size_t)(d / 16) * sizeof(int) : 0);
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
  int s_log2;       // parts of d in the logits' partial sums: 8, 4 or 2
  int e_log2;       // experts and candidates of a token, rounded up to powers of two
  int c_log2;
  int per, keep, n_top;   // experts of a group; its best that the selection looks at, and those that rank it
  uint32_t inv_per, inv_keep;   // 2^16 over them, rounded up
  uint32_t inv_f8, inv_fb, inv_groups, inv_splits;   // 2^32 over f/8, f/128, d/16 and splits, rounded up
  double* part;     // [T, E, splits] partial logits
  uint8_t* xq;      // [T, d]
  float* xs;        // [T, d/128]
  float* h;         // [T (k+1), f]
  uint8_t* hq;      // [T (k+1), f]
  float* hsg;       // [T (k+1), f/128]: scale times gate
  FewPlan* plan;
  float* sum;       // [splits, d/16, 64, 4]: the last kernel's partial sums
  int* ticket;      // [d/16]: how many of them are there
  int splits;
};

// All cache lines of the arguments at once, at a kernel's start: left to itself
// the compiler loads each argument where it is first needed, and waits there.
__device__ __forceinline__ void fetch_args(const FewArgs& p) {
  const int* a = reinterpret_cast<const int*>(&p);
  static_assert(sizeof(FewArgs) > 192 && sizeof(FewArgs) <= 256, "four lines of 64 bytes");
  asm volatile("" ::"s"(a[0]), "s"(a[16]), "s"(a[32]), "s"(a[48]));
}

// Barrier that leaves this wave's loads in flight: waits for its LDS accesses
// only (vmcnt untouched).
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Weights come through buffer loads: a 64-bit base in scalar registers and a
// 32-bit offset per lane, which keeps the address arithmetic off the vector
// units, and a bound that turns a load into nothing.  A load of an empty
// buffer, or at kNowhere, reads no memory and returns zeros, so the places
// where a stream has nothing more to load need no branch.  That matters
// twice: the compiler counts outstanding loads along straight-line code only,
// and waits for all of them after a load that may not have been issued
// (measured: 3.8 TB/s instead of 6.5); and a second copy of the loop for its
// end would have to be fetched as code, at about 0.15 us per 128 bytes the
// first time it is reached in a launch.
constexpr uint32_t kNowhere = 0x7FFFFFF0u;
typedef int i32x4 __attribute__((ext_vector_type(4)));

// The buffer of everything from a wave-uniform base on (offsets stay below
// kNowhere), or an empty one.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* base, bool there) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(uniform_ptr(base)), 0, there ? 0x7FFFFFE0 : 0,
                                           0x00020000);
}
__device__ __forceinline__ float load_scale(__amdgpu_buffer_rsrc_t b, uint32_t off) {
  return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(b, off, 0, 0));
}

// Nothing is scheduled across: left alone, the compiler gathers a loop's loads
// at its end and waits for all of them at its beginning.
__device__ __forceinline__ void pin_loads() { __builtin_amdgcn_sched_barrier(0); }

// Weight fragment loads: 16 rows of 128 bytes as two whole-line loads (8 rows
// each), then two DPP moves per register give the MFMA's operand layout.  Lane
// (g, j) loads 16 bytes of chunk 2g + (j >= 8) from row j % 8 of each half;
// rotating each 16-lane row by 8 and taking half of its lanes leaves lane
// (g, j) with chunks 2g and 2g + 1 of fragment row j.
struct Lines {
  i32x4 x, y;
};

__device__ __forceinline__ Lines load_weight(__amdgpu_buffer_rsrc_t b, uint32_t x, uint32_t y) {
  constexpr int kNonTemporal = 2;
  return {__builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(b, x, 0, kNonTemporal)),
          __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(b, y, 0, kNonTemporal))};
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

// ---- kernel 1: partial logits and the tiles of x ----
// A workgroup takes 16 experts and one of `splits` parts of d, so that the
// 3.7 MB of V3's router come through 128 CUs (5.4 us for up to 4 tokens); the
// next kernel adds the parts.  With more tokens every part costs that kernel
// more loads in each workgroup: eight parts instead of two at 16 tokens took
// 9 us off this kernel (15 -> 6) and put as many onto the next one.
// The products run on the FP64 MFMA (16 experts by 16 tokens by 4 elements):
// BF16 values are exact there, so the scores that the selection compares carry
// errors of 10^-15 only, whatever the order of the sum.  (The BF16 MFMA would
// be eight times as fast, but its logits were 3.5e-8 RMS off, 1.7e-7 at most:
// as far as neighbouring scores can be apart.)  A lane loads eight consecutive
// elements of its row and feeds them to eight MFMAs; which four elements meet
// in one does not matter as long as both operands agree.
typedef double v4d __attribute__((ext_vector_type(4)));

template <bool POW2>
__global__ __launch_bounds__(FR_THREADS) void few_route_kernel(const FewArgs p) {
  __shared__ v4d red[FR_WAVES][64];
  fetch_args(p);
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int router = (p.E + 15) / 16 << p.s_log2;
  if (blockIdx.x == 0 && p.splits > 1 && tid < p.d / 16) p.ticket[tid] = 0;
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
    const float s = tile_scale<POW2>(row_max(amax));
    uint2 q;
    q.x = f32x4_to_e4m3(v[0] / s, v[1] / s, v[2] / s, v[3] / s);
    q.y = f32x4_to_e4m3(v[4] / s, v[5] / s, v[6] / s, v[7] / s);
    *reinterpret_cast<uint2*>(p.xq + (size_t)tile * 128 + sub * 8) = q;
    if (sub == 0) p.xs[tile] = s;
    return;
  }
  const int e0 = ((int)blockIdx.x >> p.s_log2) * 16, split = (int)blockIdx.x & ((1 << p.s_log2) - 1);
  const int r16 = lane & 15, g16 = lane >> 4;
  // rows past the last expert or token repeat it; their results are not stored
  const uint16_t* wr = p.wg + (size_t)min(e0 + r16, p.E - 1) * p.d + g16 * 8;
  const uint16_t* xr = p.x + (size_t)min(r16, p.T - 1) * p.d + g16 * 8;
  const int chunks = p.d / 32;
  v4d acc = v4d{0.0, 0.0, 0.0, 0.0};
  const int stride = FR_WAVES << p.s_log2;   // the parts interleave
  for (int c0 = split * FR_WAVES + wave; c0 < chunks; c0 += stride * FR_RING) {
    uint4 a[FR_RING], b[FR_RING];
#pragma unroll
    for (int r = 0; r < FR_RING; ++r) {
      const int c = min(c0 + r * stride, chunks - 1);
      a[r] = *reinterpret_cast<const uint4*>(wr + c * 32);
      b[r] = *reinterpret_cast<const uint4*>(xr + c * 32);
    }
#pragma unroll
    for (int r = 0; r < FR_RING; ++r) {
      if (c0 + r * stride < chunks) {   // uniform over the wave
        const uint32_t au[4] = {a[r].x, a[r].y, a[r].z, a[r].w}, bu[4] = {b[r].x, b[r].y, b[r].z, b[r].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc = __builtin_amdgcn_mfma_f64_16x16x4f64(__uint_as_float(au[i] << 16), __uint_as_float(bu[i] << 16), acc,
                                                     0, 0, 0);
          acc = __builtin_amdgcn_mfma_f64_16x16x4f64(__uint_as_float(au[i] & 0xFFFF0000u),
                                                     __uint_as_float(bu[i] & 0xFFFF0000u), acc, 0, 0, 0);
        }
      }
    }
  }
  red[wave][lane] = acc;
  __syncthreads();
  // an FP64 MFMA leaves lane l with rows (experts) l / 16 + 4 i, column (token) l % 16
  if (tid < 256) {
    const int i = tid >> 6, e = e0 + g16 + 4 * i;
    double l = red[0][lane][i];
#pragma unroll
    for (int v = 1; v < FR_WAVES; ++v) l += red[v][lane][i];
    if (r16 < p.T && e < p.E) p.part[(r16 * p.E + e << p.s_log2) + split] = l;
  }
}

// ---- selection, by a whole workgroup, (token, expert) pairs over its threads ----
struct SelectLds {
  uint64_t key[FW_T][FW_MAX_E];          // biased scores in order: larger is better
  uint64_t best[FW_T][FW_MAX_E];         // [group][rank]: keys of each group's best, in order
  double sig[FW_T][FW_MAX_E];            // affinities
  uint64_t group[FW_T][64];              // the groups' sums as keys
  double gate[FW_T][FW_MAX_K];
  uint64_t kept[FW_T];                   // groups kept
  uint32_t mask[FW_T][FW_MAX_E / 32];    // experts chosen
  uint32_t active[FW_MAX_E / 32];        // experts any token chose
  int16_t chosen[FW_T][FW_MAX_K];        // ascending
  uint8_t who[FW_T][FW_MAX_E];           // the experts of `best`
};

// The partial logits of this thread's (token, expert) pairs: pair tid + 512 i
// of the tokens' rows of 2^e_log2, in 2^s_log2 parts each, 8 loads in all.
// The scores are made of them before the first weights are asked for: beside
// the chip's weight loads that took 3 us instead of 1.
struct PartialLogits {
  double2 v[8];
  float bias;       // of this thread's expert, the same for all its pairs

  __device__ __forceinline__ void load(const FewArgs& p) {
    const uint32_t e = min((int)threadIdx.x & ((1 << p.e_log2) - 1), p.E - 1);
    const uint32_t t0 = threadIdx.x >> p.e_log2, dt = FW_THREADS >> p.e_log2;
    const uint32_t h_log2 = p.s_log2 - 1;   // a pair's parts, two a load
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const uint32_t t = min(t0 + (q >> h_log2) * dt, (uint32_t)p.T - 1);
      v[q] = reinterpret_cast<const double2*>(p.part)[(t * p.E + e << h_log2) + (q & ((1 << h_log2) - 1))];
    }
    bias = p.bias ? p.bias[e] : 0.0f;
  }
  // The pairs' logits, in order.
  __device__ __forceinline__ void sums(const FewArgs& p, double (&l)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) l[i] = v[i].x + v[i].y;
    if (p.s_log2 > 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) l[i] = l[2 * i] + l[2 * i + 1];
    if (p.s_log2 > 2)
#pragma unroll
      for (int i = 0; i < 2; ++i) l[i] = l[2 * i] + l[2 * i + 1];
  }
};

// Doubles in an unsigned order, all bits of them: scores that differ in the
// last one rank by it.  Equal scores rank by the lower index (of an expert or,
// for a sum, of a group).  NaN scores rank as minus infinity, so every index
// below stays in range whatever the inputs.
__device__ __forceinline__ uint64_t score_key(double z) {
  if (!(z == z)) z = -__builtin_huge_val();
  const uint64_t u = (uint64_t)__double_as_longlong(z + 0.0);   // -0 as +0
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double key_score(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? k & 0x7FFFFFFFFFFFFFFFull : ~k));
}

// Entries of list[0..n) above k.
__device__ __forceinline__ int count_above(const uint64_t* list, int n, uint64_t k) {
  int r = 0;
#pragma unroll 4
  for (int i = 0; i < n; ++i) r += list[i] > k ? 1 : 0;
  return r;
}
// The rank of list[own]: entries above it, and equal ones before it.  (k - 1 is
// a key's lower neighbour: the smallest, minus infinity's, is above 0.)
__device__ __forceinline__ int rank_of(const uint64_t* list, int n, int own, uint64_t k) {
  int r = 0;
#pragma unroll 4
  for (int i = 0; i < n; ++i) r += list[i] > k - (i < own ? 1 : 0) ? 1 : 0;
  return r;
}

// Affinities, biased scores and keys from this thread's logits, and the cleared
// rest of the selection's LDS.
__device__ __forceinline__ void few_scores(const FewArgs& p, SelectLds& S, FewPlan& P, double (&l)[8], float bias) {
  const int tid = threadIdx.x, e_mask = (1 << p.e_log2) - 1, pairs = p.T << p.e_log2;
  static_assert(sizeof(P.slot) / 16 <= FW_THREADS && offsetof(FewPlan, slot) % 16 == 0, "cleared by 16 bytes a thread");
  if (tid < FW_MAX_E / 32) S.active[tid] = 0;
  if (tid < FW_T) S.kept[tid] = 0;
  if (tid < FW_T * FW_MAX_E / 32) S.mask[0][tid] = 0;
  if (tid < (int)sizeof(P.slot) / 16) reinterpret_cast<uint4*>(P.slot)[tid] = make_uint4(~0u, ~0u, ~0u, ~0u);
#pragma unroll 1
  for (int at = tid; at < pairs; at += FW_THREADS) {   // one copy of exp: the logits shift down to it
    const int t = at >> p.e_log2, e = at & e_mask;
    if (e < p.E) {
      const double s = 1.0 / (1.0 + exp(-l[0])), z = s + (double)bias;
      S.sig[t][e] = s;
      S.key[t][e] = score_key(z);
    }
#pragma unroll
    for (int i = 0; i < 7; ++i) l[i] = l[i + 1];
  }
}

// The batch's plan in LDS.  Ranks are counted, not sorted: an expert's rank in
// its group is the number of better ones there; the best min(k, group size) of
// each group, in order, are all that the later steps read.  `between` runs after
// each of the first four barriers: the caller issues loads there.
template <typename Between>
__device__ __forceinline__ void few_select(const FewArgs& p, SelectLds& S, FewPlan& P, bool write_out,
                                           Between between) {
  const int tid = threadIdx.x;
  const int per = p.per, keep = p.keep, n_top = p.n_top, cand = p.G * keep;
  // i / per and i / keep for i < 256 by 16-bit reciprocals (exact: the error 255 / 65536 is below 1 / 256)
  const uint32_t inv_per = p.inv_per, inv_keep = p.inv_keep;
  const int e_mask = (1 << p.e_log2) - 1, c_mask = (1 << p.c_log2) - 1;
  const int pairs = p.T << p.e_log2, cands = p.T << p.c_log2;
  lds_barrier();
  between(std::integral_constant<int, 0>{});
  for (int at = tid; at < pairs; at += FW_THREADS) {
    const int t = at >> p.e_log2, e = at & e_mask, g = (int)(e * inv_per >> 16);
    if (e >= p.E) continue;
    const uint64_t k = S.key[t][e];
    const int r = rank_of(&S.key[t][g * per], per, e - g * per, k);
    if (r < keep) {
      S.best[t][g * keep + r] = k;
      S.who[t][g * keep + r] = (uint8_t)e;
    }
  }
  lds_barrier();
  between(std::integral_constant<int, 1>{});
  for (int at = tid; at < p.T * 64; at += FW_THREADS) {
    const int t = at >> 6, g = at & 63;
    if (g >= p.G) continue;
    double s = 0.0;
#pragma unroll 1
    for (int r = 0; r < n_top; ++r) s += key_score(S.best[t][g * keep + r]);
    S.group[t][g] = score_key(s);
  }
  lds_barrier();
  between(std::integral_constant<int, 2>{});
  for (int at = tid; at < p.T * 64; at += FW_THREADS) {
    const int t = at >> 6, g = at & 63;
    if (g >= p.G) continue;
    const int r = rank_of(S.group[t], p.G, g, S.group[t][g]);
    if (r < p.M) atomicOr(reinterpret_cast<unsigned long long*>(&S.kept[t]), 1ull << g);
  }
  lds_barrier();
  between(std::integral_constant<int, 3>{});
  for (int at = tid; at < cands; at += FW_THREADS) {
    const int t = at >> p.c_log2, c = at & c_mask, g = (int)(c * inv_keep >> 16);
    const uint64_t kept = S.kept[t];
    if (c >= cand || !((kept >> g) & 1)) continue;
    const uint64_t k = S.best[t][c];
    int r = c - g * keep;
    for (uint64_t m = kept & ~(1ull << g); m; m &= m - 1) {
      const int o = __ffsll((unsigned long long)m) - 1;   // all its experts come before or after this one's
      r += count_above(&S.best[t][o * keep], keep, k - (o < g ? 1 : 0));
    }
    if (r < p.k) {
      const int e = S.who[t][c];
      atomicOr(&S.mask[t][e >> 5], 1u << (e & 31));
      atomicOr(&S.active[e >> 5], 1u << (e & 31));
    }
  }
  lds_barrier();
  // experts of a bit mask below e
  auto place = [](const uint32_t* mask, int e) {
    int a = __popc(mask[e >> 5] & ((1u << (e & 31)) - 1u));
#pragma unroll 2
    for (int i = 0; i < (e >> 5); ++i) a += __popc(mask[i]);
    return a;
  };
  // a chosen expert is one of its group's best, so the candidates hold them all
  for (int at = tid; at < cands; at += FW_THREADS) {
    const int t = at >> p.c_log2, c = at & c_mask, g = (int)(c * inv_keep >> 16);
    if (c >= cand || !((S.kept[t] >> g) & 1)) continue;
    const int e = S.who[t][c];
    if (!((S.mask[t][e >> 5] >> (e & 31)) & 1)) continue;
    const int j = place(S.mask[t], e), a = 1 + place(S.active, e);
    S.chosen[t][j] = (int16_t)e;
    S.gate[t][j] = S.sig[t][e];
    P.expert[a] = e;
    P.slot[a][t] = (uint8_t)j;
  }
  if (tid < p.T) P.slot[0][tid] = (uint8_t)p.k;
  if (tid == FW_THREADS - 1) {
    P.n_active = 1 + place(S.active, FW_MAX_E - 1) + (int)(S.active[FW_MAX_E / 32 - 1] >> 31);
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
      p.plan->gate[t * (p.k + 1) + j] = w;
    }
  }
}

// ---- kernel 2: selection, then h = SiLU(G) U in FP32 ----
// Item i: active expert i / (f/8), h columns 8 (i % (f/8)) .. +7.  Wave w owns
// the K blocks w, w + 8, ... (NB = ceil(d/1024) of them): their activations
// and scales stay in registers, and as each block's weights are consumed those
// of the item D further on are loaded into their place.
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

// Items of a turn (D), whose 16 KB a block are in flight together: 64 KB for one
// and two blocks (NB), one item from three blocks (48 KB) on.  With 64 experts
// and f 2048, us a call at T = 16: d 1024 140 with one item, 114 with two, 110
// with four; d 2048 173, 154, 156; d 2560 188, 185 (but 36.9, 38.6 at T = 4 and
// f 512); d 4096 247, 248.
constexpr int few_items(int NB) { return NB == 1 ? 4 : NB == 2 ? 2 : 1; }

template <int NB, int D>
__global__ __launch_bounds__(FW_THREADS, 1) void few_up_kernel(const FewArgs p) {
  __shared__ __attribute__((aligned(16))) SelectLds S;
  __shared__ __attribute__((aligned(16))) FewPlan P;
  fetch_args(p);
  // the waves' sums, where the selection's keys were
  v4f (*const red)[D][FW_WAVES][64] = reinterpret_cast<v4f(*)[D][FW_WAVES][64]>(&S.key);
  static_assert(2 * sizeof(*red) <= sizeof(S.key) + sizeof(S.best) && offsetof(SelectLds, best) == sizeof(S.key));
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int g16 = lane >> 4, r16 = lane & 15;
  const int KB = p.d / 128, FB = p.f / 128, per = p.f / 8;

  PartialLogits part;
  part.load(p);
  // activations of this wave's blocks; tokens past T repeat the last, a
  // missing last block the block KB - 1 (its weights read as zeros, and its
  // scale is a zero: the block's own may be infinite)
  v8i xq[NB];
  float xs[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int kb = min(wave + 8 * j, KB - 1), t = min(r16, p.T - 1);
    xq[j] = row_frag(p.xq + (size_t)t * p.d + kb * 128 + g16 * 32);
    const float scale = p.xs[t * KB + kb];
    xs[j] = wave + 8 * j < KB ? scale : 0.0f;
  }
  double logits[8];
  part.sums(p, logits);
  few_scores(p, S, P, logits, part.bias);
  pin_loads();
  // offsets of this lane's loads from an item's first gate row and its scale
  const uint32_t gate_off = (r16 & 7) * p.d + (2 * g16 + (r16 >> 3)) * 16 + wave * 128;
  const uint32_t up_off = gate_off + (uint32_t)p.f * p.d;
  const uint32_t scale_off = ((g16 < 2 ? 0 : FB) * KB + wave) * 4;
  const bool last = wave + 8 * (NB - 1) < KB;   // this wave has the last block too
  Lines b[D][NB];
  float sw[D][NB];
  auto load = [&](int i, int j, __amdgpu_buffer_rsrc_t wb, __amdgpu_buffer_rsrc_t sb) {
    const bool there = j + 1 < NB || last;
    b[i][j] = load_weight(wb, there ? gate_off + j * 1024 : kNowhere, there ? up_off + j * 1024 : kNowhere);
    sw[i][j] = load_scale(sb, there ? scale_off + j * 32 : kNowhere);
  };
  auto weights_of = [&](int e, int n8, bool there) {
    return buffer_at(p.w13 + ((size_t)e * 2 * p.f + n8 * 8) * p.d, there);
  };
  auto scales_of = [&](int e, int n8, bool there) {
    return buffer_at(p.w13_s + ((size_t)e * 2 * FB + n8 / 16) * KB, there);
  };
  // The first `per` items are the shared expert's, known before the selection:
  // their loads run beneath it, three sevenths now and a seventh after each of
  // its first steps.  A CU takes some 50 KB of loads at once; with all 115 KB
  // here the later waves stood 3 us before the first barrier.
  const bool early = (int)blockIdx.x < per;
  const __amdgpu_buffer_rsrc_t wb0 = weights_of(p.E, blockIdx.x, early), sb0 = scales_of(p.E, blockIdx.x, early);
  auto load_part = [&](auto step) {
    constexpr int from = step == 0 ? 0 : (NB * (2 + step) + 6) / 7, to = (NB * (3 + step) + 6) / 7;
    pin_loads();
#pragma unroll
    for (int j = from; j < to; ++j) {
      load(D - 1, j, wb0, sb0);
      pin_loads();   // in the loop's order
    }
  };
#pragma unroll
  for (int i = 0; i + 1 < D; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) b[i][j] = Lines{}, sw[i][j] = 0.0f;
  load_part(std::integral_constant<int, 0>{});
  few_select(p, S, P, blockIdx.x == 0,
             [&](auto i) { load_part(std::integral_constant<int, decltype(i)::value + 1>{}); });
  // the plan, but for the gates, which are workgroup 0's (the grid has 32 or more)
  if (blockIdx.x == 1 && tid < kPlan) reinterpret_cast<uint4*>(p.plan)[tid] = reinterpret_cast<const uint4*>(&P)[tid];
  const int total = __builtin_amdgcn_readfirstlane(P.n_active) * per;

  // This workgroup's items are blockIdx + q gridDim, q = 0, 1, ...; a turn takes
  // D of them, q .. q + D - 1, and loads the next turn's.  Of the first turn at
  // most the last is there, the one loaded before the selection; the others,
  // and items past the end, are zeros that nothing is loaded for.
  int rot = 0, half = 0;
  for (int q = early ? 1 - D : -D; q < 0 || (int)blockIdx.x + q * (int)gridDim.x < total; q += D) {
    asm volatile("" : "+s"(q));   // or the first turn gets a copy of the code to itself
    __amdgpu_buffer_rsrc_t wb[D], sb[D];
#pragma unroll
    for (int i = 0; i < D; ++i) {
      const int next = (int)blockIdx.x + (q + D + i) * (int)gridDim.x;
      const bool more = next < total;
      const int a = (int)__umulhi((uint32_t)next, p.inv_f8), n8 = next - a * per;
      const int e = __builtin_amdgcn_readfirstlane(P.expert[more ? a : 0]);
      wb[i] = weights_of(e, n8, more);
      sb[i] = scales_of(e, n8, more);
    }
    v4f acc[D];
#pragma unroll
    for (int i = 0; i < D; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      // widened here for the turn's D items: widened ahead of the loop it was no
      // faster, and eight blocks of it spilled (d 8192: 4.2 TB/s instead of 6)
      asm volatile("" : "+v"(xq[j]));
      v8bf x[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = widen8(xq[j][2 * c], xq[j][2 * c + 1]);
#pragma unroll
      for (int i = 0; i < D; ++i) {
        const v8i w = weight_frag(b[i][j]);
        float s = sw[i][j] * xs[j];
        asm volatile("" : "+v"(s));   // the product is made, and sw free, before it is loaded again
        pin_loads();
        load(i, j, wb[i], sb[i]);
        v4f t = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) t = mfma_bf16_16x16x32(widen8(w[2 * c], w[2 * c + 1]), x[c], t);
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][c] = fmaf(t[c], s, acc[i][c]);
        pin_loads();
      }
    }
    if (q + D > 0) {
      // The waves' partial sums through LDS, in two halves in turn: one barrier
      // per turn, since a half is written again only after the next turn's
      // barrier, which the waves that read it reach afterwards.  A wave each
      // for the turn's items.
#pragma unroll
      for (int i = 0; i < D; ++i) red[half][i][wave][lane] = acc[i];
      lds_barrier();
      const int i = (wave - rot) & (FW_WAVES - 1), item = (int)blockIdx.x + (q + i) * (int)gridDim.x;
      if (i < D && q + i >= 0 && item < total) {
        v4f s = red[half][i][0][lane];
#pragma unroll
        for (int v = 1; v < FW_WAVES; ++v) s += red[half][i][v][lane];
        // lanes 0..31 hold G (columns 4 g16 .. +3), lanes 32..63 U of the same
        // columns: each half takes two of the four
        const bool hi = g16 >= 2;
        const float g0 = hi ? s[0] : s[2], g1 = hi ? s[1] : s[3];     // what the other half needs
        const float o0 = __shfl_xor(g0, 32), o1 = __shfl_xor(g1, 32);
        const float h0 = swiglu_f32(hi ? o0 : s[0], hi ? s[2] : o0);
        const float h1 = swiglu_f32(hi ? o1 : s[1], hi ? s[3] : o1);
        const int a = (int)__umulhi((uint32_t)item, p.inv_f8), slot = P.slot[a][r16];
        if (slot != 255)
          *reinterpret_cast<float2*>(p.h + (size_t)(r16 * (p.k + 1) + slot) * p.f + (item - a * per) * 8 +
                                     (g16 & 1) * 4 + (hi ? 2 : 0)) = make_float2(h0, h1);
      }
      half ^= 1;
      rot += D;
    }
  }
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
  // fp8_quant_1x128's: by Divider, for which tiles with a scale below 2^-60
  // are lifted by an exact power of two so that its reciprocal and its
  // remainders are normal numbers.  Of an infinite scale the quotients are
  // zeros, and NaN of an infinity: what times 0 makes of either.
  template <bool POW2>
  __device__ __forceinline__ float quantise(uint2& q) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
    const float s = tile_scale<POW2>(row_max(amax));
    const bool endless = s > 0x1p126f;    // a finite one is below 2^121
    const float lift = s < 0x1p-60f ? 0x1p80f : endless ? 0.0f : 1.0f;
    const Divider div(endless ? 1.0f : s * lift);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = div(v[i] * lift);
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
// A workgroup owns some output columns, up to 16 C in C fragments: an even share
// in units of 4 (missing rows of the last fragment read as zeros), or, of narrow
// layers, 16 whose steps several workgroups share (few_splits).
// The steps (active expert, K block; 2 C KB of weights) are dealt to the waves
// in turn, with RING of them in flight per wave: 64 KB per CU with two whole
// fragments, where rings of 3 to 7 changed nothing at V3; 32 KB (48 with a ring
// of 3) with one, less where the fragment is part empty (d 2560: 8 or 12 of its
// 16 rows, 73 us at T = 16, 64 experts, f 2048, for 43 of bytes).  A step's h
// serves all fragments, and one barrier joins the waves' sums at the end.
//
// STAGE: the workgroup quantises h itself, into LDS, beneath its first weight
// loads; otherwise the tiles come from few_quant_kernel through memory, and
// lanes whose token did not choose the expert load nothing.
constexpr int FW_STAGE_BYTES = 38 * 1024;
static_assert(kFewMaxD <= 256 * 32, "a workgroup's columns fit two fragments");

template <int C, bool STAGE>
struct DownStep {
  Lines b[C];
  float sw[C];
  v8i hf;         // not STAGE
  float sh;
  int row, kb;    // STAGE: this lane's h
  bool live;      // this lane's token chose the expert
};

template <int C, int RING, bool STAGE, bool POW2>
__global__ __launch_bounds__(FW_THREADS, 1) void few_down_kernel(const FewArgs p) {
  __shared__ __attribute__((aligned(16))) FewPlan P;
  __shared__ __attribute__((aligned(16))) v4f red[C][FW_WAVES][64];
  __shared__ __attribute__((aligned(16))) uint8_t stage[STAGE ? FW_STAGE_BYTES : 16];
  fetch_args(p);
  constexpr int EARLY = 5;              // tiles of h a thread loads before the weights (9 rows of f 2048)
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int g16 = lane >> 4, r16 = lane & 15;
  const int FB = p.f / 128;
  const int tiles = p.T * (p.k + 1) * FB;
  // the plan, 16 bytes a thread (threads past its end the last again), on its
  // way together with the tiles of h
  const int at = min(tid, kPlanLoads - 1);
  const uint4 plan = reinterpret_cast<const uint4*>(p.plan)[at];
  pin_loads();
  HTile early[STAGE ? EARLY : 1];
  if (STAGE) {
#pragma unroll
    for (int i = 0; i < EARLY; ++i)
      early[i].load(p.h + (size_t)min((tid >> 4) + i * (FW_THREADS / 16), tiles - 1) * 128 + (tid & 15) * 8);
  }
  pin_loads();
  reinterpret_cast<uint4*>(&P)[at] = plan;
  lds_barrier();
  const int all = __builtin_amdgcn_readfirstlane(P.n_active) * FB;
  // Either 16 columns and a share of the steps, or all steps and a share of the
  // d/4 units of columns, of which 256 workgroups have some each.
  const bool shared = C == 1 && p.splits > 1;
  const int units = p.d / 4, groups = p.d / 16;
  const int split = shared ? (int)__umulhi(blockIdx.x, p.inv_groups) : 0, group = (int)blockIdx.x - split * groups;
  int c_begin = 16 * group, c_end = c_begin + 16, first = 0, steps = all;
  if (shared) {
    first = (int)__umulhi(all * split, p.inv_splits);
    steps = (int)__umulhi(all * (split + 1), p.inv_splits);
  } else {
    c_begin = 4 * (units >= 256 ? units * (int)blockIdx.x >> 8 : (int)blockIdx.x);
    c_end = 4 * (units >= 256 ? units * ((int)blockIdx.x + 1) >> 8 : (int)blockIdx.x + 1);
  }
  const uint32_t inv = p.inv_fb;        // a step's expert: step / FB
  const int hstride = p.f + 16;         // staged rows, 16 bytes apart in the banks
  float* const stage_s = reinterpret_cast<float*>(stage + p.T * (p.k + 1) * hstride);
  // this lane's offsets from an expert's weights and scales
  uint32_t wo[C][2], so[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = c_begin + 16 * c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = col + 8 * i + (r16 & 7);
      wo[c][i] = r < c_end ? (uint32_t)r * p.f + (2 * g16 + (r16 >> 3)) * 16 : kNowhere;
    }
    so[c] = col + 4 * g16 < c_end ? (uint32_t)(col + 4 * g16) / 128 * FB * 4 : kNowhere;
  }
  const __amdgpu_buffer_rsrc_t hb = buffer_at(p.hq, true), gb = buffer_at(p.hsg, true);

  DownStep<C, STAGE> ring[RING];
  int next = first + wave;              // the step to load next
  auto load = [&](DownStep<C, STAGE>& st) {
    const bool there = next < steps;
    const int a = !there ? 0 : FB == 1 ? next : (int)__umulhi((uint32_t)next, inv);
    const int kb = there ? next - a * FB : 0;
    const int e = __builtin_amdgcn_readfirstlane(P.expert[a]);
    const __amdgpu_buffer_rsrc_t wb = buffer_at(p.w2 + (size_t)e * p.d * p.f + kb * 128, there);
    const __amdgpu_buffer_rsrc_t sb = buffer_at(p.w2_s + (size_t)e * (p.d / 128) * FB + kb, there);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      st.b[c] = load_weight(wb, wo[c][0], wo[c][1]);
      st.sw[c] = load_scale(sb, so[c]);
    }
    const int slot = P.slot[a][r16];
    st.live = there && slot != 255;     // past the end: nothing, whatever h's scale
    const uint32_t row = r16 * (p.k + 1) + slot;
    if (STAGE) {
      st.row = st.live ? row : 0;
      st.kb = kb;
    } else {
      const uint32_t at = st.live ? row * p.f + kb * 128 + g16 * 32 : kNowhere;
      const i32x4 lo = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(hb, at, 0, 0));
      const i32x4 hi = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(hb, at + 16, 0, 0));
      st.hf = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      st.sh = load_scale(gb, st.live ? (row * FB + kb) * 4 : kNowhere);
    }
    next += FW_WAVES;
  };
  v4f acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = v4f{0.f, 0.f, 0.f, 0.f};
  auto use = [&](const DownStep<C, STAGE>& st) {
    const v8i h = STAGE ? row_frag(stage + st.row * hstride + st.kb * 128 + g16 * 32) : st.hf;
    const float sh = STAGE ? stage_s[st.row * FB + st.kb] : st.sh;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float s = sh * st.sw[c];
      v4f q = mfma_fp8_16x16x128(weight_frag(st.b[c]), h, v4f{0.f, 0.f, 0.f, 0.f});
      asm volatile("" : "+v"(q));   // the product is the whole wave's, made before lanes part
      if (st.live) {   // other tokens take nothing, not even a NaN weight's product with 0
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[c][j] = fmaf(q[j], s, acc[c][j]);
      }
    }
  };
#pragma unroll
  for (int r = 0; r < RING; ++r) {
    load(ring[r]);
    pin_loads();
  }
  if (STAGE) {
    auto put = [&](int tile, HTile& h) {
      const int row = FB == 1 ? tile : (int)__umulhi((uint32_t)tile, inv);
      uint2 q;
      const float s = h.template quantise<POW2>(q);
      *reinterpret_cast<uint2*>(stage + row * hstride + (tile - row * FB) * 128 + (tid & 15) * 8) = q;
      if ((tid & 15) == 0) stage_s[tile] = s * P.gate[row];
    };
    // One copy of the quantisation's code for the tiles loaded early, which shift
    // down to it, and one for tiles past them.
    int tile = tid >> 4;
#pragma unroll 1
    for (int i = 0; i < EARLY && i * (FW_THREADS / 16) < tiles; ++i, tile += FW_THREADS / 16) {
      put(min(tile, tiles - 1), early[0]);   // past the last tile the last again, the same bytes
#pragma unroll
      for (int j = 0; j + 1 < EARLY; ++j) early[j] = early[j + 1];
    }
#pragma unroll 1
    for (; tile < tiles; tile += FW_THREADS / 16) {
      HTile h;
      h.load(p.h + (size_t)tile * 128 + (tid & 15) * 8);
      put(tile, h);
    }
    lds_barrier();
  }
  // `turns` steps per wave (some of the last turn's are zeros), RING at a time;
  // the rest apart: with a way out of the loop's middle the compiler would take
  // any step's loads for the latest and wait for all of them in each turn.
  const int turns = (steps - first + FW_WAVES - 1) / FW_WAVES;
  int left = turns;
  for (; left >= RING; left -= RING) {
#pragma unroll
    for (int r = 0; r < RING; ++r) {
      use(ring[r]);
      pin_loads();
      load(ring[r]);
      pin_loads();
    }
  }
#pragma unroll
  for (int r = 0; r + 1 < RING; ++r)
    if (r < left) use(ring[r]);
#pragma unroll
  for (int c = 0; c < C; ++c) red[c][wave][lane] = acc[c];
  lds_barrier();
  if (wave >= C) return;
  v4f s = red[wave][0][lane];           // wave c writes fragment c
#pragma unroll
  for (int v = 1; v < FW_WAVES; ++v) s += red[wave][v][lane];
  if (shared) {
    // Every workgroup leaves its sum, and the last to do so, whichever it is,
    // adds them in their order; nobody waits.  The sums are stored at device
    // scope, past the XCD's own cache, and the wait lets the ticket be drawn
    // only once they are there (a release fence instead writes back the whole
    // cache: 10 to 20 us a call); the reader's fence and device-scope loads see
    // to it that none comes from a cache of its own.
    float* const sums = p.sum + (size_t)(group * 64 + lane) * 4;
    const size_t stride = (size_t)groups * 256;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      __hip_atomic_store(sums + split * stride + c, s[c], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    int arrived = 0;
    if (lane == 0) arrived = __hip_atomic_fetch_add(p.ticket + group, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__builtin_amdgcn_readfirstlane(arrived) != p.splits - 1) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    s = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int v = 0; v < p.splits; ++v)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        s[c] += __hip_atomic_load(sums + v * stride + c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  const int col = c_begin + 16 * wave + 4 * g16;
  if (r16 < p.T && col < c_end) {
    const size_t at = (size_t)r16 * p.d + col;
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
  const int s_log2 = pairs <= 2 ? 3 : pairs <= 4 ? 2 : 1;
  // Reciprocals: items and steps come below 257 x 4096 + 512, and times a divisor
  // below 2^32 (or the divisor is 4096, whose reciprocal is exact), so the
  // rounding up never reaches a quotient.  A divisor of 1 (f/128, splits) is a
  // case of its own.  Made here: a division in a kernel is hundreds of bytes of code,
  // and its first fetch delays the kernel's first loads (measured: 0.15 us per
  // 128 bytes).
  auto over = [](int n) { return (uint32_t)((0x100000000ull + n - 1) / n); };
  const int splits = few_splits(d, f, k);
  char* ws = static_cast<char*>(workspace);
  FewArgs p{T, d, f, E, G, M, k, (double)route_scale, x, wg, bias, w13, w13_s, w2, w2_s, residual, idx, w, out,
            s_log2, e_log2, c_log2, E / G, keep, k / M, (65536u + E / G - 1) / (E / G), (65536u + keep - 1) / keep,
            over(f / 8), over(f / 128), over(d / 16), over(splits), reinterpret_cast<double*>(ws + L.part), reinterpret_cast<uint8_t*>(ws + L.xq),
            reinterpret_cast<float*>(ws + L.xs), reinterpret_cast<float*>(ws + L.h),
            reinterpret_cast<uint8_t*>(ws + L.hq), reinterpret_cast<float*>(ws + L.hsg),
            reinterpret_cast<FewPlan*>(ws + L.plan), reinterpret_cast<float*>(ws + L.sum),
            reinterpret_cast<int*>(ws + L.ticket), splits};
  const int KB = d / 128, FB = f / 128;
  const dim3 g1(((E + 15) / 16 << s_log2) + (T * KB + FR_THREADS / 16 - 1) / (FR_THREADS / 16)), g3((T * (k + 1) * FB + 15) / 16);
  if (pow2) hipLaunchKernelGGL(few_route_kernel<true>, g1, dim3(FR_THREADS), 0, stream, p);
  else hipLaunchKernelGGL(few_route_kernel<false>, g1, dim3(FR_THREADS), 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // no more workgroups than items (each active expert has f/8)
  const dim3 g2(std::min(256, std::min(E, T * k) * (f / 8) + f / 8));
  // Several items a turn where a workgroup may have four: a layer with one each
  // takes 14.3 us with one and 16.5 with four (tiny, T = 5), one with up to six
  // 30.1 and 28.6 (d 1024, f 512, T = 4), with nine 33.0 and 30.2 (f 2048, T = 1).
  const bool many = (std::min(E, T * k) + 1) * (f / 8) >= 4 * 256;
#define MOE_FEW_UP(NB)                                                                                                \
  do {                                                                                                                \
    if (many) hipLaunchKernelGGL((few_up_kernel<NB, few_items(NB)>), g2, dim3(FW_THREADS), 0, stream, p);             \
    else hipLaunchKernelGGL((few_up_kernel<NB, 1>), g2, dim3(FW_THREADS), 0, stream, p);                              \
  } while (0)
  switch ((KB + 7) / 8) {
    case 1: MOE_FEW_UP(1); break;
    case 2: MOE_FEW_UP(2); break;
    case 3: MOE_FEW_UP(3); break;
    case 4: MOE_FEW_UP(4); break;
    case 5: MOE_FEW_UP(5); break;
    case 6: MOE_FEW_UP(6); break;
    case 7: MOE_FEW_UP(7); break;
    default: MOE_FEW_UP(8); break;
  }
#undef MOE_FEW_UP
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int rows = T * (k + 1);
  // h in the last kernel's LDS, quantised by every workgroup for itself, or by a
  // kernel of its own, us a call at the elements of h: 13.8 against 15.3 at 640,
  // 36 against 39 at 20480 (d 2048), 76.4 against 79 at 18432 (V3, T = 1), 129
  // against 127 at 36864 (V3, T = 2), 52 against 53 and 47.3 against 47.0 at
  // 40960 (d 2048, f 1024 and 512)
  constexpr int kStaged = 32768;
  const bool stage = rows * f <= kStaged;
  static_assert(kStaged + 16 * FW_T * (FW_MAX_K + 1) + kStaged / 32 <= FW_STAGE_BYTES, "h, its row padding and scales");
  if (!stage) {
    if (pow2) hipLaunchKernelGGL(few_quant_kernel<true>, g3, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL(few_quant_kernel<false>, g3, dim3(256), 0, stream, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 g4(splits > 1 ? d / 16 * splits : std::min(256, d / 4));
#define MOE_FEW_DOWN(C, RING, STAGE, POW2) \
  hipLaunchKernelGGL((few_down_kernel<C, RING, STAGE, POW2>), g4, dim3(FW_THREADS), 0, stream, p)
  if (d > 256 * 16) {   // more than 16 columns a workgroup
    if (!stage) MOE_FEW_DOWN(2, 2, false, false);
    else if (pow2) MOE_FEW_DOWN(2, 2, true, true);
    else MOE_FEW_DOWN(2, 2, true, false);
  } else {
    if (!stage) MOE_FEW_DOWN(1, 2, false, false);
    else if (pow2) MOE_FEW_DOWN(1, 3, true, true);
    else MOE_FEW_DOWN(1, 3, true, false);
  }
#undef MOE_FEW_DOWN
  return hipGetLastError();
}

}  // namespace moe
