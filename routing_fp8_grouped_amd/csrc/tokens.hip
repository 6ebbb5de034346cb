// Tokens sorted by expert and back (include/moe_experts.h): the stable sort of
// the slots, and four copies between the tokens' and the sorted order,
//   dispatch           out[pos[s]] = w[s] x[t]
//   its backward       dx[t] = sum_j w[s] drows[pos[s]] + residual[t],  dw[s] = <x[t], drows[pos[s]]>
//   collect            out[t] = sum_j w[s] y[pos[s]] + residual[t]
//   its backward       dy[pos[s]] = w[s] dout[t],  dw[s] = <dout[t], y[pos[s]]>
// which are two kernels: a token's row spread over its k rows, and k rows
// summed into the token's; either may take the k products' sums with another
// tensor along.  A token belongs to one team of threads (a workgroup, or part
// of a wave for narrow rows), so its row is read or written once, every row of
// the sorted order once, sums have one order, and nothing is atomic.  Bound by
// HBM: 16384 tokens of 7168 BF16 to eight experts each, sorted, dispatched and
// collected, move 4.2 GB in 792 us, 5.3 TB/s; few tokens by the launches.
#include <algorithm>

#include "kernels.h"
#include "types16.h"

namespace moe {

namespace {

// ---- sort ----
// Block b takes slots [b C, b C + C), each of its waves an equal part of them
// in order.  A first kernel counts every block's slots per expert; the second
// adds up all blocks' counts for itself (a few hundred KB from the caches,
// cheaper than a kernel of its own in between) and ranks its slots: the lanes
// of a wave that hold the same expert find each other by one ballot per bit of
// the expert's number, a slot's rank is its place among them, and the wave's
// running base of each expert lives in LDS.  A batch that fits one block is
// sorted by the second kernel alone.
constexpr int kSortMaxBlocks = 256;
constexpr int kSortOneBlock = 4096;   // slots of a batch sorted by one workgroup
constexpr int kSortThreads = 256, kSortThreadsOne = 1024;

int sort_chunk(long S) {
  const long c = (S + kSortMaxBlocks - 1) / kSortMaxBlocks;
  return (int)std::max(1024L, (c + 255) / 256 * 256);
}
int sort_blocks(long S) { return S <= kSortOneBlock ? 1 : (int)((S + sort_chunk(S) - 1) / sort_chunk(S)); }

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const int32_t* __restrict__ idx, int S, int E, int C,
                                                                  int32_t* __restrict__ counts) {
  extern __shared__ int cnt[];
  for (int e = threadIdx.x; e < E; e += kSortThreads) cnt[e] = 0;
  __syncthreads();
  const int lo = blockIdx.x * C, hi = min(S, lo + C);
  for (int s = lo + (int)threadIdx.x; s < hi; s += kSortThreads) {
    const uint32_t e = (uint32_t)idx[s];
    if (e < (uint32_t)E) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) counts[(size_t)blockIdx.x * E + e] = cnt[e];
}

template <int NT>
__global__ __launch_bounds__(NT) void sort_kernel(const int32_t* __restrict__ idx, int S, int E, int bits, int C,
                                                  const int32_t* __restrict__ counts, int nb,
                                                  int32_t* __restrict__ offsets, int32_t* __restrict__ pos,
                                                  int32_t* __restrict__ row_slot) {
  constexpr int NW = NT / 64;
  extern __shared__ int base[];   // [NW][E]: counts, then the next row of each wave's slots
  __shared__ int wave_tot[NW];
  __shared__ int s_live;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lo = blockIdx.x * C, hi = min(S, lo + C);
  const int part = C / NW;   // a multiple of 64 or C itself padded by the bounds below
  const int w0 = min(hi, lo + wave * part), w1 = min(hi, w0 + part);
  for (int i = tid; i < NW * E; i += NT) base[i] = 0;
  __syncthreads();
  for (int s = w0 + lane; s < w1; s += 64) {
    const uint32_t e = (uint32_t)idx[s];
    if (e < (uint32_t)E) atomicAdd(&base[wave * E + e], 1);
  }
  __syncthreads();
  // first rows: experts before, blocks before, waves before
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += NT) {
    const int e = e0 + tid;
    int total = 0, before = 0;
    if (e < E) {
      if (nb > 1) {
#pragma unroll 16
        for (int b = 0; b < nb; ++b) {
          const int c = counts[(size_t)b * E + e];
          total += c;
          before += b < (int)blockIdx.x ? c : 0;
        }
      } else {
        for (int w = 0; w < NW; ++w) total += base[w * E + e];
      }
    }
    int v = total;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(v, o);
      if (lane >= o) v += u;
    }
    if (lane == 63) wave_tot[wave] = v;
    __syncthreads();
    int at = carry + v - total;
    for (int w = 0; w < NW; ++w) {
      if (w < wave) at += wave_tot[w];
      carry += wave_tot[w];
    }
    if (e < E) {
      if (blockIdx.x == 0) offsets[e] = at;
      at += before;
      for (int w = 0; w < NW; ++w) {
        const int c = base[w * E + e];
        base[w * E + e] = at;
        at += c;
      }
    }
    __syncthreads();
  }
  if (tid == 0) {
    s_live = carry;
    if (blockIdx.x == 0) offsets[E] = carry;
  }
  __syncthreads();
  const int live = s_live;
  const uint64_t below = (uint64_t(1) << lane) - 1;
  for (int s0 = w0; s0 < w1; s0 += 64) {
    const int s = s0 + lane;
    const int id = s < w1 ? idx[s] : -1;
    const bool ok = (uint32_t)id < (uint32_t)E;
    uint64_t same = __ballot(ok);
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = __ballot((id >> b) & 1);
      same &= (id >> b) & 1 ? m : ~m;
    }
    int p = -1;
    if (ok) p = base[wave * E + id] + __popcll(same & below);
    // every lane has read the bases before the last of each expert moves them
    __builtin_amdgcn_wave_barrier();
    if (ok && (same & ~below & ~(uint64_t(1) << lane)) == 0) base[wave * E + id] = p + 1;
    __builtin_amdgcn_wave_barrier();
    if (s < w1) pos[s] = p;
    if (ok) row_slot[p] = s;
  }
  // rows that no slot has
  for (int r = max(lo, live) + tid; r < hi; r += NT) row_slot[r] = -1;
}

// ---- copies ----

struct CopyArgs {
  const void* tok;       // token-ordered input: what is spread, or the products' other operand
  const void* rows_in;   // row-ordered input: what is summed, or the products' other operand (may be `out` then)
  const void* add;       // sum: token-ordered residual (may be `out`), or NULL
  const int32_t* pos;
  const float* w;        // or NULL
  void* out;
  float* dots;           // [T, k]
  int T, k, d, rows;
};

// KB of a token's slots from slot j0 on.  A slot without a row reads row 0 in
// its place and selects zeros: no branch stands between the loads.
template <int KB>
struct Slots {
  int row[KB];
  float w[KB];
  bool ok[KB];
  __device__ __forceinline__ Slots(const CopyArgs& p, int t, int j0) {
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      const size_t s = (size_t)t * p.k + min(j0 + j, p.k - 1);
      const uint32_t r = (uint32_t)p.pos[s];
      ok[j] = j0 + j < p.k && r < (uint32_t)p.rows;
      row[j] = ok[j] ? (int)r : 0;
      w[j] = p.w ? p.w[s] : 1.0f;
    }
  }
};

// Adds the slots' rows at element `at` to acc, or their products with x to dot,
// or both.
template <class E, bool WHOLE, bool SUM, bool DOTS, bool PAST, int KB>
__device__ __forceinline__ void take(const CopyArgs& p, const Slots<KB>& s, const typename E::storage* x, int at,
                                     Values<E, WHOLE>& acc, float (&dot)[KB]) {
  using S = typename E::storage;
  using Val = Values<E, WHOLE>;
  typename Val::raw r[KB], xr{};
#pragma unroll
  for (int j = 0; j < KB; ++j) r[j] = Val::template fetch<PAST>(static_cast<const S*>(p.rows_in) + (size_t)s.row[j] * p.d + at);
  if (DOTS) xr = Val::fetch(x + at);
  const Val xv(xr);
#pragma unroll
  for (int j = 0; j < KB; ++j) {
    const Val v(r[j]);
#pragma unroll
    for (int i = 0; i < Val::n; ++i) {
      if (SUM) acc.v[i] = s.ok[j] ? fmaf(s.w[j], v.v[i], acc.v[i]) : acc.v[i];
      if (DOTS) dot[j] = fmaf(xv.v[i], v.v[i], dot[j]);
    }
  }
}

// The products' sums over a team: a workgroup (BLOCK) or `team` neighbouring
// lanes of a wave.
template <bool BLOCK, int KB>
__device__ __forceinline__ void store_dots(float (&dot)[KB], const Slots<KB>& s, int team, int lane, float* out, int n) {
  __shared__ float part[BLOCK ? 8 : 1][KB];
#pragma unroll
  for (int j = 0; j < KB; ++j) {
    dot[j] = s.ok[j] ? dot[j] : 0.0f;
    for (int o = BLOCK ? 32 : team / 2; o > 0; o >>= 1) dot[j] += __shfl_xor(dot[j], o);
  }
  if constexpr (BLOCK) {
    const int nw = blockDim.x >> 6;
    if ((lane & 63) == 0)
#pragma unroll
      for (int j = 0; j < KB; ++j) part[lane >> 6][j] = dot[j];
    __syncthreads();
    if (lane < n) {
      float v = 0.0f;
      for (int w = 0; w < nw; ++w) v += part[w][lane];
      out[lane] = v;
    }
    __syncthreads();
  } else if (lane == 0) {
#pragma unroll
    for (int j = 0; j < KB; ++j)
      if (j < n) out[j] = dot[j];
  }
}

// SUM: token row = sum of w * rows + residual.  Otherwise: rows of the token's
// slots = w * token row.  MANY: more than KB slots, KB at a time.
template <class E, bool SUM, bool DOTS, bool BLOCK, bool PAST, bool MANY, int KB>
__global__ __launch_bounds__(512) void copy_kernel(CopyArgs p, int team) {
  using S = typename E::storage;
  const int lane = BLOCK ? threadIdx.x : threadIdx.x & (team - 1);
  const int stride = BLOCK ? blockDim.x : team;
  const int64_t token = BLOCK ? workgroup() : workgroup() * (256u / (unsigned)team) + threadIdx.x / (unsigned)team;
  if (token >= p.T) return;   // whole teams
  const int t = (int)token;
  const size_t d = p.d;
  const S* tok = static_cast<const S*>(p.tok) + (size_t)t * d;
  const S* add = static_cast<const S*>(p.add) + (size_t)t * d;
  S* out = static_cast<S*>(p.out);
  // fn(element, whole chunk?) over the token's row: chunks, then the elements behind the last whole one
  auto each = [&](auto fn) {
    const int full = p.d / E::kWidth;
    for (int c = lane; c < full; c += stride) fn(c * E::kWidth, std::true_type{});
    if (lane < p.d - full * E::kWidth) fn(full * E::kWidth + lane, std::false_type{});
  };
  if constexpr (SUM) {
    const Slots<KB> s(p, t, 0);
    float dot[KB] = {};
    each([&](int at, auto whole) {
      using Val = Values<E, decltype(whole)::value>;
      typename Val::raw ar{};
      if (p.add) ar = Val::template fetch<PAST>(add + at);
      Val acc;
      take<E, decltype(whole)::value, true, DOTS && !MANY, PAST, KB>(p, s, tok, at, acc, dot);
      if constexpr (MANY)
        for (int j0 = KB; j0 < p.k; j0 += KB)
          take<E, decltype(whole)::value, true, false, PAST, KB>(p, Slots<KB>(p, t, j0), tok, at, acc, dot);
      if (p.add) {
        const Val a(ar);
#pragma unroll
        for (int i = 0; i < Val::n; ++i) acc.v[i] += a.v[i];
      }
      acc.template put<PAST>(out + t * d + at);
    });
    if constexpr (DOTS && !MANY) store_dots<BLOCK, KB>(dot, s, team, lane, p.dots + (size_t)t * p.k, p.k);
  }
  if constexpr (!SUM || (DOTS && MANY)) {
    for (int j0 = 0; j0 < p.k; j0 += KB) {
      const Slots<KB> s(p, t, j0);
      float dot[KB] = {};
      each([&](int at, auto whole) {
        using Val = Values<E, decltype(whole)::value>;
        if constexpr (DOTS) {
          Val none;
          take<E, decltype(whole)::value, false, true, PAST, KB>(p, s, tok, at, none, dot);
        }
        if constexpr (!SUM) {
          const Val x(Val::fetch(tok + at));
#pragma unroll
          for (int j = 0; j < KB; ++j) {
            Val o;
#pragma unroll
            for (int i = 0; i < Val::n; ++i) o.v[i] = s.w[j] * x.v[i];
            if (s.ok[j]) o.template put<PAST>(out + s.row[j] * d + at);
          }
        }
      });
      if constexpr (DOTS) store_dots<BLOCK, KB>(dot, s, team, lane, p.dots + (size_t)t * p.k + j0, min(KB, p.k - j0));
      if (!MANY) break;
    }
  }
}

// Threads of a token with n chunks: a part of a wave for narrow rows, else the
// workgroup of 128 to 512 threads that leaves the fewest idle in its last turn.
int team_of(int n) {
  if (n <= 128) return n <= 16 ? 16 : n <= 32 ? 32 : 64;
  int best = 128;
  for (int nt = 192; nt <= 512; nt += 64)
    if ((n + nt - 1) / nt * nt <= (n + best - 1) / best * best) best = nt;
  return best;
}

template <class E, bool SUM, bool DOTS, bool MANY, int KB>
void run_copy(const CopyArgs& p, hipStream_t stream) {
  const int team = team_of((p.d - 1) / E::kWidth + 1);
  // Wide rows that are more than the last-level cache holds go past it (V3 rows of
  // 16384 tokens there and back: 853 -> 809 us; of 4099 tokens of 2052: 67.6 -> 65.9).
  const size_t row = (size_t)p.d * sizeof(typename E::storage);
  const bool past = row * p.T * (1 + (size_t)p.k * (DOTS && !SUM ? 2 : 1)) > kCacheBytes / 2;
  auto go = [&](auto block, auto stream_past) {
    constexpr bool BLOCK = decltype(block)::value;
    hipLaunchKernelGGL((copy_kernel<E, SUM, DOTS, BLOCK, decltype(stream_past)::value, MANY, KB>),
                       grid_of(BLOCK ? p.T : ((int64_t)p.T + 256 / team - 1) / (256 / team)), dim3(BLOCK ? team : 256), 0, stream, p,
                       team);
  };
  using Yes = std::true_type;
  using No = std::false_type;
  if (team <= 64) go(No{}, No{});
  else if (past) go(Yes{}, Yes{});
  else go(Yes{}, No{});
}

template <class E, bool SUM, bool DOTS>
void run_copy_k(const CopyArgs& p, hipStream_t stream) {
  if (p.k == 1) run_copy<E, SUM, DOTS, false, 1>(p, stream);
  else if (p.k == 2) run_copy<E, SUM, DOTS, false, 2>(p, stream);
  else if (p.k <= 4) run_copy<E, SUM, DOTS, false, 4>(p, stream);
  else if (p.k <= 6) run_copy<E, SUM, DOTS, false, 6>(p, stream);
  else if (p.k <= 8) run_copy<E, SUM, DOTS, false, 8>(p, stream);
  else run_copy<E, SUM, DOTS, true, 8>(p, stream);
}

template <bool SUM>
hipError_t launch_copy(int type, const CopyArgs& p, hipStream_t stream) {
  const bool dots = p.dots != nullptr;
  if (type == 0) dots ? run_copy_k<Bf16, SUM, true>(p, stream) : run_copy_k<Bf16, SUM, false>(p, stream);
  else if (type == 1) dots ? run_copy_k<Fp16, SUM, true>(p, stream) : run_copy_k<Fp16, SUM, false>(p, stream);
  else dots ? run_copy_k<Fp32, SUM, true>(p, stream) : run_copy_k<Fp32, SUM, false>(p, stream);
  return hipGetLastError();
}

}  // namespace

size_t sort_workspace_bytes(int T, int k, int E) {
  const int nb = sort_blocks((long)T * k);
  return nb == 1 ? 0 : (size_t)nb * E * sizeof(int32_t);
}

hipError_t launch_sort(const int32_t* idx, int T, int k, int E, int32_t* offsets, int32_t* pos, int32_t* row_slot,
                       int32_t* counts, hipStream_t stream) {
  const int S = T * k, nb = sort_blocks(S);
  int bits = 0;
  while ((1 << bits) < E) ++bits;
  if (nb == 1) {
    const int C = (std::max(S, 1) + kSortThreadsOne - 1) / kSortThreadsOne * kSortThreadsOne;
    hipLaunchKernelGGL(sort_kernel<kSortThreadsOne>, dim3(1), dim3(kSortThreadsOne),
                       (size_t)E * (kSortThreadsOne / 64) * 4, stream, idx, S, E, bits, C, counts, 1, offsets, pos,
                       row_slot);
    return hipGetLastError();
  }
  const int C = sort_chunk(S);
  hipLaunchKernelGGL(sort_count_kernel, dim3(nb), dim3(kSortThreads), (size_t)E * 4, stream, idx, S, E, C, counts);
  hipLaunchKernelGGL(sort_kernel<kSortThreads>, dim3(nb), dim3(kSortThreads), (size_t)E * (kSortThreads / 64) * 4,
                     stream, idx, S, E, bits, C, counts, nb, offsets, pos, row_slot);
  return hipGetLastError();
}

hipError_t launch_spread(int type, const void* x, const int32_t* pos, const float* w, const void* y, int T, int k, int d,
                         int rows, void* out, float* dots, hipStream_t stream) {
  // a slot without a row reads row 0 in its place: without any row, the token's
  return launch_copy<false>(type, CopyArgs{x, rows ? y : x, nullptr, pos, w, out, dots, T, k, d, rows}, stream);
}

hipError_t launch_sum(int type, const void* rows_in, const int32_t* pos, const float* w, const void* x,
                      const void* residual, int T, int k, int d, int rows, void* out, float* dots, hipStream_t stream) {
  return launch_copy<true>(type, CopyArgs{x, rows ? rows_in : out, residual, pos, w, out, dots, T, k, d, rows}, stream);
}

}  // namespace moe
