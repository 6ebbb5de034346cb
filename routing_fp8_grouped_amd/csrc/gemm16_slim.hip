// The forward product of include/moe_experts.h for few rows: out = act(a b^T +
// bias) + residual where a tile kernel would leave most of the chip idle.
//
// A workgroup makes a slim tile (16 MB rows, 16 NB weight rows) alone: its eight
// waves split K, and each brings its parts of both operands from memory in whole
// lines, turns them into MFMA fragments through LDS of its own (no barrier on the
// way) and joins its sums with the others' in LDS at the end.  With one row and
// N = 4096 every CU has a workgroup, and all of its waves stream: a read of the
// weights and little else.  One row, K 7168, SwiGLU of N 4096: 11 us, the launch
// among them, 5.3 TB/s; 128 rows in 64 groups of these: 418 us for up to 3.3 GB.
#include <algorithm>
#include <cmath>

#include "gemm16.h"

namespace moe {

namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kNonTemporal = 2;
constexpr uint32_t kNowhere = 0x7FFFFFF0u;   // out of every buffer's bounds: loads zeros

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(uniform_ptr(base)), 0, 0x7FFFFFE0, 0x00020000);
}

// R x 64 elements of an operand: R / 8 loads of eight whole lines each (eight
// neighbouring lanes a row).  Fragments want one row a lane; loading them in
// that layout would touch 64 lines an instruction.
template <int R, int AUX>
struct Lines {
  u32x4 v[R / 8];
  // off: byte offset of this lane's row in each eight rows; k: first element; end: of the wave's part of K
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t buffer, const uint32_t (&off)[R / 8], int k, int end,
                                       int lane) {
    const int at = k + (lane & 7) * 8;
    const bool ok = at < end;
#pragma unroll
    for (int i = 0; i < R / 8; ++i)
      v[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(buffer, ok ? off[i] + at * 2 : kNowhere, 0, AUX));
  }
  __device__ __forceinline__ void store(unsigned char* lds, int lane) const {
#pragma unroll
    for (int i = 0; i < R / 8; ++i) {
      const int r = i * 8 + (lane >> 3);
      *reinterpret_cast<u32x4*>(lds + r * 128 + (((lane & 7) ^ op_swz(r)) << 4)) = v[i];
    }
  }
};

template <class F>
__device__ __forceinline__ F fragment(const unsigned char* lds, int r, int c) {
  return *reinterpret_cast<const F*>(lds + r * 128 + ((c ^ op_swz(r)) << 4));
}

// PR: rows of a that are loaded, 16 MB or, where no tile has more, 8.
template <class E, bool GLU, int MB, int NB, int S, int PR>
__global__ __launch_bounds__(kThreads, 2) void slim_kernel(Gemm16Args p) {
  using F = typename E::frag;
  constexpr int TM = 16 * MB, TN = GLU ? 8 * NB : 16 * NB;   // rows and columns of out in a tile
  constexpr int kStage = (MB + NB) * 2048 > MB * NB * 1024 ? (MB + NB) * 2048 : MB * NB * 1024;
  __shared__ __attribute__((aligned(16))) unsigned char stage[kWaves][kStage];
  __shared__ int first[kMaxGroups + 1];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, g16 = lane >> 4, r16 = lane & 15;
  const int cols = GLU ? p.N / 2 : p.N, nt = (cols + TN - 1) / TN;
  list_tiles(p.groups, TM, first);
  const int tm = blockIdx.x / nt, n0 = (blockIdx.x - tm * nt) * TN;
  if (tm >= first[p.groups.n]) return;
  const int g = tile_group(first, p.groups.n, tm);
  const int m0 = p.groups.at(g) + (tm - first[g]) * TM, mv = min(TM, p.groups.at(g + 1) - m0);

  // this wave's part of K, whole lines
  const int each = (p.K + kWaves * 64 - 1) / (kWaves * 64) * 64;
  const int k0 = min(p.K, wave * each), end = min(p.K, k0 + each);
  const __amdgpu_buffer_rsrc_t pb = buffer_at(p.p + (size_t)m0 * p.K), qb = buffer_at(p.q + ((size_t)g * p.N + n0) * p.K);
  uint32_t po[PR / 8], qo[2 * NB];
#pragma unroll
  for (int i = 0; i < PR / 8; ++i) {
    const int r = i * 8 + (lane >> 3);
    po[i] = r < mv ? (uint32_t)r * p.K * 2 : kNowhere;
  }
#pragma unroll
  for (int i = 0; i < 2 * NB; ++i) {
    // GLU: fragment rows 0..7 are gate rows, 8..15 the same columns' up rows
    const int r = GLU ? (i >> 1) * 8 + (lane >> 3) : i * 8 + (lane >> 3);
    qo[i] = n0 + r < cols ? (uint32_t)(r + (GLU && (i & 1) ? cols : 0)) * p.K * 2 : kNowhere;
  }
  v4f acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  // S blocks of 64 k in flight in registers.  A block that has arrived goes
  // through the wave's own LDS into fragments, and its registers take the block
  // S ahead (past the end: nothing).  No other wave is waited for.
  unsigned char* lp = stage[wave];
  unsigned char* lq = lp + MB * 2048;
  Lines<PR, 0> pl[S];
  Lines<16 * NB, MB == 1 ? kNonTemporal : 0> ql[S];
#pragma unroll
  for (int b = 0; b < S; ++b) {
    ql[b].load(qb, qo, k0 + b * 64, end, lane);
    pl[b].load(pb, po, k0 + b * 64, end, lane);
  }
  for (int k = k0; k < end; k += 64 * S) {
#pragma unroll
    for (int b = 0; b < S; ++b) {
      ql[b].store(lq, lane);
      pl[b].store(lp, lane);
      ql[b].load(qb, qo, k + (S + b) * 64, end, lane);
      pl[b].load(pb, po, k + (S + b) * 64, end, lane);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        F pf[MB], qf[NB];
#pragma unroll
        for (int i = 0; i < MB; ++i) pf[i] = fragment<F>(lp, (i * 16 + r16) & (PR - 1), s * 4 + g16);
#pragma unroll
        for (int j = 0; j < NB; ++j) qf[j] = fragment<F>(lq, j * 16 + r16, s * 4 + g16);
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
          for (int j = 0; j < NB; ++j) acc[i][j] = E::mfma(qf[j], pf[i], acc[i][j]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  __syncthreads();   // the stages become the sums' place
  v4f (*part)[MB * NB][64] = reinterpret_cast<v4f (*)[MB * NB][64]>(&stage[0][0]);
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) part[wave][i * NB + j][lane] = acc[i][j];
  __syncthreads();
  uint16_t* out = static_cast<uint16_t*>(p.out);
  for (int f = wave; f < MB * NB; f += kWaves) {
    const int i = f / NB, j = f % NB;
    v4f z = part[0][f][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) z += part[w][f][lane];
    // row r, four columns of z from zn on (lanes of g16 >= 2: up columns), of out from n on
    const int r = i * 16 + r16;
    const int n = n0 + (GLU ? j * 8 + (g16 & 1) * 4 : j * 16 + g16 * 4), zn = n + (GLU && g16 >= 2 ? cols : 0);
    const bool ok = r < mv && n < cols;
    const size_t m = m0 + r;
    if (ok) {
      if (p.bias) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(p.bias + (size_t)g * p.N + zn);
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] += unpack<E>(v[e / 2], e & 1);
      }
      if (p.pre)
        *reinterpret_cast<u32x2*>(p.pre + m * p.N + zn) = u32x2{pack2<E>(z[0], z[1]), pack2<E>(z[2], z[3])};
    }
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = GLU ? glu_value(z[e], __shfl_xor(z[e], 32)) : z[e];
    if (!GLU) activate(p.act, v);
    if (ok && !(GLU && g16 >= 2)) {
      if (p.residual) {
        const u32x2 t = *reinterpret_cast<const u32x2*>(p.residual + m * cols + n);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += unpack<E>(t[e / 2], e & 1);
      }
      *reinterpret_cast<u32x2*>(out + m * cols + n) = u32x2{pack2<E>(v[0], v[1]), pack2<E>(v[2], v[3])};
    }
  }
}

template <class E, int MB, int NB, int S, int PR = 16 * MB>
void run(const Gemm16Args& p, hipStream_t stream) {
  const bool glu = p.act == kActSwiglu;
  const int cols = glu ? p.N / 2 : p.N, tn = (glu ? 8 : 16) * NB;
  // every row tile has a row
  const long row_tiles = std::min<long>(p.groups.rows, p.groups.rows / (16 * MB) + p.groups.n);
  const unsigned grid = (unsigned)(row_tiles * ((cols + tn - 1) / tn));
  if (glu) hipLaunchKernelGGL((slim_kernel<E, true, MB, NB, S, PR>), dim3(grid), dim3(kThreads), 0, stream, p);
  else hipLaunchKernelGGL((slim_kernel<E, false, MB, NB, S, PR>), dim3(grid), dim3(kThreads), 0, stream, p);
}

// Workgroups of tiles of 16 MB rows and 16 NB weight rows, about: a row tile
// more for every group that has rows.
long slim_tiles(const Gemm16Args& p, int mb, int nb) {
  const int cols = p.act == kActSwiglu ? p.N / 2 : p.N, tn = (p.act == kActSwiglu ? 8 : 16) * nb;
  const long rows = p.groups.rows, live = std::min<long>(p.groups.n, rows);
  const long m = live <= 1 ? (rows + 16 * mb - 1) / (16 * mb) : rows / (16 * mb) + live;
  return m * ((cols + tn - 1) / tn);
}

long average_rows(const Gemm16Args& p) { return (p.groups.rows + p.groups.n - 1) / p.groups.n; }

// Tiles of 16 mb rows and 16 nb weight rows, and the us of a round of 256 of them:
// about `fixed` for its start and join, `block` per 64 k.  The first stands for two
// workgroups of 1 x 1, which is what is launched (three of these fit a CU at a
// time).  128 rows, K 7168, N 4096 take 44, 32, 27 and 37 us as 2 x 1, 2 x 2, 2 x 4
// and 4 x 4; 333 x 1000 x 1016 11.5, 8.6, 8.0 and 11.1; 3468 rows, K 400, N 352 24,
// 14, 15 and 16.
struct SlimTile {
  int mb, nb;
  double fixed, block;
};
constexpr SlimTile kSlimTiles[] = {{1, 2, 1.1, 0.085}, {2, 1, 1.1, 0.08}, {2, 2, 0.8, 0.115},
                                   {2, 4, 1.8, 0.19},  {4, 2, 2.0, 0.2},  {4, 4, 2.3, 0.3}};

// The tile by that time, but up to 16 rows a group on average go to the first, whose
// weights pass the caches, whatever the others would take: right where no group has
// many more (128 rows in 64 groups of K 7168, N 4096: 418 us, all weights read once),
// and slow where some do, since these read their weights again for every 16 rows (336
// rows in 64 groups, K 3512, N 2272: 239 us; the weights' read alone is 145).
int best_tile(const Gemm16Args& p, double& least) {
  const bool few = average_rows(p) <= 16;
  int best = 0;
  for (int i = few ? 0 : 1; i < (few ? 1 : 6); ++i) {
    const SlimTile& t = kSlimTiles[i];
    const double time = (double)((slim_tiles(p, t.mb, t.nb) + 255) / 256) * (t.fixed + p.K / 64.0 * t.block);
    if (best == 0 || time < least) {
      least = time;
      best = i;
    }
  }
  return best;
}

template <class E>
void launch_slim(const Gemm16Args& p, hipStream_t stream) {
  if (p.groups.rows <= 8) return run<E, 1, 1, 2, 8>(p, stream);   // no tile has more
  double time;
  switch (best_tile(p, time)) {
    case 0: return run<E, 1, 1, 2>(p, stream);
    case 1: return run<E, 2, 1, 2>(p, stream);
    case 2: return run<E, 2, 2, 1>(p, stream);
    case 3: return run<E, 2, 4, 1>(p, stream);
    case 4: return run<E, 4, 2, 1>(p, stream);
    default: return run<E, 4, 4, 1>(p, stream);
  }
}

}  // namespace

double gemm16_slim_time(const Gemm16Args& p) {
  if ((size_t)p.N * p.K * 2 > 0x7F000000u) return INFINITY;   // a group's matrix within one buffer's bounds
  double time;
  best_tile(p, time);
  return time;
}

hipError_t launch_gemm16_slim(int type, const Gemm16Args& p, hipStream_t stream) {
  if (type == 0) launch_slim<Bf16>(p, stream);
  else launch_slim<Fp16>(p, stream);
  return hipGetLastError();
}

}  // namespace moe
