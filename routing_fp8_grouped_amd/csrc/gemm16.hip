// Grouped and dense matrix products in 16 bits (include/moe_experts.h): the
// forward z = a b^T with bias, activation and residual in the epilogue, and the
// gradients da = dz b and db = dz^T a.
//
// One tile kernel for the three.  A product is out[m][n] = sum_k P(m, k) Q(n, k)
// with P and Q either k-contiguous ([m][k] in memory) or k-strided ([k][m]):
//   forward  P = a  [rows, K]  contiguous   Q = b [N, K]   contiguous
//   dgrad    P = dz [rows, N]  contiguous   Q = b [N, K]   strided (k is N)
//   wgrad    P = dz [rows, N]  strided      Q = a [rows, K] strided (k is the group's rows)
// K advances in blocks of 64.  Both operands of a block go from memory to LDS
// by direct loads, 1 KB an instruction, through a two-stage ring.  A
// k-contiguous operand lies there as rows of 128 bytes and is read as MFMA
// fragments with ds_read_b128; a k-strided one lies as 64 k-rows and is read
// with the transposing ds_read_b64_tr_b16, so that no operand is ever
// transposed in memory.  16-byte chunks are permuted within a row (on the
// source side of the direct load) so that a read's lanes fall on different
// banks.
//
// Places past the end of K or of the rows are loads outside the buffer's
// bounds, which return zeros: no branch and no padded copy.
#include <algorithm>

#include "activation.h"
#include "groups.h"
#include "kernels.h"
#include "types16.h"

namespace moe {

namespace {

constexpr int BK = 64;

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
};

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Direct load of 16 bytes a lane from base + off to LDS address lds + 16 lane;
// lanes at kNowhere get zeros.  As with dma16 the compiler does not track it:
// a read of its data follows ring_barrier().
constexpr uint32_t kNowhere = 0x7FFFFFF0u;
__device__ __forceinline__ i32x4 bounded(const void* base) {
  const uint64_t v = reinterpret_cast<uint64_t>(base);
  return i32x4{(int)__builtin_amdgcn_readfirstlane((uint32_t)v),
               (int)(__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32)) & 0xFFFFu), 0x7FFFFFE0, 0x00020000};
}
__device__ __forceinline__ void dma16_bounded(i32x4 buffer, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :: "v"(off), "s"(buffer), "s"(__builtin_amdgcn_readfirstlane(lds))
               : "memory");
}

// Chunk position of a k-strided operand's k-row: the four k-rows that 16 lanes
// of a transposing read touch, and the other four of the next 16 lanes, lie in
// eight different 32-byte places of 256 bytes.
__device__ __forceinline__ int tr_swz(int k) { return ((k & 3) | ((k >> 1) & 4)) << 1; }

// One operand's [R x 64] block of a tile.
template <int R, bool TR, int NW>
struct Operand {
  static constexpr int kBytes = R * BK * 2;
  static constexpr int kLoads = kBytes / 1024 / NW;   // direct loads of a wave
  static_assert(kLoads * 1024 * NW == kBytes, "whole loads");

  const uint16_t* base;     // first element of the tile, k = 0
  size_t step;              // elements from one K block to the next
  uint32_t off[kLoads];     // per-lane byte offsets

  // r0: first row of the tile in the operand (its column if k-strided); valid:
  // rows (columns) there are; ld: elements of a memory row
  __device__ __forceinline__ void start(const uint16_t* mem, size_t row0, int col0, int valid, size_t ld, int wave,
                                        int lane) {
    base = mem + row0 * ld + col0;
    step = TR ? BK * ld : BK;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int byte = (wave * kLoads + i) * 1024 + lane * 16;
      if (TR) {
        const int k = byte / (R * 2), c = ((byte % (R * 2)) >> 4) ^ tr_swz(k);
        off[i] = c * 8 < valid ? (uint32_t)(k * ld * 2) + c * 16 : kNowhere;
      } else {
        const int r = byte >> 7, c = ((byte >> 4) & 7) ^ op_swz(r);
        off[i] = r < valid ? (uint32_t)(r * ld * 2) + c * 16 : kNowhere;
      }
    }
  }
  // K block kb into `lds`; left: elements of K from this block on
  __device__ __forceinline__ void issue(int kb, int left, uint32_t lds, int wave, int lane) const {
    const i32x4 buffer = bounded(base + (size_t)kb * step);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      uint32_t o = off[i];
      if (left < BK) {
        const int byte = (wave * kLoads + i) * 1024 + lane * 16;
        const int k = TR ? byte / (R * 2) : (((byte >> 4) & 7) ^ op_swz(byte >> 7)) * 8;
        if (k >= left) o = kNowhere;
      }
      dma16_bounded(buffer, o, lds + (wave * kLoads + i) * 1024);
    }
  }
  // MFMA fragment of rows r0 .. r0+15, k in [32 s, 32 s + 32)
  template <class F>
  static __device__ __forceinline__ F frag(const unsigned char* lds, int r0, int s, int lane) {
    const int g = lane >> 4, i = lane & 15;
    if constexpr (TR) {
      typedef short v4s __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) v4s lds_v4s;
      const int k = s * 32 + g * 8 + (i >> 2);
      const int c = (r0 >> 3) + ((i >> 1) & 1), h = (i & 1) * 8;
      const uint32_t at = lds_addr(lds);
      const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_v4s*)(uintptr_t)(at + k * (R * 2) + ((c ^ tr_swz(k)) << 4) + h));
      const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_v4s*)(uintptr_t)(at + (k + 4) * (R * 2) + ((c ^ tr_swz(k + 4)) << 4) + h));
      typedef short v8s __attribute__((ext_vector_type(8)));
      return __builtin_bit_cast(F, v8s{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
    } else {
      const int r = r0 + i;
      return *reinterpret_cast<const F*>(lds + r * 128 + (((s * 4 + g) ^ op_swz(r)) << 4));
    }
  }
};

enum Kind { kForward = 0, kForwardGlu = 1, kDgrad = 2, kWgrad = 3 };

// Eight neighbouring columns of a lane from two sub-tiles' accumulators: lanes
// 16 apart trade halves.  They belong to column 16 (g & 1) + 8 (g >> 1) of the
// pair's 32, g = lane / 16.
__device__ __forceinline__ void columns8(const v4f a, const v4f b, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(a[e]), __float_as_uint(b[e]), false, false);
    f[e] = __uint_as_float(x[0]);
    f[4 + e] = __uint_as_float(x[1]);
  }
}

__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case kActRelu: return act_value<kActRelu>(z);
    case kActSilu: return act_value<kActSilu>(z);
    case kActGelu: return act_value<kActGelu>(z);
    default: return z;
  }
}

template <class E, int KIND, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64, 1) void gemm16_kernel(Gemm16Args p) {
  constexpr int NW = WM * WN, MS = BM / WM / 16, NS = BN / WN / 16;
  constexpr bool GLU = KIND == kForwardGlu;
  using F = typename E::frag;
  using P = Operand<BM, KIND == kWgrad, NW>;
  using Q = Operand<BN, KIND == kDgrad || KIND == kWgrad, NW>;
  constexpr int STG = P::kBytes + Q::kBytes;
  __shared__ __attribute__((aligned(1024))) unsigned char sm[2 * STG];
  __shared__ int first[KIND == kWgrad ? 1 : kMaxGroups + 1];

  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int wm = wave / WN, wn = wave % WN;
  const int g16 = lane >> 4, r16 = lane & 15;
  const int cols = GLU ? p.N / 2 : p.N;            // columns of out
  constexpr int TN = GLU ? BN / 2 : BN;            // columns of out in a tile
  const int nt = (cols + TN - 1) / TN, mt = (p.M + BM - 1) / BM;
  int total;
  if constexpr (KIND == kWgrad) {
    total = p.groups.n * mt * nt;
  } else {
    list_tiles(p.groups, BM, first);
    total = first[p.groups.n] * nt;
  }
  for (int L = blockIdx.x; L < total; L += gridDim.x) {
    // ---- the tile ----
    int g, m0, mv, n0;
    int kext;
    size_t row0;
    if constexpr (KIND == kWgrad) {
      g = L / (mt * nt);
      const int rem = L - g * mt * nt;
      m0 = rem / nt * BM;
      n0 = rem % nt * BN;
      mv = min(BM, p.M - m0);
      row0 = p.groups.at(g);
      kext = p.groups.count(g);
    } else {
      const int tm = L / nt;
      g = tile_group(first, p.groups.n, tm);
      const int at = p.groups.at(g);
      m0 = at + (tm - first[g]) * BM;
      n0 = (L - tm * nt) * TN;
      mv = min(BM, p.groups.at(g + 1) - m0);
      row0 = 0;
      kext = p.K;
    }
    P pl;
    Q ql;
    if constexpr (KIND == kWgrad) {
      pl.start(p.p, row0, m0, mv, p.M, wave, lane);
      ql.start(p.q, row0, n0, p.N - n0, p.N, wave, lane);
    } else {
      pl.start(p.p, m0, 0, mv, p.K, wave, lane);
      const uint16_t* b = p.q + (size_t)g * p.N * p.K;
      if constexpr (KIND == kDgrad) ql.start(b, 0, n0, p.N - n0, p.N, wave, lane);
      else if constexpr (!GLU) ql.start(b, n0, 0, p.N - n0, p.K, wave, lane);
      else {
        // the first half of the tile's rows are gate rows, the second the same
        // columns' up rows; each wave loads rows of one half
        const int h = wave >= NW / 2;
        ql.start(b, n0 + (size_t)h * (cols - BN / 2), 0, min(BN, cols - n0 + h * (BN / 2)), p.K, wave, lane);
      }
    }
    v4f acc[MS][NS];
#pragma unroll
    for (int ms = 0; ms < MS; ++ms)
#pragma unroll
      for (int ns = 0; ns < NS; ++ns) acc[ms][ns] = v4f{0.f, 0.f, 0.f, 0.f};
    const int KB = (kext + BK - 1) / BK;
    __syncthreads();   // the last tile's reads are done
    auto issue = [&](int kb) {
      const uint32_t s = lds_addr(sm + (kb & 1) * STG);
      pl.issue(kb, kext - kb * BK, s, wave, lane);
      ql.issue(kb, kext - kb * BK, s + P::kBytes, wave, lane);
    };
    if (KB > 0) issue(0);
    for (int kb = 0; kb < KB; ++kb) {
      ring_barrier();
      if (kb + 1 < KB) issue(kb + 1);
      const unsigned char* ps = sm + (kb & 1) * STG;
      const unsigned char* qs = ps + P::kBytes;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        F pf[MS];
#pragma unroll
        for (int ms = 0; ms < MS; ++ms) pf[ms] = P::template frag<F>(ps, wm * MS * 16 + ms * 16, s, lane);
#pragma unroll
        for (int ns = 0; ns < NS; ++ns) {
          const int r = GLU ? (ns < NS / 2 ? 0 : BN / 2) + wn * (NS / 2) * 16 + (ns % (NS / 2)) * 16 : (wn * NS + ns) * 16;
          const F qf = Q::template frag<F>(qs, r, s, lane);
#pragma unroll
          for (int ms = 0; ms < MS; ++ms) acc[ms][ns] = E::mfma(qf, pf[ms], acc[ms][ns]);
        }
      }
    }
    // ---- epilogue: lane (g16, r16) holds row ms*16 + r16, columns ns*16 + 4*g16 .. +3 ----
    const int lc = (g16 & 1) * 16 + (g16 >> 1) * 8;
    if constexpr (KIND == kWgrad) {
      float* out = static_cast<float*>(p.out) + (size_t)g * p.M * p.N;
#pragma unroll
      for (int ms = 0; ms < MS; ++ms) {
        const int m = m0 + wm * MS * 16 + ms * 16 + r16;
#pragma unroll
        for (int ns = 0; ns < NS; ++ns) {
          const int n = n0 + (wn * NS + ns) * 16 + 4 * g16;
          if (m < p.M && n < p.N) *reinterpret_cast<v4f*>(out + (size_t)m * p.N + n) = acc[ms][ns];
        }
      }
    } else {
      uint16_t* out = static_cast<uint16_t*>(p.out);
      constexpr int NP = GLU ? NS / 2 : NS;
#pragma unroll
      for (int ns = 0; ns < NP; ns += 2) {
        const int n = n0 + (wn * NP + ns) * 16 + lc;
        Values<E, true> bg, bu;
        if (p.bias && n < cols) {
          bg = Values<E, true>(load_chunk(p.bias + (size_t)g * p.N + n));
          if (GLU) bu = Values<E, true>(load_chunk(p.bias + (size_t)g * p.N + cols + n));
        }
#pragma unroll
        for (int ms = 0; ms < MS; ++ms) {
          const int r = wm * MS * 16 + ms * 16 + r16;
          const size_t m = m0 + r;
          Values<E, true> z, u;
          columns8(acc[ms][ns], acc[ms][ns + 1], z.v);
          if constexpr (GLU) columns8(acc[ms][NP + ns], acc[ms][NP + ns + 1], u.v);
          if (r >= mv || n >= cols) continue;
#pragma unroll
          for (int e = 0; e < 8; ++e) z.v[e] += bg.v[e];
          if (GLU)
#pragma unroll
            for (int e = 0; e < 8; ++e) u.v[e] += bu.v[e];
          if (p.pre) {
            z.put(p.pre + m * p.N + n);
            if (GLU) u.put(p.pre + m * p.N + cols + n);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) z.v[e] = GLU ? swiglu_f32(z.v[e], u.v[e]) : activate(p.act, z.v[e]);
          if (p.residual) {
            const Values<E, true> res(load_chunk(p.residual + m * cols + n));
#pragma unroll
            for (int e = 0; e < 8; ++e) z.v[e] += res.v[e];
          }
          z.put(out + m * cols + n);
        }
      }
    }
  }
}

template <int KIND>
hipError_t launch(int type, const Gemm16Args& p, long tiles_bound, hipStream_t stream) {
  const unsigned grid = (unsigned)std::min(tiles_bound, 512L);
  if (type == 0) hipLaunchKernelGGL((gemm16_kernel<Bf16, KIND, 128, 128, 2, 2>), dim3(grid), dim3(256), 0, stream, p);
  else hipLaunchKernelGGL((gemm16_kernel<Fp16, KIND, 128, 128, 2, 2>), dim3(grid), dim3(256), 0, stream, p);
  return hipGetLastError();
}

long tiles(long rows, int n_groups, int cols, int tn) { return (rows / 128 + n_groups) * ((cols + tn - 1) / tn); }

}  // namespace

hipError_t launch_gemm16(int type, const void* a, const int32_t* offsets, int n_groups, int rows, int K, int N,
                         const void* b, const void* bias, int act, const void* residual, void* pre, void* out,
                         void* workspace, hipStream_t stream) {
  (void)workspace;
  Gemm16Args p{};
  p.p = static_cast<const uint16_t*>(a);
  p.q = static_cast<const uint16_t*>(b);
  p.groups = Groups{offsets, n_groups, rows};
  p.N = N;
  p.K = K;
  p.bias = static_cast<const uint16_t*>(bias);
  p.residual = static_cast<const uint16_t*>(residual);
  p.pre = static_cast<uint16_t*>(pre);
  p.out = out;
  p.act = act;
  if (act == kActSwiglu) return launch<kForwardGlu>(type, p, tiles(rows, n_groups, N / 2, 64), stream);
  return launch<kForward>(type, p, tiles(rows, n_groups, N, 128), stream);
}

hipError_t launch_gemm16_dgrad(int type, const void* dz, const int32_t* offsets, int n_groups, int rows, int K, int N,
                               const void* b, const void* residual, void* da, void* workspace, hipStream_t stream) {
  (void)workspace;
  Gemm16Args p{};
  p.p = static_cast<const uint16_t*>(dz);
  p.q = static_cast<const uint16_t*>(b);
  p.groups = Groups{offsets, n_groups, rows};
  p.N = K;
  p.K = N;
  p.residual = static_cast<const uint16_t*>(residual);
  p.out = da;
  return launch<kDgrad>(type, p, tiles(rows, n_groups, K, 128), stream);
}

hipError_t launch_gemm16_wgrad(int type, const void* dz, const void* a, const int32_t* offsets, int n_groups, int rows,
                               int K, int N, float* db, void* workspace, hipStream_t stream) {
  (void)workspace;
  Gemm16Args p{};
  p.p = static_cast<const uint16_t*>(dz);
  p.q = static_cast<const uint16_t*>(a);
  p.groups = Groups{offsets, n_groups, rows};
  p.M = N;
  p.N = K;
  p.out = db;
  return launch<kWgrad>(type, p, (long)n_groups * ((N + 127) / 128) * ((K + 127) / 128), stream);
}

size_t gemm16_workspace_bytes(int, int, int, int, int) { return 0; }
size_t gemm16_backward_workspace_bytes(int, int, int, int) { return 0; }

}  // namespace moe
