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
// What bounds it is the feeding of the matrix units: 8192 cubed takes 795 us
// (1380 TFLOP/s; the library's product reaches 1580 to 1610), 596 of them MFMA
// alone and 666 without the loads from memory; 16384 rows, K 7168, SwiGLU of N 4096
// 725 (1330 TFLOP/s).
//
// Places past the end of K or of the rows are loads outside the buffer's
// bounds, which return zeros: no branch and no padded copy.
#include <algorithm>
#include <cmath>

#include "gemm16.h"

namespace moe {

namespace {

constexpr int BK = 64;
constexpr int SUPER = 4;   // row tiles of a super-block; 1 and 8 are slower

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Direct load of 16 bytes a lane from the buffer's byte off to LDS address lds +
// 16 lane; lanes whose off is not below the buffer's size get zeros.  As with
// dma16 the compiler does not track it: a read of its data follows
// ring_barrier().
constexpr uint32_t kNowhere = 0x7FFFFFF0u;
__device__ __forceinline__ void dma16_bounded(i32x4 buffer, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :: "v"(off), "s"(buffer), "s"(lds)
               : "memory");
}
__device__ __forceinline__ i32x4 buffer_of(uint64_t base, uint32_t bytes) {
  return i32x4{(int)__builtin_amdgcn_readfirstlane((uint32_t)base),
               (int)(__builtin_amdgcn_readfirstlane((uint32_t)(base >> 32)) & 0xFFFFu),
               (int)__builtin_amdgcn_readfirstlane(bytes), 0x00020000};
}

// Chunk position of a k-strided operand's k-row: the four k-rows that 16 lanes
// of a transposing read touch, and the other four of the next 16 lanes, lie in
// eight different 32-byte places of 256 bytes.
__device__ __forceinline__ int tr_swz(int k) { return ((k & 3) | ((k >> 1) & 4)) << 1; }

// One operand's [R x 64] block of a tile.  Each wave makes kLoads of its 1 KB
// loads: load q is rows 8 q .. 8 q + 7 (k-contiguous) or kRows k-rows from
// kRows q on.
//
// What lies outside: rows past the tile's last are out of the buffer's bounds
// (zeros); k-rows past K too.  k past K in a k-contiguous row is masked.
// Columns past the last of a k-strided operand are the next k-row's: they only
// reach results that are not stored.
template <int R, bool TR, int NW>
struct Operand {
  static constexpr int kBytes = R * BK * 2;
  static constexpr int kLoads = kBytes / 1024 / NW;
  static constexpr int kRows = TR ? 512 / R : 8;
  static_assert(kLoads * 1024 * NW == kBytes, "whole loads");

  uint64_t base;           // of the next K block to load
  uint32_t bytes, step;    // of the buffer from base on; from one block to the next
  int64_t row_bytes;       // of a memory row
  int cut;                 // k-strided: bytes of base past the start of its row
  uint32_t off[kLoads];    // the lane's bytes from base on
  uint32_t lds;            // the wave's first load within a block in LDS
  uint32_t k_lane;         // k-contiguous: first byte of the lane's k within a block

  // mem: the tile's first row (k-row) and column; col0: that column; valid: rows
  // there are (k-contiguous); load: the wave's first one in memory
  __device__ __forceinline__ void start(const uint16_t* mem, int col0, int64_t valid, int64_t ld, int lds_load,
                                        int load, int lane) {
    base = reinterpret_cast<uint64_t>(mem);
    row_bytes = ld * 2;
    bytes = TR ? 0u : (uint32_t)min(valid * row_bytes, (int64_t)0x7FF00000);
    step = TR ? (uint32_t)(BK * row_bytes) : BK * 2;
    cut = col0 * 2;
    lds = lds_load * 1024;
    const int r = TR ? lane / (R / 8) : lane >> 3;
    const int c = TR ? (lane & (R / 8 - 1)) ^ tr_swz(r) : (lane & 7) ^ op_swz(r);
    k_lane = c * 16;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      // the swizzle of load q's k-rows differs from load 0's by a constant
      const int cc = TR ? c ^ tr_swz((lds_load + i) * kRows) : c;
      off[i] = (uint32_t)(((load + i) * kRows + r) * row_bytes) + cc * 16;
    }
  }
  // The next block, of which `left` elements of K are there: its buffer, then loads i of it into LDS
  __device__ __forceinline__ i32x4 block(int left) const {
    return buffer_of(base, TR ? (uint32_t)(min(left, BK) * row_bytes - cut) : bytes);
  }
  __device__ __forceinline__ void advance() {
    base += step;
    if (!TR) bytes -= step;
  }
  __device__ __forceinline__ void load(int i, i32x4 buffer, int left, uint32_t at) const {
    uint32_t o = off[i];
    if (!TR) o = (int)k_lane < left * 2 ? o : kNowhere;
    dma16_bounded(buffer, o, __builtin_amdgcn_readfirstlane(at + lds + i * 1024));
  }
  // Where this lane reads its part of a fragment of the wave whose first one is
  // number i0: fragment i0 + i is at an offset (or, k-strided, an exclusive or).
  static __device__ __forceinline__ uint32_t lane_at(int i0, int lane) {
    const int g = lane >> 4, i = lane & 15;
    if (TR) {
      const int k = g * 8 + (i >> 2);
      return (k * (R * 2) + (tr_swz(k) << 4) + ((i & 2) << 3) + ((i & 1) << 3)) ^ (i0 << 5);
    }
    return i0 * 2048 + i * 128 + ((g ^ op_swz(i)) << 4);
  }
  // MFMA fragment of rows 16 (i0 + i) .. + 15, k in [32 s, 32 s + 32); at: the
  // LDS address of the block + lane_at(i0)
  template <class F>
  static __device__ __forceinline__ F frag(uint32_t at, int i, int s) {
    typedef __attribute__((address_space(3))) char lds_char;
    if constexpr (TR) {
      typedef short v4s __attribute__((ext_vector_type(4)));
      typedef short v8s __attribute__((ext_vector_type(8)));
      typedef __attribute__((address_space(3))) v4s lds_v4s;
      lds_char* x = (lds_char*)(uintptr_t)(at ^ (uint32_t)(i << 5));
      const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(x + s * 32 * R * 2));
      const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(x + (s * 32 + 4) * R * 2));
      return __builtin_bit_cast(F, v8s{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
    } else {
      typedef __attribute__((address_space(3))) F lds_f;
      return *(lds_f*)((lds_char*)(uintptr_t)(at ^ (uint32_t)(s << 6)) + i * 2048);
    }
  }
};

// k...Part: the sums over a part of k, FP32, into the workspace.
enum Kind { kForward, kForwardGlu, kDgrad, kWgrad, kDgradPart, kWgradPart, kForwardPart };

// Waits until at most N of the wave's vector memory operations are outstanding
// (they end in their order) and all of its LDS operations are done.
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));
}
__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }

template <class E, int KIND, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64, 1) void gemm16_kernel(Gemm16Args p) {
  constexpr int NW = WM * WN, MS = BM / WM / 16, NS = BN / WN / 16;
  constexpr bool GLU = KIND == kForwardGlu, WGRAD = KIND == kWgrad || KIND == kWgradPart;
  constexpr bool DGRAD = KIND == kDgrad || KIND == kDgradPart, PART = KIND >= kDgradPart;
  constexpr bool F32 = WGRAD || PART;   // out is FP32
  using F = typename E::frag;
  using P = Operand<BM, WGRAD, NW>;
  using Q = Operand<BN, DGRAD || WGRAD, NW>;
  __shared__ __attribute__((aligned(1024))) unsigned char sm[2 * (P::kBytes + Q::kBytes)];   // two blocks of P, two of Q
  __shared__ int first[WGRAD ? 1 : kMaxGroups + 1];

  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wm = wave / WN, wn = wave % WN;
  const int cols = GLU ? p.N / 2 : p.N;            // columns of out
  constexpr int TN = GLU ? BN / 2 : BN;            // columns of out in a tile
  const int nt = (cols + TN - 1) / TN, mt = (p.M + BM - 1) / BM;
  const uint32_t ps = lds_addr(sm), qs = ps + 2 * P::kBytes;
  const uint32_t p_at = ps + P::lane_at(wm * MS, lane), q_at = qs + Q::lane_at(GLU ? wn * (NS / 2) : wn * NS, lane);
  int total;
  if constexpr (WGRAD) {
    total = p.groups.n * mt * nt;
  } else {
    list_tiles(p.groups, BM, first);
    total = first[p.groups.n] * nt;
  }
  const int tiles = total;
  if (PART) total *= p.parts;

  // ---- tiles ----
  struct Tile {
    int g, m0, mv, n0, k, part;   // group, first row, rows there are, first column of out, length of the sum, its part
  };
  P pl;
  Q ql;
  int pleft = 0, qleft = 0;   // of K, from each operand's next block to load on
  // Tile `local` of a group of `rows` row tiles: super-blocks of SUPER row tiles,
  // in them columns of tiles
  auto place = [&](int local, int rows, int& m, int& n) {
    const int sb = local / (SUPER * nt), rem = local - sb * SUPER * nt, msb = min(SUPER, rows - sb * SUPER);
    n = rem / msb;
    m = sb * SUPER + rem - n * msb;
  };
  auto open = [&](int L) {
    Tile t;
    t.part = PART ? L / tiles : 0;
    if (PART) L -= t.part * tiles;
    // the part's first k and its length, whole blocks
    auto cut = [&](int k) {
      if (!PART) {
        t.k = k;
        return 0;
      }
      const int64_t kb = (k + BK - 1) / BK;
      const int k0 = (int)(kb * t.part / p.parts) * BK;
      t.k = min(k, (int)(kb * (t.part + 1) / p.parts) * BK) - k0;
      return k0;
    };
    const int pload = wave * P::kLoads, qload = wave * Q::kLoads;
    if constexpr (WGRAD) {
      t.g = L / (mt * nt);
      int m, n;
      place(L - t.g * mt * nt, mt, m, n);
      t.m0 = m * BM;
      t.n0 = n * BN;
      t.mv = min(BM, p.M - t.m0);
      const size_t row0 = (size_t)p.groups.at(t.g) + cut(p.groups.count(t.g));
      pl.start(p.p + row0 * p.M + t.m0, t.m0, 0, p.M, pload, pload, lane);
      ql.start(p.q + row0 * p.N + t.n0, t.n0, 0, p.N, qload, qload, lane);
    } else {
      t.g = tile_group(first, p.groups.n, L / nt);
      const int f0 = __builtin_amdgcn_readfirstlane(first[t.g]), f1 = __builtin_amdgcn_readfirstlane(first[t.g + 1]);
      int m, n;
      place(L - f0 * nt, f1 - f0, m, n);
      t.m0 = __builtin_amdgcn_readfirstlane(p.groups.at(t.g)) + m * BM;
      t.n0 = n * TN;
      t.mv = __builtin_amdgcn_readfirstlane(min(BM, p.groups.at(t.g + 1) - t.m0));
      const int k0 = cut(p.K);
      pl.start(p.p + (size_t)t.m0 * p.K + k0, 0, t.mv, p.K, pload, pload, lane);
      pl.bytes -= k0 * 2;
      const uint16_t* b = p.q + (size_t)t.g * p.N * p.K;
      if constexpr (DGRAD) ql.start(b + (size_t)k0 * p.N + t.n0, t.n0, 0, p.N, qload, qload, lane);
      else if constexpr (!GLU) {
        ql.start(b + (size_t)t.n0 * p.K + k0, 0, p.N - t.n0, p.K, qload, qload, lane);
        ql.bytes -= k0 * 2;
      } else {
        // the first half of the tile's rows are gate rows, the second the same
        // columns' up rows; each wave loads rows of one half
        const int h = wave >= NW / 2;
        ql.start(b + (size_t)(t.n0 + h * cols) * p.K, 0, cols - t.n0, p.K, qload, qload - h * (BN / 16), lane);
      }
    }
    pleft = qleft = t.k;
    return t;
  };
  auto refill_p = [&](int kb) {
    const i32x4 buffer = pl.block(pleft);
#pragma unroll
    for (int i = 0; i < P::kLoads; ++i) pl.load(i, buffer, pleft, ps + (kb & 1) * P::kBytes);
    pl.advance();
    pleft -= BK;
  };
  auto refill_q = [&](int kb) {
    const i32x4 buffer = ql.block(qleft);
#pragma unroll
    for (int i = 0; i < Q::kLoads; ++i) ql.load(i, buffer, qleft, qs + (kb & 1) * Q::kBytes);
    ql.advance();
    qleft -= BK;
  };
  // The first block is loaded while the tile before it is stored.
  constexpr int STORES = F32 ? MS * NS : 0;   // of a tile, each wave, behind that load
  auto early = [&](const Tile& t) {
    if (t.k > 0) {
      refill_p(0);
      refill_q(0);
    }
  };

  // Workgroup b runs on XCD b % 8 and takes tiles of its XCD's contiguous eighth
  // of the list, so that workgroups behind one L2 share operands.
  const int xcd = blockIdx.x & 7, hi = (int)((long)total * (xcd + 1) / 8), step_L = gridDim.x >> 3;
  int L = (int)((long)total * xcd / 8) + (blockIdx.x >> 3);
  if (L >= hi) return;
  Tile cur = open(L);
  early(cur);
  bool stored = false;   // a tile's stores follow its early loads
  while (true) {
    const int KB = (cur.k + BK - 1) / BK;
    v4f acc[MS][NS];
#pragma unroll
    for (int ms = 0; ms < MS; ++ms)
#pragma unroll
      for (int ns = 0; ns < NS; ++ns) acc[ms][ns] = v4f{0.f, 0.f, 0.f, 0.f};

    // A wave holds its m-side fragments of a step of 32 k and streams the n-side
    // ones, AHEAD of their use; the next step's m-side fragments replace these
    // behind their last use.  So the m-side place of a block is free at the
    // beginning of its second step, the n-side place at its end: a barrier each,
    // and it is refilled.  Loads are never all waited for at once, and the L2,
    // which gives at most some 12 TB/s here (23 bytes a clock and CU), is kept
    // busy: with one refill a block the tile of 256 x 256 was 5% slower.
    constexpr int AHEAD = NS > 3 ? 3 : NS - 1, SLOTS = AHEAD + 1;
    static_assert(NS % SLOTS == 0, "a fragment has the same slot in every step");
    F pf[MS], qf[SLOTS];
    auto readq = [&](int kb, int s, int ns) {
      const int i = GLU ? (ns < NS / 2 ? 0 : BN / 32) + ns % (NS / 2) : ns;
      qf[ns % SLOTS] = Q::template frag<F>(q_at + (kb & 1) * Q::kBytes, i, s);
    };
    auto readp = [&](int kb, int s, int ms) { pf[ms] = P::template frag<F>(p_at + (kb & 1) * P::kBytes, ms, s); };
    auto free_p = [&](int kb) {
      __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
      barrier();
      if (kb + 2 < KB) refill_p(kb);
    };
    // the next block has landed: all but the m-side refill that was issued after it
    auto next_landed = [&](int kb) {
      if (kb + 2 < KB) wait_vm<P::kLoads>();
      else wait_vm<0>();
      barrier();
    };
    auto step = [&](int kb, int s, bool more) {
#pragma unroll
      for (int ns = 0; ns < NS; ++ns) {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        if (s == 1 && ns == 0) free_p(kb);
        if (s == 1 && ns == NS - AHEAD && more) next_landed(kb);
        if (ns + AHEAD < NS) readq(kb, s, ns + AHEAD);
        else if (more) readq(kb + s, s ^ 1, ns + AHEAD - NS);
        if (s == 1 && ns == NS - 1 && kb + 2 < KB) refill_q(kb);
#pragma unroll
        for (int ms = 0; ms < MS; ++ms) {
          acc[ms][ns] = E::mfma(qf[ns % SLOTS], pf[ms], acc[ms][ns]);
          if (ns + 1 == NS && more) {
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            readp(kb + s, s ^ 1, ms);
          }
        }
      }
    };
    if (KB > 0) {
      if (F32 && stored) wait_vm<STORES>();   // block 0
      else wait_vm<0>();
      barrier();
      if (KB > 1) {
        refill_p(1);
        refill_q(1);
      }
      if (wm * MS * 16 < cur.mv) {
#pragma unroll
        for (int ns = 0; ns < AHEAD; ++ns) readq(0, 0, ns);
#pragma unroll
        for (int ms = 0; ms < MS; ++ms) readp(0, 0, ms);
        for (int kb = 0; kb < KB - 1; ++kb) {
          step(kb, 0, true);
          step(kb, 1, true);
        }
        step(KB - 1, 0, true);
        step(KB - 1, 1, false);
      } else {
        // none of the wave's rows is there: its loads and barriers only
        for (int kb = 0; kb < KB; ++kb) {
          free_p(kb);
          if (kb + 1 < KB) {
            next_landed(kb);
            if (kb + 2 < KB) refill_q(kb);
          }
        }
      }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);
    barrier();   // every wave has read the last block
    const Tile done = cur;
    L += step_L;
    const bool more_tiles = L < hi;
    if (more_tiles) {
      cur = open(L);
      early(cur);
    }

    // ---- epilogue: lane (g16, r16) holds row ms*16 + r16, columns ns*16 + 4*g16 .. +3 ----
    // Sixteen rows at a time go through the wave's part of the second block's
    // place, whose rows are then read in whole chunks.  Its addresses are made
    // anew for every tile (`el` hides that they are the same): kept in registers
    // over the sums they would be spilled, and reloading them would wait for the
    // stores before.
    int el = lane;
    asm volatile("" : "+v"(el));
    const int er16 = el & 15, eg16 = el >> 4;
    constexpr int kPart = 16 * NS * 64;
    static_assert(NW * kPart <= P::kBytes + Q::kBytes && P::kBytes % kPart == 0, "parts fit");
    const int part_at = wave * kPart;
    unsigned char* ep = sm + (part_at < P::kBytes ? P::kBytes + part_at : P::kBytes + Q::kBytes + part_at);
    auto stage = [&](const v4f (&row)[NS]) {
#pragma unroll
      for (int ns = 0; ns < NS; ++ns)
        *reinterpret_cast<v4f*>(ep + er16 * (NS * 64) + (((ns * 4 + eg16) ^ (er16 & 7)) << 4)) = row[ns];
    };
    auto staged = [&](int r, int c) { return *reinterpret_cast<const v4f*>(ep + r * (NS * 64) + ((c ^ (r & 7)) << 4)); };
    if constexpr (F32) {
      // Every wave makes the same number of stores (rows and columns past the end
      // are out of the buffer's bounds, which drops them), so that the wait for the
      // next tile's first block can leave them in flight.  Rows of 512 bytes a
      // store, past the caches: 1.9 GB of gradients (8192 rows in 32 groups, 7168 x
      // 2048) take 535 to 620 us over cards; on one where this took 665 it was 745
      // with 128-byte rows from registers and 770 through the caches.
      const size_t row0 = WGRAD ? ((size_t)done.part * p.groups.n + done.g) * p.M : (size_t)done.part * p.groups.rows;
      const uint64_t base = reinterpret_cast<uint64_t>(static_cast<float*>(p.out) + (row0 + done.m0) * p.N);
      const __amdgpu_buffer_rsrc_t buffer = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<void*>(uniform_ptr(reinterpret_cast<const void*>(base))), 0,
          __builtin_amdgcn_readfirstlane((uint32_t)min((int64_t)done.mv * p.N * 4, (int64_t)0x7FFFFFE0)), 0x00020000);
      constexpr int CH = NS * 4, IT = 16 * CH / 64;   // 16-byte chunks of a row; a lane's of sixteen rows
      constexpr int kNonTemporal = 2;
#pragma unroll
      for (int pass = 0; pass < MS; ++pass) {
        stage(acc[pass]);
        __builtin_amdgcn_wave_barrier();   // the wave's LDS operations are in order
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const int r = (i * 64 + el) / CH, c = el % CH, n = done.n0 + wn * NS * 16 + c * 4;
          const uint32_t at = (uint32_t)((wm * MS * 16 + pass * 16 + r) * (int64_t)p.N + n) * 4;
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, staged(r, c)), buffer, n < p.N ? at : kNowhere,
                                                 0, kNonTemporal);
        }
      }
      stored = true;
    } else {
      // What follows is one short loop: code that runs once a tile is fetched at
      // some 0.1 us per 128 bytes, and an activation spelled out for every register
      // of a tile was 140 KB of it.  What is loaded here (bias, residual) is loaded a pass
      // ahead.
      using V8 = Values<E, true>;
      constexpr int CH = GLU ? NS : 2 * NS;   // 16-byte chunks of a row of out
      constexpr int IT = 16 * CH / 64;
      static_assert(IT * 64 == 16 * CH && 64 % CH == 0, "a lane keeps its columns");
      const int er = el / CH, ec = el % CH;
      const int n = done.n0 + (wn * CH + ec) * 8;
      const bool nok = n < cols;
      u32x4 bg{}, bu{}, rv[IT];
      auto fetch = [&](int pass, int i) {
        const int r = min(wm * MS * 16 + pass * 16 + er + i * (64 / CH), done.mv - 1);
        if (p.residual) rv[i] = load_chunk(p.residual + ((size_t)done.m0 + r) * cols + (nok ? n : 0));
      };
      if (p.bias) {
        const uint16_t* bp = p.bias + (size_t)done.g * p.N + (nok ? n : 0);
        bg = load_chunk(bp);
        if (GLU) bu = load_chunk(bp + cols);
      }
#pragma unroll
      for (int i = 0; i < IT; ++i) fetch(0, i);
      if (wm * MS * 16 < done.mv)
#pragma unroll 1
      for (int pass = 0; pass < MS; ++pass) {
#pragma unroll
        for (int ms = 0; ms < MS; ++ms)
          if (pass == ms) stage(acc[ms]);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const int r = er + i * (64 / CH), tr = wm * MS * 16 + pass * 16 + r;
          const bool ok = tr < done.mv && nok;
          const size_t m = (size_t)done.m0 + tr;
          auto z8 = [&](int c) {
            V8 z;
            const v4f a = staged(r, c), b = staged(r, c + 1);
#pragma unroll
            for (int e = 0; e < 4; ++e) z.v[e] = a[e], z.v[4 + e] = b[e];
            return z;
          };
          auto add = [](V8& z, const V8& v) {
#pragma unroll
            for (int e = 0; e < 8; ++e) z.v[e] += v.v[e];
          };
          V8 z = z8(2 * ec), u;
          add(z, V8(bg));
          if (GLU) {
            u = z8(2 * (CH + ec));
            add(u, V8(bu));
          }
          if (p.pre && ok) {
            z.put(p.pre + m * p.N + n);
            if (GLU) u.put(p.pre + m * p.N + cols + n);
          }
          if constexpr (GLU) {
#pragma unroll
            for (int e = 0; e < 8; ++e) z.v[e] = glu_value(z.v[e], u.v[e]);
          } else if constexpr (KIND == kForward) {
            activate(p.act, z.v);
          }
          if (p.residual) add(z, V8(rv[i]));
          fetch(min(pass + 1, MS - 1), i);
          if (ok) z.put(static_cast<uint16_t*>(p.out) + m * cols + n);
        }
      }
    }
    if (!more_tiles) return;
  }
}

// out = the sum of the parts in order (+ residual, to the type), or FP32 (TO32).
// Rows from the last group's end on are left.
template <class E, bool TO32>
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ parts, int n, size_t size, Groups groups,
                                                   int cols, const uint16_t* residual, void* out) {
  const size_t end = TO32 ? size : (size_t)groups.at(groups.n) * cols;
  for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 8; i < end; i += (size_t)gridDim.x * 256 * 8) {
    v4f a = *reinterpret_cast<const v4f*>(parts + i), b = *reinterpret_cast<const v4f*>(parts + i + 4);
    for (int s = 1; s < n; ++s) {
      a += *reinterpret_cast<const v4f*>(parts + s * size + i);
      b += *reinterpret_cast<const v4f*>(parts + s * size + i + 4);
    }
    if constexpr (TO32) {
      *reinterpret_cast<v4f*>(static_cast<float*>(out) + i) = a;
      *reinterpret_cast<v4f*>(static_cast<float*>(out) + i + 4) = b;
    } else {
      Values<E, true> v;
      if (residual) v = Values<E, true>(load_chunk(residual + i));
#pragma unroll
      for (int e = 0; e < 4; ++e) v.v[e] += a[e], v.v[4 + e] += b[e];
      v.put(static_cast<uint16_t*>(out) + i);
    }
  }
}

// The forward's epilogue on the parts' sums, eight columns of out a thread.
template <class E>
__global__ __launch_bounds__(256) void join_forward_kernel(const float* __restrict__ parts, int n, Gemm16Args p) {
  using V8 = Values<E, true>;
  const bool glu = p.act == kActSwiglu;
  const int cols = glu ? p.N / 2 : p.N;
  const size_t end = (size_t)p.groups.at(p.groups.n) * (cols / 8), size = (size_t)p.groups.rows * p.N;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < end; i += (size_t)gridDim.x * 256) {
    const int m = (int)(i / (cols / 8)), c = (int)(i - (size_t)m * (cols / 8)) * 8;
    int g = 0;
    if (p.bias && p.groups.offsets) {   // the last group that starts at or before the row
      int hi = p.groups.n - 1;
      while (g < hi) {
        const int mid = (g + hi + 1) >> 1;
        if (p.groups.at(mid) <= m) g = mid; else hi = mid - 1;
      }
    }
    auto z8 = [&](int col) {
      const float* at = parts + (size_t)m * p.N + col;
      v4f a = *reinterpret_cast<const v4f*>(at), b = *reinterpret_cast<const v4f*>(at + 4);
      for (int s = 1; s < n; ++s) {
        a += *reinterpret_cast<const v4f*>(at + s * size);
        b += *reinterpret_cast<const v4f*>(at + s * size + 4);
      }
      V8 z;
      if (p.bias) z = V8(load_chunk(p.bias + (size_t)g * p.N + col));
#pragma unroll
      for (int e = 0; e < 4; ++e) z.v[e] += a[e], z.v[4 + e] += b[e];
      if (p.pre) z.put(p.pre + (size_t)m * p.N + col);
      return z;
    };
    V8 z = z8(c);
    if (glu) {
      const V8 u = z8(cols + c);
#pragma unroll
      for (int e = 0; e < 8; ++e) z.v[e] = glu_value(z.v[e], u.v[e]);
    } else {
      activate(p.act, z.v);
    }
    const size_t at = (size_t)m * cols + c;
    if (p.residual) {
      const V8 r(load_chunk(p.residual + at));
#pragma unroll
      for (int e = 0; e < 8; ++e) z.v[e] += r.v[e];
    }
    z.put(static_cast<uint16_t*>(p.out) + at);
  }
}

// Tiles of a product with `m` rows (over all groups) and n columns, about: half
// a row tile more for every group that has rows, and at least one.
long tiles_of(long m, int groups, int n, int bm, int bn) {
  const long live = std::min<long>(groups, m);
  const long rows = live <= 1 ? (m + bm - 1) / bm : std::max(live, (2 * m / bm + live + 1) / 2);
  return rows * ((n + bn - 1) / bn);
}

constexpr int kCus = 256;

// 256 x 256 tiles, one to a CU, or 128 x 128, two: whichever takes less time by
// rounds of tiles.  Measured per block of 64 k with every CU busy: 1.6 us a
// round of 256 x 256 tiles, 1.0 a round of 512 of 128 x 128 (8192 cubed: 0.81
// against 1.0 ms).
bool big_tiles(long t256, long t128) {
  return 8 * ((t256 + kCus - 1) / kCus) <= 5 * ((t128 + 2 * kCus - 1) / (2 * kCus));
}

template <int KIND, class E>
void launch_kind(const Gemm16Args& p, bool big, long tiles_bound, hipStream_t stream) {
  const long wgs = (tiles_bound + 7) / 8 * 8;
  if constexpr (KIND < kDgradPart)
    if (big) {
      hipLaunchKernelGGL((gemm16_kernel<E, KIND, 256, 256, 4, 2>), dim3((unsigned)std::min(wgs, (long)kCus)), dim3(512), 0,
                         stream, p);
      return;
    }
  hipLaunchKernelGGL((gemm16_kernel<E, KIND, 128, 128, 2, 2>), dim3((unsigned)std::min(wgs, 2L * kCus)), dim3(256), 0,
                     stream, p);
}

template <int KIND>
void launch(int type, const Gemm16Args& p, bool big, long tiles_bound, hipStream_t stream) {
  if (type == 0) launch_kind<KIND, Bf16>(p, big, tiles_bound, stream);
  else launch_kind<KIND, Fp16>(p, big, tiles_bound, stream);
}

// Products over rows: tiles of both sizes, their bound for the launch.
struct RowTiles {
  bool big;
  long bound;
  RowTiles(int rows, int n_groups, int cols, bool glu) {
    const int c256 = glu ? 128 : 256, c128 = glu ? 64 : 128;
    big = big_tiles(tiles_of(rows, n_groups, cols, 256, c256), tiles_of(rows, n_groups, cols, 128, c128));
    const int bm = big ? 256 : 128, bn = big ? c256 : c128;
    bound = ((long)rows / bm + n_groups) * ((cols + bn - 1) / bn);
  }
};

// Parts of k for products whose tiles may be too few for the chip: the number
// with the least time in us by what was measured: a block of 64 k takes 0.65 with
// at most one 128 x 128 tile to a CU and 1.0 a round of two; joining takes 2.5 for
// its launch and the parts' bytes, written and read, at 6 TB/s (so measured from 17
// to 400 MB of them).  Above 64 MB they are counted at 3: not the bytes are slower
// there, but whole rounds overstate a partly filled last one, which one part has and
// two have not.  640 tiles over a sum of 4096 are modelled as 128 us in one part and
// 126 in two of 84 MB; they take 95 and 103.  Both gradients of 8192 rows in 32
// groups, K 2048, N 7168, take 881 to 965 us over cards, 1020 with the rows' in two
// parts of 134 MB together.  Between 64 MB and 84 the border is not measured.  (2048 x
// 2048 from a sum over 16384: one part 194 us, two 149, four 160; 256 x 256 over
// 8192: 70, 42, 26, 19 and 18.5 with 1 to 16; 6867 x 128 over 4088: 45, 28, 23, 25
// and 35.)
int parts_of(long t128, int k, double elements, double* time = nullptr) {
  int best = 1;
  double least = 0;
  for (int p = 1; p <= 16; p *= 2) {
    const long blocks = ((k + BK - 1) / BK + p - 1) / p, wgs = t128 * p;
    if (p > 1 && blocks < 2) break;
    const double rounds = wgs <= kCus ? 0.65 : (double)((wgs + 2 * kCus - 1) / (2 * kCus));
    const double bytes = elements * 4 * p;
    const double t = blocks * rounds + (p > 1 ? 2.5 + 2 * bytes / (bytes > 64e6 ? 3e6 : 6e6) : 0.0);
    if (p == 1 || t < least) {
      least = t;
      best = p;
    }
  }
  if (time) *time = least;
  return best;
}
// The forward's: 0 where slim tiles take less time, 16 rows and fewer among them.
// Both read the groups' weights, the slim tiles faster (128 rows in 64 groups, K
// 7168, N 4096: 418 against 540 us); both are counted as reading them once, though
// slim tiles read those of a group with several row tiles again.  Of 120 random
// products of at most 30 GFLOP 114 take at most 8% longer than the fastest of slim
// tiles and 1 to 16 parts, the others up to 25%; larger ones were not in that set.
int forward_parts(const Gemm16Args& p) {
  double slim = gemm16_slim_time(p), tile;
  const long t128 = tiles_of(p.groups.rows, p.groups.n, p.N, 128, 128);
  const int parts = parts_of(t128, p.K, (double)p.groups.rows * p.N, &tile);
  if (p.groups.rows <= 16 && !std::isinf(slim)) return 0;
  const double weights = 2.0 * std::min(p.groups.n, p.groups.rows) * p.N * p.K;
  slim = std::max(slim, weights / 7.5e6);
  tile = std::max(tile, weights / 5.5e6) + 0.7;
  return slim <= tile ? 0 : parts;
}
int dgrad_parts(int rows, int n_groups, int K, int N) {
  return parts_of(tiles_of(rows, n_groups, K, 128, 128), N, (double)rows * K);
}
int wgrad_parts(int rows, int n_groups, int K, int N) {
  return parts_of((long)n_groups * ((N + 127) / 128) * ((K + 127) / 128), rows / n_groups, (double)n_groups * N * K);
}

template <bool TO32>
void join(int type, const float* parts, int n, size_t size, const Groups& groups, int cols, const void* residual,
          void* out, hipStream_t stream) {
  const unsigned grid = (unsigned)std::min<size_t>((size / 8 + 255) / 256, 2048);
  const uint16_t* res = static_cast<const uint16_t*>(residual);
  if (type == 0) hipLaunchKernelGGL((join_kernel<Bf16, TO32>), dim3(grid), dim3(256), 0, stream, parts, n, size, groups, cols, res, out);
  else hipLaunchKernelGGL((join_kernel<Fp16, TO32>), dim3(grid), dim3(256), 0, stream, parts, n, size, groups, cols, res, out);
}

}  // namespace

size_t gemm16_workspace_bytes(int rows, int n_groups, int K, int N, int act) {
  Gemm16Args p{};
  p.groups = Groups{nullptr, n_groups, rows};
  p.N = N;
  p.K = K;
  p.act = act;
  const int parts = forward_parts(p);
  return parts > 1 ? (size_t)parts * rows * N * 4 : 0;
}

size_t gemm16_backward_workspace_bytes(int rows, int n_groups, int K, int N) {
  const int d = dgrad_parts(rows, n_groups, K, N), w = wgrad_parts(rows, n_groups, K, N);
  return std::max(d > 1 ? (size_t)d * rows * K * 4 : 0, w > 1 ? (size_t)w * n_groups * N * K * 4 : 0);
}

hipError_t launch_gemm16(int type, const void* a, const int32_t* offsets, int n_groups, int rows, int K, int N,
                         const void* b, const void* bias, int act, const void* residual, void* pre, void* out,
                         void* workspace, hipStream_t stream) {
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
  p.parts = forward_parts(p);
  if (p.parts > 1) {
    Gemm16Args sums = p;
    sums.out = workspace;
    launch<kForwardPart>(type, sums, false, ((long)rows / 128 + n_groups) * ((N + 127) / 128) * p.parts, stream);
    const size_t chunks = (size_t)rows * (act == kActSwiglu ? N / 2 : N) / 8;
    const dim3 grid((unsigned)std::min<size_t>((chunks + 255) / 256, 4096));
    const float* parts = static_cast<const float*>(workspace);
    if (type == 0) hipLaunchKernelGGL(join_forward_kernel<Bf16>, grid, dim3(256), 0, stream, parts, p.parts, p);
    else hipLaunchKernelGGL(join_forward_kernel<Fp16>, grid, dim3(256), 0, stream, parts, p.parts, p);
    return hipGetLastError();
  }
  if (p.parts == 0) return launch_gemm16_slim(type, p, stream);
  const RowTiles t(rows, n_groups, act == kActSwiglu ? N / 2 : N, act == kActSwiglu);
  if (act == kActSwiglu) launch<kForwardGlu>(type, p, t.big, t.bound, stream);
  else launch<kForward>(type, p, t.big, t.bound, stream);
  return hipGetLastError();
}

hipError_t launch_gemm16_dgrad(int type, const void* dz, const int32_t* offsets, int n_groups, int rows, int K, int N,
                               const void* b, const void* residual, void* da, void* workspace, hipStream_t stream) {
  Gemm16Args p{};
  p.p = static_cast<const uint16_t*>(dz);
  p.q = static_cast<const uint16_t*>(b);
  p.groups = Groups{offsets, n_groups, rows};
  p.N = K;
  p.K = N;
  p.residual = static_cast<const uint16_t*>(residual);
  p.out = da;
  p.parts = dgrad_parts(rows, n_groups, K, N);
  const RowTiles t(rows, n_groups, K, false);
  if (p.parts > 1) {
    p.out = workspace;
    launch<kDgradPart>(type, p, false, ((long)rows / 128 + n_groups) * ((K + 127) / 128) * p.parts, stream);
    join<false>(type, static_cast<const float*>(workspace), p.parts, (size_t)rows * K, p.groups, K, residual, da, stream);
  } else {
    launch<kDgrad>(type, p, t.big, t.bound, stream);
  }
  return hipGetLastError();
}

hipError_t launch_gemm16_wgrad(int type, const void* dz, const void* a, const int32_t* offsets, int n_groups, int rows,
                               int K, int N, float* db, void* workspace, hipStream_t stream) {
  Gemm16Args p{};
  p.p = static_cast<const uint16_t*>(dz);
  p.q = static_cast<const uint16_t*>(a);
  p.groups = Groups{offsets, n_groups, rows};
  p.M = N;
  p.N = K;
  p.out = db;
  p.parts = rows > 0 ? wgrad_parts(rows, n_groups, K, N) : 1;
  const long t256 = (long)n_groups * ((N + 255) / 256) * ((K + 255) / 256);
  const long t128 = (long)n_groups * ((N + 127) / 128) * ((K + 127) / 128);
  if (p.parts > 1) {
    p.out = workspace;
    launch<kWgradPart>(type, p, false, t128 * p.parts, stream);
    join<true>(type, static_cast<const float*>(workspace), p.parts, (size_t)n_groups * N * K, p.groups, K, nullptr, db,
               stream);
  } else {
    // groups differ in rows, so in time: many tiles even it out (8192 rows in 33
    // groups to 512 x 512: 30 us with the 132 large tiles, 17 with the small)
    const bool big = big_tiles(t256, t128) && (n_groups == 1 || t256 >= 8 * kCus);
    launch<kWgrad>(type, p, big, big ? t256 : t128, stream);
  }
  return hipGetLastError();
}

}  // namespace moe
