// Row ranges of the groups of include/moe_experts.h's products, and lists of
// row tiles over them.
#pragma once

#include "common.h"

namespace moe {

constexpr int kMaxGroups = 1024;
// Rows of a product: what kernels and host add to a row number or a number of
// rows (a tile's rows less one, a chunk's, the groups) stays within an int.
constexpr int kMaxRows = INT32_MAX - (kMaxGroups - 1);

// First row of group g (g = n: the end of the last).  Ranges never leave [0, rows).
struct Groups {
  const int32_t* offsets;   // NULL: one group of all rows
  int n, rows;
  __device__ __forceinline__ int at(int g) const {
    if (!offsets) return g ? rows : 0;
    return min(max(offsets[g], 0), rows);
  }
  __device__ __forceinline__ int count(int g) const { return max(0, at(g + 1) - at(g)); }
};

// first[g] = tiles of `size` rows in the groups before g, by the first wave of
// the workgroup, which then synchronises.
__device__ __forceinline__ void list_tiles(const Groups& g, int size, int* first) {
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int carry = 0;
    for (int base = 0; base < g.n; base += 64) {
      int v = base + lane < g.n ? (g.count(base + lane) + size - 1) / size : 0;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(v, o);
        if (lane >= o) v += u;
      }
      if (base + lane < g.n) first[base + lane + 1] = carry + v;
      carry += __shfl(v, 63);
    }
    if (lane == 0) first[0] = 0;
  }
  __syncthreads();
}

// The group of tile i < first[n].
__device__ __forceinline__ int tile_group(const int* first, int n, int i) {
  int a = 0, b = n - 1;
  while (a < b) {
    const int mid = (a + b + 1) >> 1;
    if (first[mid] <= i) a = mid; else b = mid - 1;
  }
  return __builtin_amdgcn_readfirstlane(a);
}

}  // namespace moe
