// Groups of rows given by offsets in device memory: their first rows, and how
// many pieces of `unit` rows lie before each.
#pragma once

#include "common.cuh"
#include "sparse.h"

namespace rmx {

// first[0 .. G] and before[0 .. G], by all threads of a block of NT (a multiple
// of 32): first is offsets[0 .. G] with values below 0, past M or falling
// replaced by the nearest that are not; before[g] counts the pieces of the
// groups before g.  Ends with a block barrier.
template <int NT>
__device__ __forceinline__ void ragged_scan(const int32_t* offsets, int G, int M, int unit, int* first, int* before) {
  constexpr int WARPS = NT / 32;
  __shared__ int tmp[2][WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // A thread takes `per` neighbouring groups (G <= kMaxExperts).
  const int per = (G + NT - 1) / NT, g0 = min(G, (int)threadIdx.x * per), g1 = min(G, g0 + per);
  // Running maximum: of a thread's own offsets, over the warp, over the warps.
  int top = 0;
  for (int g = g0; g < g1; ++g) top = max(top, min(offsets[g], M));
  int inc = top;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc = max(inc, u);
  }
  if (lane == 31) tmp[0][warp] = inc;
  int prev = __shfl_up_sync(0xffffffffu, inc, 1);
  if (lane == 0) prev = 0;
  __syncthreads();
  for (int w = 0; w < warp; ++w) prev = max(prev, tmp[0][w]);
  for (int g = g0; g < g1; ++g) {
    prev = max(prev, min(offsets[g], M));
    first[g] = prev;
  }
  if (threadIdx.x == NT - 1) first[G] = max(prev, min(offsets[G], M));
  __syncthreads();
  int n = 0;
  for (int g = g0; g < g1; ++g) n += (first[g + 1] - first[g] + unit - 1) / unit;
  inc = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) tmp[1][warp] = inc;
  __syncthreads();
  int base = inc - n;
  for (int w = 0; w < warp; ++w) base += tmp[1][w];
  for (int g = g0; g < g1; ++g) {
    before[g] = base;
    base += (first[g + 1] - first[g] + unit - 1) / unit;
  }
  if (threadIdx.x == NT - 1) before[G] = base;
  __syncthreads();
}
// The group that piece b lies in: before[g] <= b < before[g + 1], b < before[G].
__device__ __forceinline__ int ragged_group(const int* before, int G, int b) {
  int lo = 0, hi = G;  // before[lo] <= b < before[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= b) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace rmx
