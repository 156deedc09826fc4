// Dropout's random bits: Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011), a block cipher of ten
// rounds over a 128-bit counter with a 64-bit key.  A counter serves eight
// neighbouring columns of a row with 16 bits each, so a thread that holds 16
// bytes of 16-bit values draws once for them.
#pragma once

#include "common.cuh"
#include "sparse.h"

namespace rmx {

// The generator's state, read once by each thread.
struct DropBits {
  uint32_t k0, k1, o0, o1;
  uint32_t lim;  // thresh << 16
  int mode;
};
__device__ __forceinline__ DropBits drop_bits(const Drop& d) {
  DropBits b{};
  b.mode = d.mode;
  if (d.mode == DROP_BITS) {
    const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(d.state);
    b.k0 = (uint32_t)s.x;
    b.k1 = (uint32_t)(s.x >> 32);
    b.o0 = (uint32_t)s.y;
    b.o1 = (uint32_t)(s.y >> 32);
    b.lim = d.thresh << 16;
  }
  return b;
}

// Which of columns 8 * grp .. 8 * grp + 7 of a row are kept, a bit each.
__device__ __forceinline__ uint32_t keep8(const DropBits& b, long long row, int grp) {
  uint32_t c0 = (uint32_t)grp | (uint32_t)(row >> 32) << 24, c1 = (uint32_t)row, c2 = b.o0, c3 = b.o1;
  uint32_t k0 = b.k0, k1 = b.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  const uint32_t w[4] = {c0, c1, c2, c3};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m |= (w[i] << 16) >= b.lim ? 1u << (2 * i) : 0u;
    m |= w[i] >= b.lim ? 2u << (2 * i) : 0u;
  }
  return m;
}

// The keep bits of a lane's eight elements, bit i for element i.  VEC: eight
// neighbouring columns, one draw.  Else element i is column c0 + L * i (c0 the
// lane's first): eight neighbouring lanes share a draw, and each of them makes
// the one for another i.  Every lane of the warp takes part.
template <int L, bool VEC> __device__ __forceinline__ uint32_t keep_of(const DropBits& b, long long row, int c0) {
  if constexpr (VEC) {
    return keep8(b, row, c0 >> 3);
  } else {
    const int sub = threadIdx.x & 7;
    const uint32_t mine = keep8(b, row, (c0 + L * sub) >> 3);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m |= ((__shfl_sync(0xffffffffu, mine, i, 8) >> sub) & 1u) << i;
    return m;
  }
}

// v * scale where kept, exactly 0 elsewhere.
__device__ __forceinline__ void drop_pairs(uint32_t keep, float scale, float2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i].x = keep & (1u << (2 * i)) ? v[i].x * scale : 0.f;
    v[i].y = keep & (2u << (2 * i)) ? v[i].y * scale : 0.f;
  }
}

}  // namespace rmx
