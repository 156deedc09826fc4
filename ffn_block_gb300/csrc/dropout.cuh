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

// The eight columns 8 * grp .. 8 * grp + 7 of a row: 16 bits each, two to a word,
// the lower half first.
__device__ __forceinline__ void bits8(const DropBits& b, long long row, int grp, uint32_t (&c)[4]) {
  c[0] = (uint32_t)grp | (uint32_t)(row >> 32) << 24;
  c[1] = (uint32_t)row;
  c[2] = b.o0;
  c[3] = b.o1;
  uint32_t k0 = b.k0, k1 = b.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = (uint64_t)c[0] * 0xD2511F53u, p1 = (uint64_t)c[2] * 0xCD9E8D57u;
    c[0] = (uint32_t)(p1 >> 32) ^ c[1] ^ k0;
    c[1] = (uint32_t)p1;
    c[2] = (uint32_t)(p0 >> 32) ^ c[3] ^ k1;
    c[3] = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}
__device__ __forceinline__ uint32_t keep_mask(const DropBits& b, const uint32_t (&w)[4]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m |= (w[i] << 16) >= b.lim ? 1u << (2 * i) : 0u;
    m |= w[i] >= b.lim ? 2u << (2 * i) : 0u;
  }
  return m;
}
// Which of one group's are kept, a bit each.
__device__ __forceinline__ uint32_t keep8(const DropBits& b, long long row, int grp) {
  uint32_t w[4];
  bits8(b, row, grp, w);
  return keep_mask(b, w);
}
// v * scale where kept, exactly 0 elsewhere.
__device__ __forceinline__ void drop_by_words(const DropBits& b, float scale, const uint32_t (&w)[4], float2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 s = mul2(v[i], f2(scale));
    v[i].x = (w[i] << 16) >= b.lim ? s.x : 0.f;
    v[i].y = w[i] >= b.lim ? s.y : 0.f;
  }
}

// Dropout of a lane's eight elements: v * scale where kept, exactly 0 elsewhere.
// VEC: eight neighbouring columns, one draw.  Else element i is column c0 + L * i
// (c0 the lane's first): eight neighbouring lanes share a draw, and each of them
// makes the one for another i.  Every lane of the warp takes part.
template <int L, bool VEC>
__device__ __forceinline__ void drop_values(const DropBits& b, float scale, long long row, int c0, float2 (&v)[4]) {
  if (b.mode == DROP_NONE) return;
  if (b.mode == DROP_ALL) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2(0.f);
    return;
  }
  if constexpr (VEC) {
    uint32_t w[4];
    bits8(b, row, c0 >> 3, w);
    drop_by_words(b, scale, w, v);
  } else {
    const int sub = threadIdx.x & 7;
    const uint32_t mine = keep8(b, row, (c0 + L * sub) >> 3);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float& e = i & 1 ? v[i / 2].y : v[i / 2].x;
      e = (__shfl_sync(0xffffffffu, mine, i, 8) >> sub) & 1u ? e * scale : 0.f;
    }
  }
}

}  // namespace rmx
