// Device helpers of the row passes of the 8-bit operators: which columns a
// thread holds, int8 rounding and packing, checkpoint scales, reductions.
//
// A row is cut into blocks of 8 * L columns, one to L lanes (8, 16 or 32: a
// short row takes a part of a warp) at a time, eight columns to a lane.  VEC
// (rows start on 16-byte boundaries): a lane holds eight consecutive columns,
// moved as 16-byte vectors.  Else (odd row lengths): columns lane, lane + L,
// ..., so that the lanes' one-element accesses are consecutive.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "q8.h"

namespace rmx {

constexpr uint32_t kInfBits = 0x7f800000u;
constexpr float kRound = 12582912.0f;  // 1.5 * 2^23

inline bool rows_aligned(int C, int esize) { return ((long long)C * esize) % 16 == 0; }

// ---------------------------------------------------------------- columns
template <typename T> struct alignas(16) Chunk {
  T v[8];
};
template <int L, bool VEC> __device__ __forceinline__ int col0(int blk, int lane) {
  return blk * (8 * L) + (VEC ? lane * 8 : lane);
}
// Column of element i, given that of element 0.
template <int L, bool VEC> __device__ __forceinline__ int col(int c0, int i) { return c0 + (VEC ? i : L * i); }

// Eight values of a row of C columns; columns past C read as zero.
template <typename T, int L, bool VEC>
__device__ __forceinline__ Chunk<T> load_chunk(const T* row, int c0, int C) {
  Chunk<T> k;
  if constexpr (VEC) {
    uint4* d = reinterpret_cast<uint4*>(&k);
    const uint4* s = reinterpret_cast<const uint4*>(row + c0);
    constexpr int V = 16 / (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < 8 / V; ++i) d[i] = c0 + i * V < C ? s[i] : make_uint4(0, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) k.v[i] = col<L, VEC>(c0, i) < C ? row[col<L, VEC>(c0, i)] : from_f<T>(0.f);
  }
  return k;
}
template <typename T, int L, bool VEC>
__device__ __forceinline__ void store_chunk(T* row, int c0, int C, const float2 (&f)[4]) {
  if constexpr (VEC) {
    if (sizeof(T) == 2) {
      if (c0 < C) st8(row + c0, f);
    } else {
      if (c0 < C) *reinterpret_cast<float4*>(row + c0) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
      if (c0 + 4 < C) *reinterpret_cast<float4*>(row + c0 + 4) = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col<L, VEC>(c0, i) < C) row[col<L, VEC>(c0, i)] = from_f<T>(i & 1 ? f[i / 2].y : f[i / 2].x);
  }
}
__device__ __forceinline__ void to_pairs(const Chunk<bf16>& k, float2 (&v)[4]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&k);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = bf16x2_to_f2(w[i]);
}
__device__ __forceinline__ void to_pairs(const Chunk<f16>& k, float2 (&v)[4]) {
  const __half2* h = reinterpret_cast<const __half2*>(&k);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __half22float2(h[i]);
}
__device__ __forceinline__ void to_pairs(const Chunk<float>& k, float2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = make_float2(k.v[2 * i], k.v[2 * i + 1]);
}

// ---------------------------------------------------------------- int8
// The nearest integer (ties to even) to x * f, |x * f| < 2^22, in the low byte
// of the result, two's complement: 1.5 * 2^23 + x * f in one fused operation.
__device__ __forceinline__ float2 round2(float2 x, float f) { return fma2(x, f2(f), f2(kRound)); }
// The low bytes of eight such results.
__device__ __forceinline__ uint2 low_bytes(const float2 (&t)[4]) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __byte_perm(__float_as_uint(t[i].x), __float_as_uint(t[i].y), 0x0040);
  return make_uint2(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410));
}
// Eight int8 of a row whose pitch holds them; `keep` false writes zeros.
template <int L, bool VEC>
__device__ __forceinline__ void store_bytes(int8_t* row, int c0, int P, const float2 (&t)[4], bool keep) {
  if constexpr (VEC) {
    if (c0 < P) *reinterpret_cast<uint2*>(row + c0) = keep ? low_bytes(t) : make_uint2(0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col<L, VEC>(c0, i) < P)
        row[col<L, VEC>(c0, i)] = keep ? (int8_t)__float_as_uint(i & 1 ? t[i / 2].y : t[i / 2].x) : (int8_t)0;
  }
}
template <int L, bool VEC> __device__ __forceinline__ uint2 load_bytes(const int8_t* row, int c0, int P) {
  if constexpr (VEC) return c0 < P ? *reinterpret_cast<const uint2*>(row + c0) : make_uint2(0, 0);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (col<L, VEC>(c0, i) < P) w[i / 4] |= (uint32_t)(uint8_t)row[col<L, VEC>(c0, i)] << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}
// The largest scale of 127 steps: 127 times it is still finite (1 / 127 of the
// largest float32, rounded, is one unit too much).
constexpr float kMaxScale = 0x1.020406p+121f;
// Eight int8 as floats 2^23 + 128 + q: byte ^ 0x80 in the low mantissa byte of
// 2^23.  Subtracting kBias is exact.
constexpr float kBias = 8388736.0f;  // 2^23 + 128
__device__ __forceinline__ void biased(uint2 w, float2 (&f)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t u = (h ? w.y : w.x) ^ 0x80808080u;
    f[2 * h] = make_float2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7540)),
                           __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7541)));
    f[2 * h + 1] = make_float2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7542)),
                               __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7543)));
  }
}

// ---------------------------------------------------------------- magnitudes
// Larger of a and |b|, |c|; NaN if one of them is.
__device__ __forceinline__ float max_abs(float a, float2 b) {
  float r;
  asm("{\n\t.reg .f32 x, y;\n\tabs.f32 x, %2;\n\tabs.f32 y, %3;\n\tmax.NaN.f32 %0, %1, x, y;\n\t}"
      : "=f"(r)
      : "f"(a), "f"(b.x), "f"(b.y));
  return r;
}

// ---------------------------------------------------------------- checkpoint scales
// Range of group exponents that keeps q * 2^e exact (and finite) in the
// storage type: the step 2^e no finer than its smallest subnormal (fp16) or
// normal (bf16, fp32), 127 steps no more than its largest value.
template <typename T> struct CkptRange {
  static constexpr int lo = std::is_same<T, f16>::value ? -24 : -126;
  static constexpr int hi = std::is_same<T, f16>::value ? 9 : 121;
};
// Exponent of a group whose largest magnitude has the bits `u`: the smallest
// e with max / 2^e <= 127.5, i.e. 6 below max's own exponent, or 5 when its
// mantissa is above 127.5 / 64.
template <typename T> __device__ __forceinline__ int ckpt_exp(uint32_t u) {
  if (u >= kInfBits) return kCkptNaN;
  const int e = (int)(u >> 23) - 127 - 6 + ((u & 0x7fffffu) > 0x7f0000u ? 1 : 0);
  return min(max(e, CkptRange<T>::lo), CkptRange<T>::hi);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// Value of one step of a group; NaN for a NaN group.  Exponents the packer
// does not write are read as the nearest it does.
__device__ __forceinline__ float ckpt_step(int e) {
  return e == kCkptNaN ? __uint_as_float(0x7fc00000u) : pow2(min(max(e, -126), 121));
}

// Exponents of the 8 * L columns of block blk of a row, a byte each (L / 4).
template <int L> __device__ __forceinline__ uint2 load_exps(const int8_t* e, int blk, int groups) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < L / 4; ++i)
    if (blk * (L / 4) + i < groups) w[i / 4] |= (uint32_t)(uint8_t)e[blk * (L / 4) + i] << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}
// That of element i (not VEC): columns lane + L * i, so group L * i / 32.
template <int L> __device__ __forceinline__ int exp_of(uint2 e, int i) {
  const int g = L * i / 32;
  return (int8_t)((g < 4 ? e.x : e.y) >> (8 * (g & 3)));
}

// ---------------------------------------------------------------- reductions
// Over L neighbouring lanes, in a fixed order.
template <int L> __device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int L> __device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  if constexpr (L == 32) {
    return __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}
// Sum of s and maximum of the non-negative u over the W x L threads of a row,
// in a fixed order.  `red` holds 4 * W words per row slot; `slot` alternates.
template <int W, int L>
__device__ __forceinline__ void row_reduce(float& s, uint32_t& u, uint32_t* red, int rib, int w, int& slot) {
  s = lanes_sum<L>(s);
  u = lanes_max<L>(u);
  if constexpr (W > 1) {
    uint32_t* r = red + (rib * 2 + slot) * 2 * W;
    if ((threadIdx.x & 31) == 0) {
      r[w] = __float_as_uint(s);
      r[W + w] = u;
    }
    __syncthreads();
    s = 0.f;
    u = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      s += __uint_as_float(r[i]);
      u = max(u, r[W + i]);
    }
    slot ^= 1;
  }
}

#define RMX_BY_DTYPE(dt, ...)            \
  switch (dt) {                          \
    case 0: { using T = float; __VA_ARGS__; }   \
    case 1: { using T = bf16; __VA_ARGS__; }    \
    case 2: { using T = f16; __VA_ARGS__; }     \
    default: return cudaErrorInvalidValue; \
  }

}  // namespace rmx
