// 8-bit floating rows: quantisation of rows (with or without a gather before
// it), of rows and columns of grouped rows in one pass, and reading back.
//
// A block of 128 values keeps q * 2^(e - 127).  Scaling by a power of two is
// exact, so the only rounding is the conversion to 8 bits.  The exponent comes
// from the largest magnitude's bits: 448 and 57344 are both 7/8 of a power of
// two, so e follows from its exponent and from whether its mantissa passes 1.75.
// Rows alone are bound by HBM (131,072 rows of 1280 bf16 columns 76 us, 99% of the copy
// rate): 16-bit values in, bytes out.

#include <float.h>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "q8_rows.cuh"
#include "ragged.cuh"
#include "sparse.h"

namespace rmx {
namespace {

constexpr int kNaNExp = 255;

// Exponent byte of a block whose largest magnitude has the bits `top`: the
// smallest e >= 0 with max <= 1.75 * 2^LIM * 2^(e - 127), LIM = 8 (e4m3: 448) or
// 15 (e5m2: 57344).
template <bool E5> __device__ __forceinline__ int block_exp(uint32_t top) {
  if (top >= kInfBits) return kNaNExp;
  const int e = (int)(top >> 23) - (E5 ? 15 : 8) + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, 0);
}
// 2^(127 - e): what a block's values are multiplied by; 0 for a NaN block.
__device__ __forceinline__ float block_inv(int e) {
  // e <= 248, so the result is a normal number, and 2^127 at e = 0.
  return e == kNaNExp ? 0.f : __uint_as_float((uint32_t)(254 - e) << 23);
}
template <bool E5> __device__ __forceinline__ uint32_t to_f8x2(float lo, float hi) {
  uint16_t r;
  if (E5) asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Eight values times inv, as bytes; a NaN block (inv 0) gives zeros.
template <bool E5> __device__ __forceinline__ uint2 to_f8x8(const float2 (&v)[4], float inv) {
  if (inv == 0.f) return make_uint2(0, 0);
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = mul2(v[i], f2(inv));
    h[i] = to_f8x2<E5>(u.x, u.y);
  }
  return make_uint2(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410));
}
// Bits of the largest magnitude of eight values; NaN comes out above infinity
// above every number.
__device__ __forceinline__ uint32_t top_of(const Chunk<float>& k) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(k.v[i]) & 0x7fffffffu);
  return m;
}
template <typename T> __device__ __forceinline__ uint32_t top_of(const Chunk<T>& k) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&k);
  uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
  return m;  // two halves, see as_f32_bits
}
// The larger of two such results.
template <typename T> __device__ __forceinline__ uint32_t top_max(uint32_t a, uint32_t b) {
  return sizeof(T) == 4 ? max(a, b) : __vmaxu2(a, b);
}
// Such a result as the bits of a float32.
template <typename T> __device__ __forceinline__ uint32_t as_f32_bits(uint32_t m) {
  if (sizeof(T) == 4) return m;
  const uint32_t top = max(m >> 16, m & 0xffffu);
  if (std::is_same<T, bf16>::value) return top << 16;
  return __float_as_uint(__half2float(__ushort_as_half((unsigned short)top)));
}

// A block belongs to eight lanes: lane l has columns 8 l .. 8 l + 7 and 64 + 8 l
// .. (so that neighbouring lanes' accesses are neighbours).  Rows that are not whole
// 16-byte vectors (not VEC) come value by value: 65,536 rows of 1001 16-bit columns
// 47 us; four neighbouring columns of a block to each of 32 lanes 59; the two vectors
// that eight columns lie in, shifted into place, 59.
template <typename T, bool VEC> __device__ __forceinline__ Chunk<T> load_eight(const T* row, int c0, int C) {
  if constexpr (VEC) {
    return load_chunk<T, 32, true>(row, c0, C);
  } else {
    Chunk<T> k;
#pragma unroll
    for (int i = 0; i < 8; ++i) k.v[i] = c0 + i < C ? row[c0 + i] : from_f<T>(0.f);
    return k;
  }
}

// Blocks of 128 columns at a time to each eight lanes.
constexpr int kBatch = 2;
template <typename T, bool VEC, bool E5, bool GATHER>
__global__ void __launch_bounds__(256) k_quant_f8(const QuantRows a, const int bpr, const int EP, const long long total) {
  pdl_enter();
  const int l = threadIdx.x & 7;
  const long long step = (long long)gridDim.x * 32 * kBatch;
  const T* x = static_cast<const T*>(a.x);
  // Whole warps stay in the loop together (their shuffles take every lane).
  for (long long w0 = ((long long)blockIdx.x * 32 + (threadIdx.x >> 5) * 4) * kBatch; w0 < total; w0 += step) {
    Chunk<T> k[kBatch][2];
    long long row[kBatch];
    int blk[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const long long b = w0 + j * 4 + ((threadIdx.x >> 3) & 3);
      row[j] = -1;
      blk[j] = 0;
      long long from = 0;
      if (b < total) {
        const long long r = total < (1ll << 31) ? (long long)((uint32_t)b / (uint32_t)bpr) : b / bpr;
        blk[j] = (int)(b - r * bpr);
        row[j] = from = r;
        if (GATHER) {
          const int s = a.source[r];
          if ((uint32_t)s < (uint32_t)a.R) from = (uint32_t)s / (uint32_t)a.k;
          else row[j] = -1;
        }
      }
      const T* p = x + (size_t)from * a.C;
      const int C = row[j] >= 0 ? a.C : 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) k[j][h] = load_eight<T, VEC>(p, blk[j] * 128 + 64 * h + 8 * l, C);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      uint32_t m = top_max<T>(top_of(k[j][0]), top_of(k[j][1]));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) m = top_max<T>(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (row[j] < 0) continue;
      const int e = block_exp<E5>(as_f32_bits<T>(m));
      const float inv = block_inv(e);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c0 = blk[j] * 128 + 64 * h + 8 * l;
        float2 v[4];
        to_pairs(k[j][h], v);
        *reinterpret_cast<uint2*>(a.q + (size_t)row[j] * (bpr * 128) + c0) = to_f8x8<E5>(v, inv);
        if (GATHER && a.out) {
          T* o = static_cast<T*>(a.out) + (size_t)row[j] * a.C;
          if constexpr (VEC) {
            store_chunk<T, 32, true>(o, c0, a.C, v);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (c0 + i < a.C) o[c0 + i] = k[j][h].v[i];
          }
        }
      }
      if (l == 0) {
        uint8_t* ex = a.e + (size_t)row[j] * EP;
        ex[blk[j]] = (uint8_t)e;
        if (blk[j] == bpr - 1)
          for (int i = bpr; i < EP; ++i) ex[i] = 0;
      }
    }
  }
}

// The value of an exponent byte's step; NaN for a NaN block.
__device__ __forceinline__ float block_step(int e) {
  if (e == kNaNExp) return __uint_as_float(0x7fc00000u);
  return e == 0 ? 0x1p-127f : __uint_as_float((uint32_t)e << 23);
}
// Two bytes as floats.
template <bool E5> __device__ __forceinline__ float2 from_f8x2(uint32_t w) {
  uint32_t h;
  if (E5) asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
  else asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}
template <typename T> struct Largest;
template <> struct Largest<float> { static constexpr float value = FLT_MAX; };
template <> struct Largest<bf16> { static constexpr float value = 0x1.fep127f; };
template <> struct Largest<f16> { static constexpr float value = 65504.f; };
// q * step in the storage type; where q is finite, so is the result.
template <typename T> __device__ __forceinline__ float read_back(float q, float step) {
  const float v = q * step;
  if (!(fabsf(q) <= FLT_MAX)) return v;
  return fabsf(v) > Largest<T>::value ? copysignf(Largest<T>::value, v) : v;  // (a NaN step stays NaN)
}

template <typename T, bool E5>
__global__ void __launch_bounds__(256) k_dequant_f8(long long total, int bpr, int EP, int C, const uint8_t* q,
                                                    const uint8_t* e, T* x) {
  pdl_enter();
  const int l = threadIdx.x & 7;
  const long long step = (long long)gridDim.x * 32;
  for (long long b = (long long)blockIdx.x * 32 + (threadIdx.x >> 3); b < total; b += step) {
    const long long row = total < (1ll << 31) ? (long long)((uint32_t)b / (uint32_t)bpr) : b / bpr;
    const int blk = (int)(b - row * bpr);
    const float s = block_step(e[(size_t)row * EP + blk]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c0 = blk * 128 + 64 * h + 8 * l;
      const uint2 w = *reinterpret_cast<const uint2*>(q + (size_t)row * (bpr * 128) + c0);
      float2 v[4] = {from_f8x2<E5>(w.x & 0xffffu), from_f8x2<E5>(w.x >> 16), from_f8x2<E5>(w.y & 0xffffu),
                     from_f8x2<E5>(w.y >> 16)};
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = make_float2(read_back<T>(v[i].x, s), read_back<T>(v[i].y, s));
      store_chunk<T, 32, true>(x + (size_t)row * C, c0, C, v);
    }
  }
}
// Other rows: a warp takes 256 columns, a lane columns lane, lane + 32, ..., so that
// neighbours write one run (65,536 rows of 1001 16-bit columns 53 us; with eight
// neighbouring columns a lane, as above, 204).
template <typename T, bool E5>
__global__ void __launch_bounds__(256) k_dequant_f8_odd(long long total, int bpr, int EP, int wpr, int C, const uint8_t* q,
                                                        const uint8_t* e, T* x) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const long long step = (long long)gridDim.x * 8;
  for (long long b = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); b < total; b += step) {
    const long long row = total < (1ll << 31) ? (long long)((uint32_t)b / (uint32_t)wpr) : b / wpr;
    const int c0 = (int)(b - row * wpr) * 256;
    const uint8_t* p = q + (size_t)row * (bpr * 128);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = c0 + 32 * i < C ? p[c0 + 32 * i + lane] : 0u;
    float s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) s[h] = c0 + 128 * h < C ? block_step(e[(size_t)row * EP + c0 / 128 + h]) : 0.f;
    float2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = from_f8x2<E5>(w[2 * i] | w[2 * i + 1] << 8);
      v[i] = make_float2(read_back<T>(v[i].x, s[i / 2]), read_back<T>(v[i].y, s[i / 2]));
    }
    store_chunk<T, 32, false>(x + (size_t)row * C, c0 + lane, C, v);
  }
}

// ---------------------------------------------------------------- rows and columns
// A CTA takes tiles of 128 rows of a group by 128 columns through shared memory; the
// grid is what fits at once.  Row pass: eight lanes a row, straight from the loads (the
// next tile's are issued before this one's column pass).
// Column pass: a thread two columns of 32 rows, held in registers between the
// maximum and the conversion; its words in a row of shared memory are its
// neighbours', without bank conflicts, and it writes whole 32-byte sectors.
// 32,768 sorted rows of 1280 bf16 columns 42 us, of 2560 with sums 82 (60 to 74% of the
// copy rate); neither DRAM nor issue is near its limit, so most likely a tile's two
// block barriers bound it.
constexpr int kTile = 128, kThreads = 256;

template <typename T> struct Pair2;
template <> struct Pair2<float> {
  using W = float2;
  static __device__ __forceinline__ float2 pair(W w) { return w; }
};
template <> struct Pair2<bf16> {
  using W = uint32_t;
  static __device__ __forceinline__ float2 pair(W w) { return bf16x2_to_f2(w); }
};
template <> struct Pair2<f16> {
  using W = uint32_t;
  static __device__ __forceinline__ float2 pair(W w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
};
// Bits of the larger magnitudes, kept per column of the pair: 16-bit types in
// the halves of m0, float32 in m0 and m1.
__device__ __forceinline__ void pair_top(float2 w, uint32_t& m0, uint32_t& m1) {
  m0 = max(m0, __float_as_uint(w.x) & 0x7fffffffu);
  m1 = max(m1, __float_as_uint(w.y) & 0x7fffffffu);
}
__device__ __forceinline__ void pair_top(uint32_t w, uint32_t& m0, uint32_t&) { m0 = __vmaxu2(m0, w & 0x7fff7fffu); }
template <typename T> __device__ __forceinline__ uint32_t half_bits(uint32_t h) {
  if (std::is_same<T, bf16>::value) return h << 16;
  return __float_as_uint(__half2float(__ushort_as_half((unsigned short)h)));
}
// 32 bytes to one sector, `whole` where p is on a boundary of 32 bytes (pointers are
// only known to be on one of 16); else as two vectors.
__device__ __forceinline__ void st_sector(uint8_t* p, const uint32_t (&o)[8], bool whole) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(o[0]), "r"(o[1]), "r"(o[2]),
                 "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// Resident CTAs an SM.
template <typename T, bool SUMS> constexpr int quant_blocks = sizeof(T) == 2 && !SUMS ? 3 : 2;
template <typename T, bool VEC, bool E5, bool SUMS>
__global__ void __launch_bounds__(kThreads, (quant_blocks<T, SUMS>))
    k_quant_groups(const QuantGroups a, const int ctiles, const int EP) {
  pdl_enter();
  extern __shared__ uint4 smem_q[];
  T* tile = reinterpret_cast<T*>(smem_q);  // [128][128]
  int* first = reinterpret_cast<int*>(tile + kTile * kTile);  // ragged: [G + 1] and [G + 1]
  int* before = first + a.G + 1;
  __shared__ __align__(8) uint32_t ctop[4][kTile];  // read and written in pairs
  __shared__ __align__(8) float csum[4][kTile];
  uint32_t blocks = (uint32_t)a.blocks;
  if (a.offsets) {
    ragged_scan<kThreads>(a.offsets, a.G, a.M, kTile, first, before);
    blocks = (uint32_t)before[a.G];
  }
  // Tiles go to the CTAs in turn, so that what is read at one time lies together.
  const uint32_t end = blocks * (uint32_t)ctiles;  // below 2^31
  uint32_t at = blockIdx.x;
  if (at >= end) return;
  // A block of rows: its group, its number there, its first row, how many it has.
  struct Block {
    int blk, g, b, rows;
    long long row0;
  };
  auto block_of = [&](int blk) {
    Block k;
    k.blk = blk;
    if (a.offsets) {
      k.g = ragged_group(before, a.G, blk);
      k.b = blk - before[k.g];
      k.rows = min(kTile, first[k.g + 1] - first[k.g] - k.b * kTile);
      k.row0 = first[k.g] + k.b * kTile;
    } else {
      const int per = (a.M + kTile - 1) / kTile;
      k.g = blk / per;
      k.b = blk - k.g * per;
      k.rows = min(kTile, a.M - k.b * kTile);
      k.row0 = (long long)k.b * kTile;
    }
    return k;
  };
  Block cur = block_of((int)(at / (uint32_t)ctiles));
  int ct = (int)at - cur.blk * ctiles;
  const int t = threadIdx.x, l = t & 7;
  const int cp = t & 63, quarter = t >> 6, r0 = quarter * 32;
  const bool whole = (reinterpret_cast<uintptr_t>(a.qt) & 31) == 0;  // what is added to qt below is a multiple of 32

  Chunk<T> k[4][2];  // rows t / 8 + 32 i, columns 8 l and 64 + 8 l
  const size_t x_step = 32 * (size_t)a.row_stride, q_pitch = (size_t)ctiles * kTile;
  const size_t q_step = 32 * (size_t)a.q_row * q_pitch, e_step = 32 * (size_t)a.q_row * EP;
  auto base = [&](const Block& k) {
    return static_cast<const T*>(a.x) + (size_t)k.g * a.group_stride + (size_t)k.row0 * a.row_stride;
  };
  auto load = [&](const Block& n, int c0) {
    const T* p = base(n) + (size_t)(t >> 3) * a.row_stride + c0;
    if (n.rows == kTile && c0 + kTile <= a.C) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) k[i][h] = *reinterpret_cast<const Chunk<T>*>(p + i * x_step + 64 * h + 8 * l);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          k[i][h] = load_chunk<T, 32, true>(p + i * x_step, 64 * h + 8 * l, (t >> 3) + 32 * i < n.rows ? a.C - c0 : 0);
    }
  };
  if constexpr (VEC) load(cur, ct * kTile);
  for (; at < end; at += gridDim.x) {
    const int c0 = ct * kTile, g = cur.g, b = cur.b, blk = cur.blk, rows = cur.rows;
    if constexpr (!VEC) {
      const T* x = base(cur);
      // A warp takes 16 rows, four at a time, neighbours' columns one run.
      const int lane = t & 31;
#pragma unroll 1
      for (int r = (t >> 5) * 4; r < kTile; r += kThreads / 8) {
        T v[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            v[i][j] = r + i < rows && c0 + 32 * j + lane < a.C ? x[(size_t)(r + i) * a.row_stride + c0 + 32 * j + lane] : from_f<T>(0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) tile[(r + i) * kTile + 32 * j + lane] = v[i][j];
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) k[i][h] = load_chunk<T, 32, true>(tile + ((t >> 3) + 32 * i) * kTile, 64 * h + 8 * l, kTile);
    }
    const size_t qr0 = (size_t)g * a.q_group + (size_t)(cur.row0 + (t >> 3)) * a.q_row;
    uint8_t* const pq = a.q + qr0 * q_pitch + 8 * l;
    uint8_t* const pe = a.e + qr0 * EP;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (t >> 3) + 32 * i;
      if constexpr (VEC) {
#pragma unroll
        for (int h = 0; h < 2; ++h) *reinterpret_cast<Chunk<T>*>(tile + r * kTile + 64 * h + 8 * l) = k[i][h];
      }
      if (!a.q) continue;
      uint32_t m = top_max<T>(top_of(k[i][0]), top_of(k[i][1]));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) m = top_max<T>(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (r >= rows) continue;
      const int e = block_exp<E5>(as_f32_bits<T>(m));
      const float inv = block_inv(e);
      uint8_t* const q = pq + i * q_step + c0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float2 v[4];
        to_pairs(k[i][h], v);
        *reinterpret_cast<uint2*>(q + 64 * h) = to_f8x8<E5>(v, inv);
      }
      if (l == 0) {
        uint8_t* ex = pe + i * e_step;
        ex[c0 / kTile] = (uint8_t)e;
        if (c0 + kTile >= a.C)
          for (int j = ctiles; j < EP; ++j) ex[j] = 0;
      }
    }
    __syncthreads();
    const uint32_t next = at + gridDim.x;
    if (next < end) {
      cur = block_of((int)(next / (uint32_t)ctiles));
      ct = (int)next - cur.blk * ctiles;
      if constexpr (VEC) load(cur, ct * kTile);
    }
    if (!SUMS && !a.qt) {
      __syncthreads();
      continue;
    }
    using W = typename Pair2<T>::W;
    const W* words = reinterpret_cast<const W*>(tile) + r0 * 64 + cp;  // [128][64]
    W w[32];
    uint32_t m0 = 0, m1 = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      w[i] = words[i * 64];
      pair_top(w[i], m0, m1);
    }
    if (sizeof(T) == 2) {
      m1 = half_bits<T>(m0 >> 16);
      m0 = half_bits<T>(m0 & 0xffffu);
    }
    *reinterpret_cast<uint2*>(&ctop[quarter][2 * cp]) = make_uint2(m0, m1);
    if constexpr (SUMS) {
      float2 sum = f2(0.f);
#pragma unroll
      for (int i = 0; i < 32; ++i) sum = add2(sum, Pair2<T>::pair(w[i]));
      *reinterpret_cast<float2*>(&csum[quarter][2 * cp]) = sum;
    }
    __syncthreads();  // (also: every word has been read before the next tile's are written)
    if constexpr (SUMS) {
      if (t < kTile && c0 + t < a.C) a.part[(size_t)blk * a.C + c0 + t] = (csum[0][t] + csum[1][t]) + (csum[2][t] + csum[3][t]);
      if (!a.qt) continue;
    }
    // Both columns at once.
    int ex2[2];
    float2 inv2;
    {
      const uint2 q0 = *reinterpret_cast<const uint2*>(&ctop[0][2 * cp]), q1 = *reinterpret_cast<const uint2*>(&ctop[1][2 * cp]),
                  q2 = *reinterpret_cast<const uint2*>(&ctop[2][2 * cp]), q3 = *reinterpret_cast<const uint2*>(&ctop[3][2 * cp]);
      ex2[0] = block_exp<E5>(max(max(q0.x, q1.x), max(q2.x, q3.x)));
      ex2[1] = block_exp<E5>(max(max(q0.y, q1.y), max(q2.y, q3.y)));
      inv2 = make_float2(block_inv(ex2[0]), block_inv(ex2[1]));
    }
    uint32_t o2[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float2 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = mul2(Pair2<T>::pair(w[4 * i + j]), inv2);
      }
      o2[0][i] = __byte_perm(to_f8x2<E5>(v[0].x, v[1].x), to_f8x2<E5>(v[2].x, v[3].x), 0x5410);
      o2[1][i] = __byte_perm(to_f8x2<E5>(v[0].y, v[1].y), to_f8x2<E5>(v[2].y, v[3].y), 0x5410);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = c0 + 2 * cp + h, e = ex2[h];
      uint32_t (&o)[8] = o2[h];
      if (e == kNaNExp) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = 0;
      }
      if (c >= a.C) continue;
      if (a.offsets) {
        // Block by block, [blocks][C][128], the exponents in fours, [blocks / 4][C][4].
        st_sector(a.qt + ((size_t)blk * a.C + c) * kTile + r0, o, whole);
        if (quarter == 0) a.et[((size_t)(blk >> 2) * a.C + c) * 4 + (blk & 3)] = (uint8_t)e;
      } else {
        const size_t cr = (size_t)g * a.C + c;
        st_sector(a.qt + cr * a.tp + (size_t)b * kTile + r0, o, whole);
        if (quarter == 0) {
          uint8_t* ex = a.et + cr * a.tep;
          ex[b] = (uint8_t)e;
          if ((b + 1) * kTile >= a.M)
            for (int i = b + 1; i < a.tep; ++i) ex[i] = 0;
        }
      }
    }
  }
}

// A group's column sums from its blocks' in their order; a thread a column.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_group_sums(const QuantGroups a) {
  pdl_enter();
  extern __shared__ int scan[];
  int* first = scan;
  int* before = first + a.G + 1;
  const int ct = (a.C + kThreads - 1) / kThreads;
  const int g = blockIdx.x / ct, c = (blockIdx.x - g * ct) * kThreads + threadIdx.x;
  long long b0, b1;
  if (a.offsets) {
    ragged_scan<kThreads>(a.offsets, a.G, a.M, kTile, first, before);
    b0 = before[g];
    b1 = before[g + 1];
  } else {
    const int per = (a.M + kTile - 1) / kTile;
    b0 = (long long)g * per;
    b1 = b0 + per;
  }
  if (c >= a.C) return;
  float s = 0.f;
#pragma unroll 8
  for (long long b = b0; b < b1; ++b) s += a.part[(size_t)b * a.C + c];
  static_cast<T*>(a.sums)[(size_t)g * a.C + c] = from_f<T>(s);
}

unsigned grid_of(long long units, int per_block) {
  const long long want = (units + per_block - 1) / per_block, most = (long long)sm_count() * 64;
  return (unsigned)(want < most ? want : most);
}

template <typename T, bool VEC, bool E5> cudaError_t quant(const QuantRows& a, cudaStream_t st) {
  const int bpr = f8_blocks(a.C), EP = f8_exps(a.C);
  const long long total = a.R * bpr;
  auto k = a.source ? k_quant_f8<T, VEC, E5, true> : k_quant_f8<T, VEC, E5, false>;
  return launch_k(k, dim3(grid_of(total, 32 * kBatch)), dim3(256), 0, st, 1, a, bpr, EP, total);
}
template <typename T, bool VEC, bool E5>
cudaError_t dequant(long long R, int C, const uint8_t* q, const uint8_t* e, void* x, cudaStream_t st) {
  const int bpr = f8_blocks(C), EP = f8_exps(C);
  if constexpr (VEC) {
    const long long total = R * bpr;
    return launch_k(k_dequant_f8<T, E5>, dim3(grid_of(total, 32)), dim3(256), 0, st, 1, total, bpr, EP, C, q, e, (T*)x);
  } else {
    const int wpr = (bpr + 1) / 2;
    const long long total = R * wpr;
    return launch_k(k_dequant_f8_odd<T, E5>, dim3(grid_of(total, 8)), dim3(256), 0, st, 1, total, bpr, EP, wpr, C, q, e, (T*)x);
  }
}
template <typename T, bool VEC, bool E5> cudaError_t quant_groups(const QuantGroups& a, cudaStream_t st) {
  const int ctiles = f8_blocks(a.C);
  const int smem = kTile * kTile * (int)sizeof(T) + (a.offsets ? 2 * (a.G + 1) * (int)sizeof(int) : 0);
  auto k = a.part ? k_quant_groups<T, VEC, E5, true> : k_quant_groups<T, VEC, E5, false>;
  cudaError_t e = allow_smem(k, smem, kTile * kTile * (int)sizeof(T) + 2 * (kMaxExperts + 1) * (int)sizeof(int));
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)a.blocks * ctiles, fit = (long long)sm_count() * (a.part ? quant_blocks<T, true> : quant_blocks<T, false>);
  return launch_k(k, dim3((unsigned)(tiles < fit ? tiles : fit)), dim3(kThreads), smem, st, 1, a, ctiles, f8_exps(a.C));
}

#define BY_FORM(f, T, C, fmt, ...)                                                         \
  (rows_aligned(C, sizeof(T)) ? (fmt ? f<T, true, true>(__VA_ARGS__) : f<T, true, false>(__VA_ARGS__)) \
                              : (fmt ? f<T, false, true>(__VA_ARGS__) : f<T, false, false>(__VA_ARGS__)))

}  // namespace

cudaError_t launch_quant_f8(const QuantRows& a, cudaStream_t st) {
  RMX_BY_DTYPE(a.dtype, return BY_FORM(quant, T, a.C, a.format, a, st))
}
cudaError_t launch_dequant_f8(long long R, int C, int dtype, int format, const uint8_t* q, const uint8_t* e, void* x,
                              cudaStream_t st) {
  RMX_BY_DTYPE(dtype, return BY_FORM(dequant, T, C, format, R, C, q, e, x, st))
}
cudaError_t launch_quant_f8_groups(const QuantGroups& a, cudaStream_t st) {
  RMX_BY_DTYPE(a.dtype, return BY_FORM(quant_groups, T, a.C, a.format, a, st))
}
cudaError_t launch_quant_f8_sums(const QuantGroups& a, cudaStream_t st) {
  const int smem = a.offsets ? 2 * (a.G + 1) * (int)sizeof(int) : 0;
  const unsigned grid = (unsigned)(a.G * ((a.C + kThreads - 1) / kThreads));
  RMX_BY_DTYPE(a.dtype, return launch_k(k_group_sums<T>, dim3(grid), dim3(kThreads), smem, st, 1, a))
}

}  // namespace rmx
