// Row passes of the 8-bit operators: RMS norm with the residual's addition
// and an int8 output, row quantisation, 8-bit checkpoints, and the weights'
// quantisation.
//
// All are bound by HBM traffic: each reads every input once and writes every
// output once, a row held in registers between its reduction and its output.
// A row belongs to 8 or 16 lanes, or to one, four or sixteen warps, whichever
// hold it in at most five blocks of eight columns a lane.
//
// Measured (GB300, bf16): x + r, norm and quantisation of 65536 x 1280 with h
// written 86 us, 6.3 TB/s to HBM, 94% of the measured copy rate; read back
// 36 us; a checkpoint of it packed in 34 us and read back in 37 (6 TB/s).

#include <float.h>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "q8.h"
#include "q8_rows.cuh"

namespace rmx {
namespace {

// ---------------------------------------------------------------- RMS norm forward
// n = h * rstd * gamma with h = x + r: rstd needs one sum over the row, the
// int8 scale the row's largest |n| = rstd * max|h * gamma|, so both come from
// one reduction, and q = round(h * gamma * 127 / max|h * gamma|) needs no
// rstd at all.
template <typename T, int L, int W, int NCH, bool VEC>
__global__ void __launch_bounds__(W * L < 256 ? 256 : W * L, W * L < 256 ? 2 : 1) k_rows_fwd(const RowsFwd a) {
  pdl_enter();
  constexpr int TH = W * L < 256 ? 256 : W * L, RPB = TH / (W * L);
  __shared__ uint32_t red[W > 1 ? RPB * 4 * W : 1];
  const int lane = threadIdx.x & (L - 1), rib = threadIdx.x / (W * L), w = (threadIdx.x - rib * (W * L)) / L;
  const float inv_n = 1.f / (float)a.C;
  int slot = 0;
  Chunk<T> g[NCH];
  if (a.norm) {
#pragma unroll
    for (int j = 0; j < NCH; ++j)
      g[j] = load_chunk<T, L, VEC>(static_cast<const T*>(a.gamma), col0<L, VEC>(w + j * W, lane), a.C);
  }
  for (long long base = (long long)blockIdx.x * RPB; base < a.R; base += (long long)gridDim.x * RPB) {
    const long long row = base + rib;
    const bool live = row < a.R;
    const size_t at = (size_t)(live ? row : 0) * a.C;
    const int C = live ? a.C : 0;
    float2 v[NCH][4];
    Chunk<T> cx[NCH], cr[NCH];
#pragma unroll
    for (int j = 0; j < NCH; ++j) cx[j] = load_chunk<T, L, VEC>(static_cast<const T*>(a.x) + at, col0<L, VEC>(w + j * W, lane), C);
    if (a.r) {
#pragma unroll
      for (int j = 0; j < NCH; ++j)
        cr[j] = load_chunk<T, L, VEC>(static_cast<const T*>(a.r) + at, col0<L, VEC>(w + j * W, lane), C);
    }
    float2 ss = f2(0.f);
    float am = 0.f;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      to_pairs(cx[j], v[j]);
      if (a.r) {
        float2 r[4];
        to_pairs(cr[j], r);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = add2(v[j][i], r[i]);
      }
      if (a.h) store_chunk<T, L, VEC>(static_cast<T*>(a.h) + at, col0<L, VEC>(w + j * W, lane), C, v[j]);
      if (a.norm) {
        float2 gm[4];
        to_pairs(g[j], gm);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ss = fma2(v[j][i], v[j][i], ss);
          v[j][i] = mul2(v[j][i], gm[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) am = max_abs(am, v[j][i]);
    }
    float sum = ss.x + ss.y;
    uint32_t top = __float_as_uint(am);  // NaN above infinity above every number
    row_reduce<W, L>(sum, top, red, rib, w, slot);
    if (!live) continue;
    const float rstd = a.norm ? rsqrtf(fmaf(sum, inv_n, a.eps)) : 1.f;
    if (a.rstd && w == 0 && lane == 0) a.rstd[row] = rstd;
    if (a.y) {
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        float2 o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = mul2(v[j][i], f2(rstd));
        store_chunk<T, L, VEC>(static_cast<T*>(a.y) + at, col0<L, VEC>(w + j * W, lane), C, o);
      }
    }
    if (a.q) {
      // A row that holds an infinity or a NaN has no scale: NaN, and zeros.  Its
      // largest value is mx * rstd: rstd is infinite where the squares' mean
      // (and eps) is zero, and zero where it is past float32.
      float mx = __uint_as_float(top);
      const float largest = mx * rstd;
      const bool fine = fabsf(largest) <= FLT_MAX;
      if (w == 0 && lane == 0) a.scale[row] = fine ? fminf(mx / 127.f * rstd, kMaxScale) : __uint_as_float(0x7fc00000u);
      if (mx < 0x1p-100f) {
        // Tiny rows are lifted so that 127 / max stays finite.
        mx *= 0x1p100f;
#pragma unroll
        for (int j = 0; j < NCH; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[j][i] = mul2(v[j][i], f2(0x1p100f));
      }
      const float mul = largest > 0.f ? 127.f / mx : 0.f;
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        float2 t[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = round2(v[j][i], mul);
        store_bytes<L, VEC>(a.q + (size_t)row * a.P, col0<L, VEC>(w + j * W, lane), a.P, t, fine);
      }
    }
  }
}

// A row's threads, by its length.  Rows of 40 columns: one row a warp 526 us,
// 8 lanes a row 123 us (1,000,000 rows, with the read back); of 8192: four warps
// with eight blocks each 172 us, sixteen with two 135 us (8000 rows).  Up to 1280
// columns one warp holds a row, without a barrier between its threads.  Above,
// four warps with room for 4096 columns each pay for the places they leave empty
// and for the barrier: of as many elements, rows of 1280 take 88 us, 1288 189,
// 1536 162, 2048 132, 2560 115, 4096 94.
template <typename T, bool VEC>
cudaError_t rows_fwd(const RowsFwd& a, cudaStream_t st) {
  auto go = [&](auto k, int threads_of_row) {
    const int th = threads_of_row < 256 ? 256 : threads_of_row, rpb = th / threads_of_row;
    const long long want = (a.R + rpb - 1) / rpb;
    const long long most = (long long)sm_count() * 16;
    return launch_k(k, dim3((unsigned)(want < most ? want : most)), dim3(th), 0, st, 1, a);
  };
  if (a.P <= 64) return go(k_rows_fwd<T, 8, 1, 1, VEC>, 8);
  if (a.P <= 128) return go(k_rows_fwd<T, 16, 1, 1, VEC>, 16);
  if (a.P <= 256) return go(k_rows_fwd<T, 32, 1, 1, VEC>, 32);
  if (a.P <= 512) return go(k_rows_fwd<T, 32, 1, 2, VEC>, 32);
  if (a.P <= 1280) return go(k_rows_fwd<T, 32, 1, 5, VEC>, 32);
  if (a.P <= 4096) return go(k_rows_fwd<T, 32, 4, 4, VEC>, 128);
  if (a.P <= 8192) return go(k_rows_fwd<T, 32, 16, 2, VEC>, 512);
  return go(k_rows_fwd<T, 32, 16, 4, VEC>, 512);
}

// ---------------------------------------------------------------- element passes
// A flat run over the blocks of 8 * L columns of padded int8 rows.
struct Flat {
  int C, P, bpr;         // blocks per row
  long long total;       // rows * bpr
};
// L lanes take kBatch neighbouring blocks at a time, all loads first.
constexpr int kBatch = 4;
// Row and block of a flat position; one division for a batch.
struct Place {
  long long row;
  int blk;
};
__device__ __forceinline__ Place place_of(const Flat& f, long long b) {
  Place p;
  if (f.total < (1ll << 31)) p.row = (uint32_t)b / (uint32_t)f.bpr;
  else p.row = b / f.bpr;
  p.blk = (int)(b - p.row * f.bpr);
  return p;
}
__device__ __forceinline__ void next_place(const Flat& f, Place& p) {
  const bool wrap = p.blk + 1 == f.bpr;
  p.blk = wrap ? 0 : p.blk + 1;
  p.row += wrap ? 1 : 0;
}

// Bits of the largest magnitude of a group of 32: the eight values of this lane
// and of the three beside it.  16-bit types compare as integers two at a time,
// without the sign; NaN comes out above infinity above every number.
__device__ __forceinline__ uint32_t group_max(const Chunk<float>& k) {
  float am = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) am = max_abs(am, make_float2(k.v[i], k.v[i + 1]));
  uint32_t u = __float_as_uint(am);
  u = max(u, __shfl_xor_sync(0xffffffffu, u, 1));
  return max(u, __shfl_xor_sync(0xffffffffu, u, 2));
}
template <typename T> __device__ __forceinline__ uint32_t group_max(const Chunk<T>& k) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&k);
  uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const uint32_t top = max(m >> 16, m & 0xffffu);
  if constexpr (std::is_same<T, bf16>::value) return top << 16;
  return __float_as_uint(__half2float(__ushort_as_half((unsigned short)top)));
}
// Eight values of a group as int8, and the group's exponent.
template <typename T> __device__ __forceinline__ uint2 pack_group(const Chunk<T>& k, int& ex) {
  const uint32_t u = group_max(k);
  ex = ckpt_exp<T>(u);
  const float inv = pow2(-ex);  // exact, and so is the scaling: the only rounding is to the integer
  float2 v[4];
  to_pairs(k, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = round2(v[i], inv);
  if (__uint_as_float(u) * inv >= 127.5f) {
    // 128 steps: the upper clamp, and exactly 127.5.
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i].x = fminf(fmaxf(v[i].x, kRound - 127.f), kRound + 127.f);
      v[i].y = fminf(fmaxf(v[i].y, kRound - 127.f), kRound + 127.f);
    }
  }
  return ex == kCkptNaN ? make_uint2(0, 0) : low_bytes(v);
}

// Rows that are a whole number of groups lie in memory as one run of groups,
// and so do their exponents: a checkpoint of `total` blocks of 256 columns,
// whatever the rows' length.  Addresses are one base and constants, a third of
// the general form's instructions, which bound it: pack and read back of
// 65536 x 1280 16-bit values take 92 us in that form, 75 us in this.
template <typename T>
__global__ void __launch_bounds__(256) k_ckpt_pack_flat(long long total, const T* x, int8_t* q, int8_t* e) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const long long b0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * kBatch;
  if (b0 >= total) return;
  const T* xp = x + b0 * 256 + lane * 8;
  int8_t* qp = q + b0 * 256 + lane * 8;
  int8_t* ep = e + b0 * 8 + (lane >> 2);
  auto store = [&](const Chunk<T>& k, int j) {
    int ex;
    *reinterpret_cast<uint2*>(qp + j * 256) = pack_group(k, ex);
    if ((lane & 3) == 0) ep[j * 8] = (int8_t)ex;
  };
  if (b0 + kBatch <= total) {
    Chunk<T> k[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) k[j] = load_chunk<T, 32, true>(xp + j * 256, 0, 8);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) store(k[j], j);
  } else {
    for (int j = 0; b0 + j < total; ++j) store(load_chunk<T, 32, true>(xp + j * 256, 0, 8), j);
  }
}
// The same for q8 rows of a whole number of blocks (f.bpr of them), each block
// with its row's scale (65536 x 1280: 43 us in the general form, 36 in this).
template <typename T>
__global__ void __launch_bounds__(256) k_dequant_flat(const Flat f, const int8_t* q, const float* scale, T* x) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const long long b0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * kBatch;
  if (b0 >= f.total) return;
  const int8_t* qp = q + b0 * 256 + lane * 8;
  T* xp = x + b0 * 256 + lane * 8;
  Place p = place_of(f, b0);
  auto store = [&](uint2 b, float s, int j) {
    float2 v[4];
    biased(b, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(add2(v[i], f2(-kBias)), f2(s));
    store_chunk<T, 32, true>(xp + j * 256, 0, 8, v);
  };
  if (b0 + kBatch <= f.total) {
    uint2 b[kBatch];
    float s[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) b[j] = *reinterpret_cast<const uint2*>(qp + j * 256);
#pragma unroll
    for (int j = 0; j < kBatch; ++j, next_place(f, p)) s[j] = scale[p.row];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) store(b[j], s[j], j);
  } else {
    for (int j = 0; b0 + j < f.total; ++j, next_place(f, p))
      store(*reinterpret_cast<const uint2*>(qp + j * 256), scale[p.row], j);
  }
}
template <typename T>
__global__ void __launch_bounds__(256) k_unpack_flat(long long total, const int8_t* q, const int8_t* e, T* x) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const long long b0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * kBatch;
  if (b0 >= total) return;
  const int8_t* qp = q + b0 * 256 + lane * 8;
  const int8_t* ep = e + b0 * 8 + (lane >> 2);
  T* xp = x + b0 * 256 + lane * 8;
  auto store = [&](uint2 b, int ex, int j) {
    const float s = ckpt_step(ex);
    float2 v[4];
    biased(b, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(add2(v[i], f2(-kBias)), f2(s));
    store_chunk<T, 32, true>(xp + j * 256, 0, 8, v);
  };
  if (b0 + kBatch <= total) {
    uint2 b[kBatch];
    int ex[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) b[j] = *reinterpret_cast<const uint2*>(qp + j * 256);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) ex[j] = ep[j * 8];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) store(b[j], ex[j], j);
  } else {
    for (int j = 0; b0 + j < total; ++j) store(*reinterpret_cast<const uint2*>(qp + j * 256), ep[j * 8], j);
  }
}

// The 32 columns of a group are four neighbouring lanes (VEC) or 32 / L
// elements of each of the L lanes.
template <typename T, int L, bool VEC>
__global__ void __launch_bounds__(256) k_ckpt_pack(const Flat f, const T* x, int8_t* q, int8_t* e) {
  pdl_enter();
  const int lane = threadIdx.x & (L - 1);
  const long long step = (long long)gridDim.x * (256 / L) * kBatch;
  const int groups = f.P / kQ8Group;
  // Whole warps stay in the loop together: the shuffles below take every lane.
  for (long long w0 = ((long long)blockIdx.x * (256 / L) + (threadIdx.x >> 5) * (32 / L)) * kBatch; w0 < f.total;
       w0 += step) {
    const long long b0 = w0 + ((threadIdx.x & 31) / L) * kBatch;
    Chunk<T> k[kBatch];
    long long row[kBatch];
    int c0[kBatch];
    Place p = place_of(f, b0);
#pragma unroll
    for (int j = 0; j < kBatch; ++j, next_place(f, p)) {
      const bool live = b0 + j < f.total;
      row[j] = live ? p.row : 0;
      c0[j] = col0<L, VEC>(p.blk, lane);
      k[j] = load_chunk<T, L, VEC>(x + row[j] * f.C, c0[j], live ? f.C : 0);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const bool live = b0 + j < f.total;
      if constexpr (VEC) {
        int ex;
        const uint2 b = pack_group(k[j], ex);
        if (live && c0[j] < f.P) *reinterpret_cast<uint2*>(q + row[j] * f.P + c0[j]) = b;
        if (live && (lane & 3) == 0 && c0[j] < f.P) e[row[j] * groups + c0[j] / kQ8Group] = (int8_t)ex;
      } else {
        constexpr int PER = 32 / L;  // elements of a lane in a group
        float2 v[4];
        to_pairs(k[j], v);
        // Lane g works out group g's exponent, for all (40000 x 1001: 75 -> 56 us).
        uint32_t top = 0;
#pragma unroll
        for (int g = 0; g < L / 4; ++g) {
          uint32_t u = 0;
#pragma unroll
          for (int i = g * PER; i < (g + 1) * PER; ++i)
            u = max(u, __float_as_uint(i & 1 ? v[i / 2].y : v[i / 2].x) & 0x7fffffffu);
          u = lanes_max<L>(u);
          top = lane == g ? u : top;
        }
        const int mine = ckpt_exp<T>(top);
        const float inv = pow2(-mine);  // 0 for a group without a scale
        const bool rare = mine == kCkptNaN || __uint_as_float(top) * inv >= 127.5f;
        const bool any = __any_sync(0xffffffffu, rare);
#pragma unroll
        for (int g = 0; g < L / 4; ++g) {
          const float scale = __shfl_sync(0xffffffffu, inv, g, L);
#pragma unroll
          for (int i = g * PER; i < (g + 1) * PER; ++i) {
            float& t = i & 1 ? v[i / 2].y : v[i / 2].x;
            t = fmaf(t, scale, kRound);
            if (any) {
              // 128 steps (as in pack_group), or no scale: zeros.
              t = scale == 0.f ? kRound : fminf(fmaxf(t, kRound - 127.f), kRound + 127.f);
            }
          }
        }
        store_bytes<L, VEC>(q + row[j] * f.P, c0[j], live ? f.P : 0, v, true);
        const int grp = (c0[j] - lane) / kQ8Group + lane;
        if (live && lane < L / 4 && grp < groups) e[row[j] * groups + grp] = (int8_t)mine;
      }
    }
  }
}

// CK: checkpoint (one exponent per group), else one scale per row.  The output
// rows have `pitch` elements; columns C .. pitch-1 become zeros.
template <typename T, bool CK, int L, bool VEC>
__global__ void __launch_bounds__(256) k_unpack(const Flat f, const int8_t* q, const void* s, T* x, int pitch) {
  pdl_enter();
  const int lane = threadIdx.x & (L - 1);
  const long long step = (long long)gridDim.x * (256 / L) * kBatch;
  const int groups = f.P / kQ8Group;
  for (long long b0 = ((long long)blockIdx.x * (256 / L) + threadIdx.x / L) * kBatch; b0 < f.total; b0 += step) {
    uint2 b[kBatch], ex[kBatch];
    float sc[kBatch];
    long long row[kBatch];
    int c0[kBatch];
    Place p = place_of(f, b0);
#pragma unroll
    for (int j = 0; j < kBatch; ++j, next_place(f, p)) {
      const bool live = b0 + j < f.total;
      row[j] = live ? p.row : 0;
      c0[j] = col0<L, VEC>(p.blk, lane);
      b[j] = load_bytes<L, VEC>(q + row[j] * f.P, c0[j], live ? f.P : 0);
      sc[j] = 0.f;
      ex[j] = make_uint2(0, 0);
      if (!live) continue;
      if (!CK) sc[j] = static_cast<const float*>(s)[row[j]];
      else if (!VEC) ex[j] = load_exps<L>(static_cast<const int8_t*>(s) + row[j] * groups, p.blk, groups);
      else if (c0[j] < f.P) sc[j] = ckpt_step(static_cast<const int8_t*>(s)[row[j] * groups + c0[j] / kQ8Group]);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (b0 + j >= f.total) break;
      float2 v[4];
      biased(b[j], v);
      if (CK && !VEC) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float& t = i & 1 ? v[i / 2].y : v[i / 2].x;
          t = (t - kBias) * ckpt_step(exp_of<L>(ex[j], i));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = mul2(add2(v[i], f2(-kBias)), f2(sc[j]));
      }
      if (pitch > f.C && c0[j] + (VEC ? 8 : 7 * L + 1) > f.C) {
        // Columns C .. pitch - 1: zeros whatever the padding holds (a NaN
        // scale would not leave them so).
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col<L, VEC>(c0[j], i) >= f.C) (i & 1 ? v[i / 2].y : v[i / 2].x) = 0.f;
      }
      store_chunk<T, L, VEC>(x + row[j] * pitch, c0[j], pitch, v);
    }
  }
}

// Lanes for a block: as few as hold a short row (a checkpoint of 1,000,000 rows
// of 40 columns, both ways: a warp a row 231 us, 8 lanes a row 68 us).
int lanes_of(int C) { return q8_pitch(C) <= 64 ? 8 : q8_pitch(C) <= 128 ? 16 : 32; }
Flat flat_of(long long R, int C, int lanes) {
  Flat f;
  f.C = C;
  f.P = q8_pitch(C);
  f.bpr = (f.P + 8 * lanes - 1) / (8 * lanes);
  f.total = R * f.bpr;
  return f;
}
dim3 flat_grid(const Flat& f, int lanes) {
  const long long per = (long long)(256 / lanes) * kBatch;
  const long long want = (f.total + per - 1) / per, most = (long long)sm_count() * 16;
  return dim3((unsigned)(want < most ? want : most));
}
template <typename T, int L>
cudaError_t ckpt_pack(long long R, int C, const T* x, int8_t* q, int8_t* e, cudaStream_t st) {
  const Flat f = flat_of(R, C, L);
  return launch_k(rows_aligned(C, sizeof(T)) ? k_ckpt_pack<T, L, true> : k_ckpt_pack<T, L, false>, flat_grid(f, L),
                  dim3(256), 0, st, 1, f, x, q, e);
}
template <typename T, bool CK, int L>
cudaError_t unpack_rows(long long R, int C, const int8_t* q, const void* s, T* x, int pitch, cudaStream_t st) {
  const Flat f = flat_of(R, C, L);
  return launch_k(rows_aligned(pitch, sizeof(T)) ? k_unpack<T, CK, L, true> : k_unpack<T, CK, L, false>,
                  flat_grid(f, L), dim3(256), 0, st, 1, f, q, s, x, pitch);
}

// ---------------------------------------------------------------- column sums
// Column sums of a float32 [R][J] matrix.  A thread owns V neighbouring columns
// (a 16-byte vector, or one element where rows are no whole number of vectors)
// and sums the rows of slice blockIdx.y in order; with one slice it stores the
// result, else the slices' partials are summed by launch_colsums.
template <int V>
__global__ void __launch_bounds__(256) k_colpart(long long R, long long J, int slices, const float* x, float* part,
                                                 float* out) {
  pdl_enter();
  const long long j = ((long long)blockIdx.x * 256 + threadIdx.x) * V;
  if (j >= J) return;
  const long long r0 = R * blockIdx.y / slices, r1 = R * (blockIdx.y + 1) / slices;
  float s[V] = {};
#pragma unroll 8
  for (long long r = r0; r < r1; ++r) {
    float v[V];
    if constexpr (V == 1) v[0] = x[r * J + j];
    else load_vec(x + r * J + j, v);
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] += v[i];
  }
  float* to = slices == 1 ? out : part + blockIdx.y * J;
#pragma unroll
  for (int i = 0; i < V; ++i) to[j + i] = s[i];
}

// ---------------------------------------------------------------- weights
// Block: 32 channels of one group.  First the channels' largest magnitudes
// over K, then 32 x 32 tiles transposed through shared memory.
template <typename T>
__global__ void __launch_bounds__(256) k_weight_q8(int K, int N, int P, const T* w, int8_t* q, float* scale) {
  pdl_enter();
  __shared__ float tile[32][33];
  __shared__ uint32_t mx[8][32];
  const int g = blockIdx.y, n0 = blockIdx.x * 32;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const T* wg = w + (size_t)g * K * N;
  uint32_t am = 0;
  if (n0 + tx < N)
    for (int k = ty; k < K; k += 8) am = max(am, __float_as_uint(to_f(wg[(size_t)k * N + n0 + tx])) & 0x7fffffffu);
  mx[ty][tx] = am;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) am = max(am, mx[i][tx]);
  if (ty == 0 && n0 + tx < N)
    scale[(size_t)g * N + n0 + tx] = am < kInfBits ? fminf(__uint_as_float(am) / 127.f, kMaxScale) : __uint_as_float(0x7fc00000u);
  const bool fine = am < kInfBits;
  const float lift = __uint_as_float(am) < 0x1p-100f ? 0x1p100f : 1.f;
  const float mul = am && fine ? 127.f / (__uint_as_float(am) * lift) : 0.f;
  for (int k0 = 0; k0 < P; k0 += 32) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
      const int k = k0 + ty + i;
      // thread (ty, tx) holds channel n0 + tx: quantised here, transposed in the tile
      const bool in = k < K && n0 + tx < N && fine;
      tile[ty + i][tx] = in ? (to_f(wg[(size_t)k * N + n0 + tx]) * lift) * mul : 0.f;
    }
    __syncthreads();
    // 256 threads write 32 channels x 8 words of 4 columns.
    const int n = threadIdx.x >> 3, kk = (threadIdx.x & 7) * 4;
    if (n0 + n < N) {
      float2 t[4] = {};
      t[0] = make_float2(tile[kk][n] + kRound, tile[kk + 1][n] + kRound);
      t[1] = make_float2(tile[kk + 2][n] + kRound, tile[kk + 3][n] + kRound);
      *reinterpret_cast<uint32_t*>(q + ((size_t)g * N + n0 + n) * P + k0 + kk) = low_bytes(t).x;
    }
  }
}

}  // namespace

cudaError_t launch_rows_fwd(const RowsFwd& a, cudaStream_t st) {
  RMX_BY_DTYPE(a.dtype, return rows_aligned(a.C, sizeof(T)) ? rows_fwd<T, true>(a, st) : rows_fwd<T, false>(a, st))
}

cudaError_t launch_dequant_rows(long long R, int C, int dtype, const int8_t* q, const float* scale, void* x,
                                cudaStream_t st) {
  if (C % 256 == 0 && R * (C / 256) < (1ll << 35)) {
    const Flat f = flat_of(R, C, 32);
    RMX_BY_DTYPE(dtype, return launch_k(k_dequant_flat<T>, dim3((unsigned)((f.total + 8 * kBatch - 1) / (8 * kBatch))),
                                        dim3(256), 0, st, 1, f, q, scale, static_cast<T*>(x)))
  }
  const int L = lanes_of(C);
  RMX_BY_DTYPE(dtype, {
    T* xt = static_cast<T*>(x);
    return L == 8    ? unpack_rows<T, false, 8>(R, C, q, scale, xt, C, st)
           : L == 16 ? unpack_rows<T, false, 16>(R, C, q, scale, xt, C, st)
                     : unpack_rows<T, false, 32>(R, C, q, scale, xt, C, st);
  })
}

// Whether a checkpoint can be taken as one run of 256-column blocks.
static bool ckpt_flat(long long R, int C) { return C % kQ8Group == 0 && R * C % 256 == 0 && R * C / 256 < (1ll << 35); }
static dim3 ckpt_flat_grid(long long R, int C) {
  return dim3((unsigned)((R * C / 256 + 8 * kBatch - 1) / (8 * kBatch)));
}

cudaError_t launch_ckpt_pack(long long R, int C, int dtype, const void* x, int8_t* q, int8_t* e, cudaStream_t st) {
  if (ckpt_flat(R, C)) {
    RMX_BY_DTYPE(dtype, return launch_k(k_ckpt_pack_flat<T>, ckpt_flat_grid(R, C), dim3(256), 0, st, 1, R * C / 256,
                                        static_cast<const T*>(x), q, e))
  }
  const int L = lanes_of(C);
  RMX_BY_DTYPE(dtype, {
    const T* xt = static_cast<const T*>(x);
    return L == 8    ? ckpt_pack<T, 8>(R, C, xt, q, e, st)
           : L == 16 ? ckpt_pack<T, 16>(R, C, xt, q, e, st)
                     : ckpt_pack<T, 32>(R, C, xt, q, e, st);
  })
}

cudaError_t launch_ckpt_unpack(long long R, int C, int dtype, const int8_t* q, const int8_t* e, void* x, int pitch,
                               cudaStream_t st) {
  if (pitch == C && ckpt_flat(R, C)) {
    RMX_BY_DTYPE(dtype, return launch_k(k_unpack_flat<T>, ckpt_flat_grid(R, C), dim3(256), 0, st, 1, R * C / 256, q, e,
                                        static_cast<T*>(x)))
  }
  const int L = lanes_of(C);
  RMX_BY_DTYPE(dtype, {
    T* xt = static_cast<T*>(x);
    return L == 8    ? unpack_rows<T, true, 8>(R, C, q, e, xt, pitch, st)
           : L == 16 ? unpack_rows<T, true, 16>(R, C, q, e, xt, pitch, st)
                     : unpack_rows<T, true, 32>(R, C, q, e, xt, pitch, st);
  })
}

// Slices of rows: enough blocks for eight a SM, at least 16 rows each.
int colpart_slices(long long R, long long J) {
  const long long V = J % 4 == 0 ? 4 : 1, blocks = (J / V + 255) / 256;
  long long s = (8ll * sm_count() + blocks - 1) / blocks;
  if (s > R / 16) s = R / 16;
  return (int)(s < 1 ? 1 : s > kColpartMax ? kColpartMax : s);
}
cudaError_t launch_colpart(long long R, long long J, const float* x, float* part, float* out, cudaStream_t st) {
  const bool vec = J % 4 == 0;
  const int s = colpart_slices(R, J);
  const dim3 grid((unsigned)((J / (vec ? 4 : 1) + 255) / 256), s);
  return launch_k(vec ? k_colpart<4> : k_colpart<1>, grid, dim3(256), 0, st, 1, R, J, s, x, part, out);
}

cudaError_t launch_weight_q8(int G, int K, int N, int dtype, const void* w, int8_t* q, float* scale,
                             cudaStream_t st) {
  const dim3 grid((N + 31) / 32, G);
  RMX_BY_DTYPE(dtype, return launch_k(k_weight_q8<T>, grid, dim3(256), 0, st, 1, K, N, q8_pitch(K),
                                      static_cast<const T*>(w), q, scale))
}

}  // namespace rmx
