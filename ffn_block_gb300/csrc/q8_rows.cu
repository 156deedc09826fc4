// Row passes of the 8-bit operators: RMS norm with the residual's addition
// and an int8 output, row quantisation, 8-bit checkpoints, the RMS norm
// backward, and the weights' quantisation.
//
// All are bound by HBM traffic: each reads every input once and writes every
// output once, a row held in registers between its reduction and its output.
// A thread owns chunks of 8 consecutive columns; a row belongs to 32, 128 or
// 512 threads, whichever holds it in at most 5 chunks a thread.

#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "q8.h"

namespace rmx {
namespace {

constexpr uint32_t kAbs = 0x7fffffffu;
constexpr uint32_t kInfBits = 0x7f800000u;

// ---------------------------------------------------------------- chunks
// Eight storage-type values of a row, columns c .. c+7, as loaded (16-bit
// types: 16 bytes).  Columns past C read as zero.  vec: rows start on
// 16-byte boundaries.
template <typename T> struct alignas(16) Chunk {
  T v[8];
};
template <typename T>
__device__ __forceinline__ Chunk<T> load_chunk(const T* row, int c, int C, bool vec) {
  Chunk<T> k;
  uint4* d = reinterpret_cast<uint4*>(&k);
  if (vec && c + 8 <= C) {
    const uint4* s = reinterpret_cast<const uint4*>(row + c);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) d[i] = s[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) k.v[i] = c + i < C ? row[c + i] : from_f<T>(0.f);
  }
  return k;
}
template <typename T>
__device__ __forceinline__ void store_chunk(T* row, int c, int C, bool vec, const float (&f)[8]) {
  if (vec && c + 8 <= C) {
    Chunk<T> k;
#pragma unroll
    for (int i = 0; i < 8; ++i) k.v[i] = from_f<T>(f[i]);
    const uint4* s = reinterpret_cast<const uint4*>(&k);
    uint4* d = reinterpret_cast<uint4*>(row + c);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) d[i] = s[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < C) row[c + i] = from_f<T>(f[i]);
  }
}
__host__ __device__ inline bool rows_aligned(int C, int esize) { return (C * esize) % 16 == 0; }

// ---------------------------------------------------------------- int8
// Nearest integer (ties to even) of |v| < 2^22 in the low byte: adding
// 1.5 * 2^23 leaves the integer in the low mantissa bits, two's complement.
__device__ __forceinline__ uint32_t round_bits(float v) { return __float_as_uint(v + 12582912.0f); }
__device__ __forceinline__ uint2 pack_bytes(const uint32_t (&b)[8]) {
  uint2 r;
  r.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  r.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
  return r;
}
// Four int8 of a word as floats: byte ^ 0x80 = q + 128 becomes the low
// mantissa byte of 2^23, and subtracting 2^23 + 128 is exact.
__device__ __forceinline__ void unpack_bytes(uint32_t w, float* f) {
  const uint32_t u = w ^ 0x80808080u;
  f[0] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7540)) - 8388736.0f;
  f[1] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7541)) - 8388736.0f;
  f[2] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7542)) - 8388736.0f;
  f[3] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7543)) - 8388736.0f;
}
__device__ __forceinline__ void unpack8(uint2 w, float (&f)[8]) {
  unpack_bytes(w.x, f);
  unpack_bytes(w.y, f + 4);
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
  return e == kCkptNaN ? __uint_as_float(0x7fc00000u) : pow2(max(e, -126));
}

// ---------------------------------------------------------------- reductions
// Sum of s and maximum of u over the TPR threads of a row, in a fixed order.
// `red` holds 2 * 2 * (TPR / 32) words per row slot; `slot` alternates.
template <int TPR>
__device__ __forceinline__ void row_reduce(float& s, uint32_t& u, uint32_t* red, int& slot) {
  s = warp_sum(s);
  u = __reduce_max_sync(0xffffffffu, u);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int w = (threadIdx.x & (TPR - 1)) >> 5, rib = threadIdx.x / TPR;
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

// ---------------------------------------------------------------- RMS norm forward
// n = h * rstd * gamma with h = x + r: rstd needs one sum over the row, the
// int8 scale the row's largest |n| = rstd * max|h * gamma|, so both come from
// one reduction, and q = round(h * gamma * 127 / max|h * gamma|) needs no
// rstd at all.
template <typename T, int TPR, int NCH>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) k_rows_fwd(const RowsFwd a) {
  pdl_enter();
  constexpr int TH = TPR < 256 ? 256 : TPR, RPB = TH / TPR;
  __shared__ uint32_t red[RPB * 4 * (TPR / 32)];
  const int sub = threadIdx.x & (TPR - 1), rib = threadIdx.x / TPR;
  const bool vec = rows_aligned(a.C, sizeof(T));
  const float inv_n = 1.f / (float)a.C;
  int slot = 0;
  Chunk<T> g[NCH];
  if (a.norm) {
#pragma unroll
    for (int j = 0; j < NCH; ++j) g[j] = load_chunk(static_cast<const T*>(a.gamma), (sub + j * TPR) * 8, a.C, vec);
  }
  for (long long base = (long long)blockIdx.x * RPB; base < a.R; base += (long long)gridDim.x * RPB) {
    const long long row = base + rib;
    const bool live = row < a.R;
    const T* x = static_cast<const T*>(a.x) + (live ? row : 0) * a.C;
    const T* r = a.r ? static_cast<const T*>(a.r) + (live ? row : 0) * a.C : nullptr;
    float v[NCH][8];
    float ss = 0.f;
    uint32_t am = 0;
    Chunk<T> cx[NCH], cr[NCH];
#pragma unroll
    for (int j = 0; j < NCH; ++j) cx[j] = load_chunk(x, (sub + j * TPR) * 8, live ? a.C : 0, vec);
    if (r) {
#pragma unroll
      for (int j = 0; j < NCH; ++j) cr[j] = load_chunk(r, (sub + j * TPR) * 8, live ? a.C : 0, vec);
    }
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = to_f(cx[j].v[i]);
      if (r) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] += to_f(cr[j].v[i]);
      }
      if (a.h && live) store_chunk(static_cast<T*>(a.h) + row * a.C, (sub + j * TPR) * 8, a.C, vec, v[j]);
      if (a.norm) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(v[j][i], v[j][i], ss);
          v[j][i] *= to_f(g[j].v[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) am = max(am, __float_as_uint(v[j][i]) & kAbs);
    }
    row_reduce<TPR>(ss, am, red, slot);
    if (!live) continue;
    const float rstd = a.norm ? rsqrtf(fmaf(ss, inv_n, a.eps)) : 1.f;
    if (a.rstd && sub == 0) a.rstd[row] = rstd;
    if (a.y) {
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = v[j][i] * rstd;
        store_chunk(static_cast<T*>(a.y) + row * a.C, (sub + j * TPR) * 8, a.C, vec, o);
      }
    }
    if (a.q) {
      // A row that holds an infinity or a NaN has no scale: NaN, and zeros.
      // Tiny rows are lifted by 2^100 so that 127 / max stays finite.
      const bool fine = am < kInfBits;
      const float mx = __uint_as_float(am);
      const float lift = mx < 0x1p-100f ? 0x1p100f : 1.f;
      const float mul = am ? 127.f / (mx * lift) : 0.f;
      if (sub == 0) a.scale[row] = fine ? mx / 127.f * rstd : __uint_as_float(0x7fc00000u);
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const int c = (sub + j * TPR) * 8;
        if (c >= a.P) continue;
        uint32_t b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = round_bits((v[j][i] * lift) * mul);
        const uint2 p = pack_bytes(b);
        *reinterpret_cast<uint2*>(a.q + row * a.P + c) = fine ? p : make_uint2(0, 0);
      }
    }
  }
}

template <typename T>
cudaError_t rows_fwd(const RowsFwd& a, cudaStream_t st) {
  auto go = [&](auto k, int tpr) {
    const int th = tpr < 256 ? 256 : tpr, rpb = th / tpr;
    const long long want = (a.R + rpb - 1) / rpb;
    const long long most = (long long)sm_count() * 16;
    return launch_k(k, dim3((unsigned)(want < most ? want : most)), dim3(th), 0, st, 1, a);
  };
  const int ch = (a.P + 7) / 8;  // the chunks of a padded int8 row
  if (ch <= 64) return go(k_rows_fwd<T, 32, 2>, 32);
  if (ch <= 160) return go(k_rows_fwd<T, 32, 5>, 32);
  if (ch <= 256) return go(k_rows_fwd<T, 128, 2>, 128);
  if (ch <= 512) return go(k_rows_fwd<T, 128, 4>, 128);
  if (ch <= 1024) return go(k_rows_fwd<T, 512, 2>, 512);
  return go(k_rows_fwd<T, 512, 4>, 512);
}

// ---------------------------------------------------------------- element passes
// Flat passes over the 8-column chunks of padded int8 rows.
struct Flat {
  long long R;
  int C, P, cpr;         // chunks per row
  long long total;       // R * cpr
};
__device__ __forceinline__ void flat_at(const Flat& f, long long i, long long& row, int& c) {
  if (f.total < (1ll << 31)) {
    const uint32_t r = (uint32_t)i / (uint32_t)f.cpr;
    row = r;
    c = (int)((uint32_t)i - r * (uint32_t)f.cpr) * 8;
  } else {
    row = i / f.cpr;
    c = (int)(i - row * f.cpr) * 8;
  }
}

// A group of 32 columns is four neighbouring chunks, so four neighbouring
// lanes: its largest magnitude takes two shuffles.
template <typename T>
__global__ void __launch_bounds__(256) k_ckpt_pack(const Flat f, const T* x, int8_t* q, int8_t* e) {
  pdl_enter();
  const bool vec = rows_aligned(f.C, sizeof(T));
  const long long step = (long long)gridDim.x * 256;
  // cpr is a multiple of 4 and so is the total: a group's lanes are live together.
  for (long long i0 = (long long)blockIdx.x * 256; i0 < f.total; i0 += step) {
    const long long i = i0 + threadIdx.x;
    const bool live = i < f.total;
    long long row = 0;
    int c = 0;
    if (live) flat_at(f, i, row, c);
    const Chunk<T> k = load_chunk(x + row * f.C, c, live ? f.C : 0, vec);
    float v[8];
    uint32_t am = 0;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      v[n] = to_f(k.v[n]);
      am = max(am, __float_as_uint(v[n]) & kAbs);
    }
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
    if (!live) continue;
    const int ex = ckpt_exp<T>(am);
    const float inv = pow2(-ex);  // exact, and so is the scaling: the only rounding is to the integer
    uint32_t b[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) b[n] = round_bits(fminf(fmaxf(v[n] * inv, -127.f), 127.f));
    const uint2 p = pack_bytes(b);
    *reinterpret_cast<uint2*>(q + row * f.P + c) = ex == kCkptNaN ? make_uint2(0, 0) : p;
    if ((c & 31) == 0) e[row * (f.P / kQ8Group) + c / kQ8Group] = (int8_t)ex;
  }
}

// MODE 0: checkpoint (one exponent per group), 1: one scale per row.  The
// output rows have `pitch` elements; columns C .. pitch-1 become zeros.
template <typename T, int MODE>
__global__ void __launch_bounds__(256) k_unpack(const Flat f, const int8_t* q, const void* s, T* x, int pitch) {
  pdl_enter();
  const bool vec = rows_aligned(pitch, sizeof(T));
  const long long step = (long long)gridDim.x * 256;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < f.total; i += step) {
    long long row;
    int c;
    flat_at(f, i, row, c);
    if (c >= pitch) continue;
    const float sc = MODE == 0 ? ckpt_step(static_cast<const int8_t*>(s)[row * (f.P / kQ8Group) + c / kQ8Group])
                               : static_cast<const float*>(s)[row];
    float v[8];
    unpack8(*reinterpret_cast<const uint2*>(q + row * f.P + c), v);
#pragma unroll
    for (int n = 0; n < 8; ++n) v[n] = c + n < f.C ? v[n] * sc : 0.f;
    store_chunk(x + row * pitch, c, pitch, vec, v);
  }
}

Flat flat_of(long long R, int C) {
  Flat f;
  f.R = R;
  f.C = C;
  f.P = q8_pitch(C);
  f.cpr = f.P / 8;
  f.total = R * f.cpr;
  return f;
}
unsigned flat_grid(const Flat& f) {
  const long long want = (f.total + 255) / 256, most = (long long)sm_count() * 32;
  return (unsigned)(want < most ? want : most);
}

// ---------------------------------------------------------------- RMS norm backward
// With xh = h * rstd and t = dn * gamma:
//   dx = rstd * (t - xh * mean(t * xh)) (+ dh),  dgamma = sum over rows of dn * xh.
// A thread owns the same columns of every row its block takes, so dgamma's
// partials stay in registers until the block has done its rows; the blocks'
// partial rows are summed in a fixed order afterwards.
template <typename T, int TPR, int NCH, bool CK>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) k_rows_bwd(const RowsBwd a) {
  pdl_enter();
  constexpr int TH = TPR < 256 ? 256 : TPR, RPB = TH / TPR;
  __shared__ uint32_t red[RPB * 4 * (TPR / 32)];
  extern __shared__ float cols[];  // RPB > 1: [C] partials of the block
  const int sub = threadIdx.x & (TPR - 1), rib = threadIdx.x / TPR;
  const bool vec = rows_aligned(a.C, sizeof(T));
  const float inv_n = 1.f / (float)a.C;
  int slot = 0;
  Chunk<T> g[NCH];
  float acc[NCH][8];
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    g[j] = load_chunk(static_cast<const T*>(a.gamma), (sub + j * TPR) * 8, a.C, vec);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[j][i] = 0.f;
  }
  for (long long base = (long long)blockIdx.x * RPB; base < a.R; base += (long long)gridDim.x * RPB) {
    const long long row = base + rib;
    const bool live = row < a.R;
    const long long rr = live ? row : 0;
    const int Cl = live ? a.C : 0;
    Chunk<T> dn[NCH], hs[CK ? 1 : NCH], dh[NCH];
    uint2 hq[CK ? NCH : 1];
    float hstep[CK ? NCH : 1];
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int c = (sub + j * TPR) * 8;
      dn[j] = load_chunk(static_cast<const T*>(a.dn) + rr * a.C, c, Cl, vec);
      if constexpr (CK) {
        const bool in = live && c < a.P;
        hq[j] = in ? *reinterpret_cast<const uint2*>(a.q + rr * a.P + c) : make_uint2(0, 0);
        hstep[j] = in ? ckpt_step(a.e[rr * (a.P / kQ8Group) + c / kQ8Group]) : 0.f;
      } else {
        hs[j] = load_chunk(static_cast<const T*>(a.h) + rr * a.C, c, Cl, vec);
      }
    }
    if (a.dh) {
#pragma unroll
      for (int j = 0; j < NCH; ++j) dh[j] = load_chunk(static_cast<const T*>(a.dh) + rr * a.C, (sub + j * TPR) * 8, Cl, vec);
    }
    const float rstd = live ? a.rstd[row] : 0.f;
    auto xhat = [&](int j, float (&xh)[8]) {
      if constexpr (CK) {
        unpack8(hq[j], xh);
        const float s = hstep[j] * rstd;
#pragma unroll
        for (int i = 0; i < 8; ++i) xh[i] *= s;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) xh[i] = to_f(hs[j].v[i]) * rstd;
      }
    };
    float dot = 0.f;
    uint32_t unused = 0;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float xh[8];
      xhat(j, xh);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = to_f(dn[j].v[i]) * xh[i];
        if (live) acc[j][i] += p;
        dot = fmaf(p, to_f(g[j].v[i]), dot);
      }
    }
    row_reduce<TPR>(dot, unused, red, slot);
    if (!live) continue;
    const float m = dot * inv_n;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float xh[8], o[8];
      xhat(j, xh);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = rstd * (to_f(dn[j].v[i]) * to_f(g[j].v[i]) - xh[i] * m);
      if (a.dh) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += to_f(dh[j].v[i]);
      }
      store_chunk(static_cast<T*>(a.dx) + row * a.C, (sub + j * TPR) * 8, a.C, vec, o);
    }
  }
  float* pg = a.pg + (size_t)blockIdx.x * a.C;
  if constexpr (RPB == 1) {
#pragma unroll
    for (int j = 0; j < NCH; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = (sub + j * TPR) * 8 + i;
        if (c < a.C) pg[c] = acc[j][i];
      }
  } else {
    for (int w = 0; w < RPB; ++w) {
      if (rib == w) {
#pragma unroll
        for (int j = 0; j < NCH; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int c = (sub + j * TPR) * 8 + i;
            if (c < a.C) cols[c] = w ? cols[c] + acc[j][i] : acc[j][i];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.C; c += TH) pg[c] = cols[c];
  }
}

int rows_bwd_tpr(int C) {
  const int ch = (q8_pitch(C) + 7) / 8;
  return ch <= 160 ? 32 : ch <= 512 ? 128 : 512;
}

template <typename T, bool CK>
cudaError_t rows_bwd(const RowsBwd& a, cudaStream_t st) {
  auto go = [&](auto k, int tpr) {
    const int th = tpr < 256 ? 256 : tpr;
    const size_t smem = tpr < 256 ? (size_t)a.C * sizeof(float) : 0;
    return launch_k(k, dim3((unsigned)rows_bwd_blocks(a.R, a.C)), dim3(th), smem, st, 1, a);
  };
  const int ch = (a.P + 7) / 8;
  if (ch <= 64) return go(k_rows_bwd<T, 32, 2, CK>, 32);
  if (ch <= 160) return go(k_rows_bwd<T, 32, 5, CK>, 32);
  if (ch <= 256) return go(k_rows_bwd<T, 128, 2, CK>, 128);
  if (ch <= 512) return go(k_rows_bwd<T, 128, 4, CK>, 128);
  if (ch <= 1024) return go(k_rows_bwd<T, 512, 2, CK>, 512);
  return go(k_rows_bwd<T, 512, 4, CK>, 512);
}

// ---------------------------------------------------------------- column partials
// One thread per column pair position: block (x, y) sums rows of slice y for
// 256 consecutive columns, rows in order.
template <typename T>
__global__ void __launch_bounds__(256) k_colpart(long long R, long long J, int slices, const T* x, float* part) {
  pdl_enter();
  const long long j = (long long)blockIdx.x * 256 + threadIdx.x;
  if (j >= J) return;
  const long long r0 = R * blockIdx.y / slices, r1 = R * (blockIdx.y + 1) / slices;
  float s = 0.f;
#pragma unroll 8
  for (long long r = r0; r < r1; ++r) s += to_f(x[r * J + j]);
  part[blockIdx.y * J + j] = s;
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
    for (int k = ty; k < K; k += 8) am = max(am, __float_as_uint(to_f(wg[(size_t)k * N + n0 + tx])) & kAbs);
  mx[ty][tx] = am;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) am = max(am, mx[i][tx]);
  if (ty == 0 && n0 + tx < N)
    scale[(size_t)g * N + n0 + tx] = am < kInfBits ? __uint_as_float(am) / 127.f : __uint_as_float(0x7fc00000u);
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
      uint32_t b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = i < 4 ? round_bits(tile[kk + i][n]) : 0u;
      *reinterpret_cast<uint32_t*>(q + ((size_t)g * N + n0 + n) * P + k0 + kk) = pack_bytes(b).x;
    }
  }
}

}  // namespace

#define RMX_BY_DTYPE(dt, ...)            \
  switch (dt) {                          \
    case 0: { using T = float; __VA_ARGS__; }\
    case 1: { using T = bf16; __VA_ARGS__; }\
    case 2: { using T = f16; __VA_ARGS__; }\
    default: return cudaErrorInvalidValue; \
  }

cudaError_t launch_rows_fwd(const RowsFwd& a, cudaStream_t st) { RMX_BY_DTYPE(a.dtype, return rows_fwd<T>(a, st)) }

cudaError_t launch_dequant_rows(long long R, int C, int dtype, const int8_t* q, const float* scale, void* x,
                                cudaStream_t st) {
  const Flat f = flat_of(R, C);
  RMX_BY_DTYPE(dtype, return launch_k(k_unpack<T, 1>, dim3(flat_grid(f)), dim3(256), 0, st, 1, f, q,
                                      static_cast<const void*>(scale), static_cast<T*>(x), C))
}

cudaError_t launch_ckpt_pack(long long R, int C, int dtype, const void* x, int8_t* q, int8_t* e, cudaStream_t st) {
  const Flat f = flat_of(R, C);
  RMX_BY_DTYPE(dtype, return launch_k(k_ckpt_pack<T>, dim3(flat_grid(f)), dim3(256), 0, st, 1, f,
                                      static_cast<const T*>(x), q, e))
}

cudaError_t launch_ckpt_unpack(long long R, int C, int dtype, const int8_t* q, const int8_t* e, void* x, int pitch,
                               cudaStream_t st) {
  const Flat f = flat_of(R, C);
  RMX_BY_DTYPE(dtype, return launch_k(k_unpack<T, 0>, dim3(flat_grid(f)), dim3(256), 0, st, 1, f, q,
                                      static_cast<const void*>(e), static_cast<T*>(x), pitch))
}

int rows_bwd_blocks(long long R, int C) {
  const int tpr = rows_bwd_tpr(C), rpb = tpr < 256 ? 256 / tpr : 1;
  const long long want = (R + rpb - 1) / rpb;
  long long most = (long long)sm_count() * 2;
  if (most > kRowsBwdMaxBlocks) most = kRowsBwdMaxBlocks;
  return (int)(want < most ? want : most);
}
cudaError_t launch_rows_bwd(const RowsBwd& a, cudaStream_t st) {
  RMX_BY_DTYPE(a.dtype, return a.h ? rows_bwd<T, false>(a, st) : rows_bwd<T, true>(a, st))
}

int colpart_slices(long long R) { return (int)(R < 64 ? (R < 1 ? 1 : R) : 64); }
cudaError_t launch_colpart(long long R, long long J, int dtype, const void* x, float* part, cudaStream_t st) {
  const int s = colpart_slices(R);
  const dim3 grid((unsigned)((J + 255) / 256), s);
  RMX_BY_DTYPE(dtype, return launch_k(k_colpart<T>, grid, dim3(256), 0, st, 1, R, J, s, static_cast<const T*>(x), part))
}

cudaError_t launch_weight_q8(int G, int K, int N, int dtype, const void* w, int8_t* q, float* scale,
                             cudaStream_t st) {
  const dim3 grid((N + 31) / 32, G);
  RMX_BY_DTYPE(dtype, return launch_k(k_weight_q8<T>, grid, dim3(256), 0, st, 1, K, N, q8_pitch(K),
                                      static_cast<const T*>(w), q, scale))
}

}  // namespace rmx
