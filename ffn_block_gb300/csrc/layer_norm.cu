// Layer norm with dropout and the residual before it, its backward, and dropout
// by itself.
//
//   h = drop(x) + r;  y = (h - mean) * rstd * gamma + beta
//   dr = rstd * (t - mean(t) - xh * mean(t * xh)) + dh,  t = dy * gamma, xh = (h - mean) * rstd
//
// Bound by HBM: one pass over the data each, the row in registers between its
// moments and its output.  The moments are taken in two steps (mean, then the
// squared deviations), so a row far from zero loses nothing.

#include "common.cuh"
#include "dropout.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "q8_rows.cuh"
#include "sparse.h"

namespace rmx {
namespace {

// Sums of N values over the L lanes and W warps of a row, in a fixed order.
// `red` holds two slots of N floats a warp, used in turn; the row's warps meet
// at a barrier of their own.
template <int L, int N>
__device__ __forceinline__ void row_sums(float (&s)[N], float* red, int slot, int w, int W, int barrier) {
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = lanes_sum<L>(s[i]);
  if (L < 32 || W == 1) return;
  float* r = red + slot * N * W;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[N * w + i] = s[i];
  }
  asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(32 * W) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = 0.f;
  for (int j = 0; j < W; ++j) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += r[N * j + i];
  }
}

// Zeroes the elements past the row's end.
template <int L, bool VEC> __device__ __forceinline__ void mask_end(float2 (&v)[4], int c0, int C) {
  if (col<L, VEC>(c0, 7) < C) return;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (col<L, VEC>(c0, i) >= C) (i & 1 ? v[i / 2].y : v[i / 2].x) = 0.f;
}

// ---------------------------------------------------------------- dropout
// A unit is a block of 8 * L columns of a row, a lane takes eight of them;
// kUnits units at a time, so that their loads are in flight together.
constexpr int kUnits = 4;
template <typename T, int L, bool VEC>
__global__ void __launch_bounds__(256) k_dropout(long long row0, uint32_t units, int bpr, int C, const Drop d,
                                                 const T* x, const T* r, T* out) {
  pdl_enter();
  const int lane = threadIdx.x & (L - 1);
  const DropBits bits = drop_bits(d);
  constexpr int PER = 256 / L;
  const uint32_t u0 = blockIdx.x * (PER * kUnits) + threadIdx.x / L;
  Chunk<T> cx[kUnits], cr[kUnits];
  long long row[kUnits];
  int c0[kUnits];
  bool live[kUnits];
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const uint32_t u = u0 + (uint32_t)(j * PER);
    live[j] = u < units;
    const uint32_t ur = live[j] ? u / (uint32_t)bpr : 0u;
    row[j] = row0 + ur;
    c0[j] = col0<L, VEC>(live[j] ? (int)(u - ur * (uint32_t)bpr) : 0, lane);
    const int end = live[j] ? C : 0;
    cx[j] = load_chunk<T, L, VEC>(x + (size_t)row[j] * C, c0[j], end);
    if (r) cr[j] = load_chunk<T, L, VEC>(r + (size_t)row[j] * C, c0[j], end);
  }
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    float2 v[4];
    to_pairs(cx[j], v);
    if (bits.mode == DROP_BITS) drop_pairs(keep_of<L, VEC>(bits, row[j], c0[j]), d.scale, v);
    else if (bits.mode == DROP_ALL) drop_pairs(0, 0.f, v);
    if (r) {
      float2 w[4];
      to_pairs(cr[j], w);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = add2(v[i], w[i]);
    }
    if (live[j]) store_chunk<T, L, VEC>(out + (size_t)row[j] * C, c0[j], C, v);
  }
}

template <typename T, int L, bool VEC>
cudaError_t dropout(long long R, int C, const Drop& d, const void* x, const void* r, void* out, cudaStream_t st) {
  const int bpr = (C + 8 * L - 1) / (8 * L);
  // 32-bit unit numbers: the largest tensors go in ranges of rows.
  const long long most = (1ll << 30) / bpr;
  for (long long row0 = 0; row0 < R; row0 += most) {
    const long long rows = R - row0 < most ? R - row0 : most;
    const uint32_t units = (uint32_t)(rows * bpr);
    const uint32_t per = 256 / L * kUnits;
    cudaError_t e = launch_k(k_dropout<T, L, VEC>, dim3((units + per - 1) / per), dim3(256), 0, st, 1, row0, units, bpr,
                             C, d, (const T*)x, (const T*)r, (T*)out);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}
template <typename T>
cudaError_t dropout_t(long long R, int C, const Drop& d, const void* x, const void* r, void* out, cudaStream_t st) {
  const bool vec = rows_aligned(C, sizeof(T));
  if (C <= 64) return vec ? dropout<T, 8, true>(R, C, d, x, r, out, st) : dropout<T, 8, false>(R, C, d, x, r, out, st);
  return vec ? dropout<T, 32, true>(R, C, d, x, r, out, st) : dropout<T, 32, false>(R, C, d, x, r, out, st);
}

// ---------------------------------------------------------------- forward
// A row belongs to L lanes of W warps (W > 1 only with L = 32), with NCH blocks
// of 8 * L columns each; rpb rows at a time to a thread block.
template <typename T, int L, int NCH, bool VEC>
__global__ void __launch_bounds__(512) k_layer_norm(const LnFwd a, const int W, const int rpb) {
  pdl_enter();
  __shared__ float red[64];
  const int lane = threadIdx.x & (L - 1), part = threadIdx.x / L, rib = part / W, w = part - rib * W;
  const DropBits bits = drop_bits(a.drop);
  const float inv_n = 1.f / (float)a.C;
  float* my_red = red + rib * 2 * W;
  const long long step = (long long)gridDim.x * rpb;
  const int first_of_warp = L == 32 ? rib : (threadIdx.x >> 5) * (32 / L);
  auto c_of = [&](int j) { return col0<L, VEC>(w + j * W, lane); };
  for (long long row = (long long)blockIdx.x * rpb + rib; row - rib + first_of_warp < a.R; row += step) {
    const bool live = L == 32 || row < a.R;
    const size_t at = (size_t)(live ? row : 0) * a.C;
    const int C = live ? a.C : 0;
    Chunk<T> cx[NCH], cr[NCH];
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      cx[j] = load_chunk<T, L, VEC>(static_cast<const T*>(a.x) + at, c_of(j), C);
      if (a.r) cr[j] = load_chunk<T, L, VEC>(static_cast<const T*>(a.r) + at, c_of(j), C);
    }
    float2 v[NCH][4], s2 = f2(0.f);
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      to_pairs(cx[j], v[j]);
      if (bits.mode == DROP_BITS) drop_pairs(keep_of<L, VEC>(bits, row, c_of(j)), a.drop.scale, v[j]);
      else if (bits.mode == DROP_ALL) drop_pairs(0, 0.f, v[j]);
      if (a.r) {
        float2 r[4];
        to_pairs(cr[j], r);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = add2(v[j][i], r[i]);
      }
      if (a.h && live) store_chunk<T, L, VEC>(static_cast<T*>(a.h) + at, c_of(j), a.C, v[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) s2 = add2(s2, v[j][i]);
    }
    float s[1] = {s2.x + s2.y};
    row_sums<L, 1>(s, my_red, 0, w, W, 1 + rib);
    const float mean = s[0] * inv_n;
    s2 = f2(0.f);
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = add2(v[j][i], f2(-mean));
      mask_end<L, VEC>(v[j], c_of(j), a.C);
#pragma unroll
      for (int i = 0; i < 4; ++i) s2 = fma2(v[j][i], v[j][i], s2);
    }
    s[0] = s2.x + s2.y;
    row_sums<L, 1>(s, my_red, 1, w, W, 1 + rib);
    const float rstd = 1.f / sqrtf(s[0] * inv_n + a.eps);
    if (live && w == 0 && lane == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = mul2(v[j][i], f2(rstd));
      float2 g[4];
      if (a.gamma) {
        to_pairs(load_chunk<T, L, VEC>(static_cast<const T*>(a.gamma), c_of(j), a.C), g);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = mul2(v[j][i], g[i]);
      }
      if (a.beta) {
        to_pairs(load_chunk<T, L, VEC>(static_cast<const T*>(a.beta), c_of(j), a.C), g);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = add2(v[j][i], g[i]);
      }
      if (live) store_chunk<T, L, VEC>(static_cast<T*>(a.y) + at, c_of(j), a.C, v[j]);
    }
  }
}

struct Spread {
  int L, W, nch, rpb, threads;
};
// Up to 1280 columns a warp (or a part of it) has the row to itself, without a
// barrier; above, as few warps as hold it with four blocks each.
Spread fwd_spread(int C) {
  Spread s;
  const int blocks = (C + 255) / 256;
  s.L = C <= 64 ? 8 : C <= 128 ? 16 : 32;
  s.nch = blocks <= 1 ? 1 : blocks == 2 ? 2 : blocks == 5 ? 5 : 4;
  s.W = (blocks + s.nch - 1) / s.nch;
  s.rpb = s.W == 1 ? 256 / s.L : s.W < 8 ? 8 / s.W : 1;
  s.threads = s.L * s.W * s.rpb;
  return s;
}
template <typename T, bool VEC> cudaError_t layer_norm(const LnFwd& a, cudaStream_t st) {
  const Spread s = fwd_spread(a.C);
  auto k = s.L == 8     ? k_layer_norm<T, 8, 1, VEC>
           : s.L == 16  ? k_layer_norm<T, 16, 1, VEC>
           : s.nch == 1 ? k_layer_norm<T, 32, 1, VEC>
           : s.nch == 2 ? k_layer_norm<T, 32, 2, VEC>
           : s.nch == 4 ? k_layer_norm<T, 32, 4, VEC>
                        : k_layer_norm<T, 32, 5, VEC>;
  const long long want = (a.R + s.rpb - 1) / s.rpb, most = (long long)sm_count() * 16;
  return launch_k(k, dim3((unsigned)(want < most ? want : most)), dim3(s.threads), 0, st, 1, a, s.W, s.rpb);
}

// ---------------------------------------------------------------- backward
template <typename T, int L, int NCH, bool VEC>
__global__ void __launch_bounds__(512) k_layer_norm_bwd(const LnBwd a, const int W, const int rpb) {
  pdl_enter();
  __shared__ float red[128];
  extern __shared__ float cols[];  // partials of the block's sets of warps, [sets - 1][2][C]
  const int lane = threadIdx.x & (L - 1), part = threadIdx.x / L, rib = part / W, w = part - rib * W;
  const DropBits bits = drop_bits(a.drop);
  const float inv_n = 1.f / (float)a.C;
  float* my_red = red + rib * 4 * W;
  auto c_of = [&](int j) { return col0<L, VEC>(w + j * W, lane); };
  float2 ag[NCH][4], ab[NCH][4];
#pragma unroll
  for (int j = 0; j < NCH; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) ag[j][i] = ab[j][i] = f2(0.f);
  const long long step = (long long)gridDim.x * rpb;
  int slot = 0;
  const int first_of_warp = L == 32 ? rib : (threadIdx.x >> 5) * (32 / L);
  for (long long row = (long long)blockIdx.x * rpb + rib; row - rib + first_of_warp < a.R; row += step, slot ^= 1) {
    const bool live = L == 32 || row < a.R;
    const size_t at = (size_t)(live ? row : 0) * a.C;
    const int C = live ? a.C : 0;
    Chunk<T> cy[NCH], ch[NCH], cd[NCH];
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      cy[j] = load_chunk<T, L, VEC>(static_cast<const T*>(a.dy) + at, c_of(j), C);
      ch[j] = load_chunk<T, L, VEC>(static_cast<const T*>(a.h) + at, c_of(j), C);
      if (a.dh) cd[j] = load_chunk<T, L, VEC>(static_cast<const T*>(a.dh) + at, c_of(j), C);
    }
    const float rstd = live ? a.rstd[row] : 0.f, shift = live ? -a.mean[row] * rstd : 0.f;
    auto both = [&](int j, float2 (&xh)[4], float2 (&t)[4]) {
      to_pairs(ch[j], xh);
      to_pairs(cy[j], t);
#pragma unroll
      for (int i = 0; i < 4; ++i) xh[i] = fma2(xh[i], f2(rstd), f2(shift));
    };
    auto weigh = [&](int j, float2 (&t)[4]) {
      if (!a.gamma) return;
      float2 g[4];
      to_pairs(load_chunk<T, L, VEC>(static_cast<const T*>(a.gamma), c_of(j), a.C), g);
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = mul2(t[i], g[i]);
    };
    float2 m1 = f2(0.f), m2 = f2(0.f);
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float2 xh[4], t[4];
      both(j, xh, t);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ag[j][i] = fma2(t[i], xh[i], ag[j][i]);
        ab[j][i] = add2(t[i], ab[j][i]);
      }
      weigh(j, t);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m1 = add2(m1, t[i]);
        m2 = fma2(t[i], xh[i], m2);
      }
    }
    float m[2] = {m1.x + m1.y, m2.x + m2.y};
    row_sums<L, 2>(m, my_red, slot, w, W, 1 + rib);
    const float2 c1 = f2(-m[0] * inv_n), c2 = f2(-m[1] * inv_n), rs = f2(rstd);
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float2 xh[4], t[4];
      both(j, xh, t);
      weigh(j, t);
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = mul2(fma2(xh[i], c2, add2(t[i], c1)), rs);
      if (a.dh) {
        float2 d[4];
        to_pairs(cd[j], d);
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = add2(t[i], d[i]);
      }
      if (live) store_chunk<T, L, VEC>(static_cast<T*>(a.dr) + at, c_of(j), a.C, t);
      if (a.dx) {
        if (bits.mode == DROP_BITS) drop_pairs(keep_of<L, VEC>(bits, row, c_of(j)), a.drop.scale, t);
        else if (bits.mode == DROP_ALL) drop_pairs(0, 0.f, t);
        if (live) store_chunk<T, L, VEC>(static_cast<T*>(a.dx) + at, c_of(j), a.C, t);
      }
    }
  }
  // The block's partials: parts of a warp in a tree of shuffles, then the sets
  // of warps in order, the first adding the others' to its own.
  const int sets = L == 32 ? rpb : blockDim.x / 32, set = L == 32 ? rib : threadIdx.x >> 5;
  auto each = [&](auto f) {
#pragma unroll
    for (int j = 0; j < NCH; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = col<L, VEC>(c_of(j), i);
        f(i & 1 ? ag[j][i / 2].y : ag[j][i / 2].x, i & 1 ? ab[j][i / 2].y : ab[j][i / 2].x, c);
      }
  };
  each([&](float& g, float& b, int c) {
#pragma unroll
    for (int o = L; o < 32; o <<= 1) {
      g += __shfl_xor_sync(0xffffffffu, g, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (set > 0 && c < a.C) {
      cols[(2 * (set - 1)) * a.C + c] = g;
      cols[(2 * (set - 1) + 1) * a.C + c] = b;
    }
  });
  if (sets > 1) __syncthreads();
  if (set > 0) return;
#pragma unroll 1
  for (int r = 1; r < sets; ++r)
    each([&](float& g, float& b, int c) {
      if (c < a.C) {
        g += cols[(2 * (r - 1)) * a.C + c];
        b += cols[(2 * (r - 1) + 1) * a.C + c];
      }
    });
  float* pg = a.pg + (size_t)blockIdx.x * a.C;
  float* pb = a.pb + (size_t)blockIdx.x * a.C;
  each([&](float& g, float& b, int c) {
    if (c < a.C) {
      pg[c] = g;
      pb[c] = b;
    }
  });
}

Spread bwd_spread(int C) {
  Spread s;
  const int blocks = (C + 255) / 256;
  s.L = C <= 64 ? 8 : C <= 128 ? 16 : 32;
  s.nch = blocks <= 16 ? 1 : blocks <= 32 ? 2 : 4;
  s.W = (blocks + s.nch - 1) / s.nch;
  s.rpb = s.W == 1 ? 256 / s.L : s.W < 10 ? 10 / s.W : 1;
  s.threads = s.L * s.W * s.rpb;
  return s;
}
template <typename T, bool VEC> cudaError_t layer_norm_bwd(const LnBwd& a, cudaStream_t st) {
  const Spread s = bwd_spread(a.C);
  const int sets = s.L == 32 ? s.rpb : s.threads / 32;
  const size_t smem = (size_t)(sets - 1) * 2 * a.C * sizeof(float);  // 18 KB at most
  auto k = s.L == 8     ? k_layer_norm_bwd<T, 8, 1, VEC>
           : s.L == 16  ? k_layer_norm_bwd<T, 16, 1, VEC>
           : s.nch == 1 ? k_layer_norm_bwd<T, 32, 1, VEC>
           : s.nch == 2 ? k_layer_norm_bwd<T, 32, 2, VEC>
                        : k_layer_norm_bwd<T, 32, 4, VEC>;
  return launch_k(k, dim3((unsigned)ln_bwd_rows_blocks(a)), dim3(s.threads), smem, st, 1, a, s.W, s.rpb);
}

}  // namespace

cudaError_t launch_dropout(long long R, int C, int dtype, const Drop& d, const void* x, const void* r, void* out,
                           cudaStream_t st) {
  RMX_BY_DTYPE(dtype, return dropout_t<T>(R, C, d, x, r, out, st))
}
cudaError_t launch_layer_norm(const LnFwd& a, cudaStream_t st) {
  RMX_BY_DTYPE(a.dtype, return rows_aligned(a.C, sizeof(T)) ? layer_norm<T, true>(a, st) : layer_norm<T, false>(a, st))
}
int ln_bwd_rows_blocks(const LnBwd& a) {
  const Spread s = bwd_spread(a.C);
  const long long want = (a.R + s.rpb - 1) / s.rpb;
  long long most = (long long)sm_count() * 3;
  if (most > kLnBwdMaxBlocks) most = kLnBwdMaxBlocks;
  return (int)(want < most ? want : most);
}
cudaError_t launch_layer_norm_bwd(const LnBwd& a, cudaStream_t st) {
  RMX_BY_DTYPE(a.dtype,
               return rows_aligned(a.C, sizeof(T)) ? layer_norm_bwd<T, true>(a, st) : layer_norm_bwd<T, false>(a, st))
}

}  // namespace rmx
