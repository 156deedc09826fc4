// RMS norm backward of the 8-bit operators.
//
// With xh = h * rstd and t = dn * gamma:
//   dx = rstd * (t - xh * mean(t * xh)) (+ dh),  dgamma = sum over rows of dn * xh.
// Bound by HBM traffic: dn, dh and h (or its 8-bit checkpoint) in, dx out, a
// row held in registers, packed as loaded, between its reduction and its
// output.  A thread owns the same columns of every row its block takes, so
// dgamma's partials stay in registers until the block has done its rows; the
// blocks' partial rows are summed in a fixed order afterwards.

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "q8.h"
#include "q8_rows.cuh"

namespace rmx {
namespace {

template <typename T, int TPR, int NCH, bool CK, bool VEC>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, TPR < 256 ? 2 : 1) k_rows_bwd(const RowsBwd a) {
  pdl_enter();
  constexpr int TH = TPR < 256 ? 256 : TPR, RPB = TH / TPR, W = TPR / 32;
  __shared__ uint32_t red[RPB * 4 * W];
  extern __shared__ float cols[];  // RPB > 1: [C] partials of the block
  const int lane = threadIdx.x & 31, w = (threadIdx.x & (TPR - 1)) >> 5, rib = threadIdx.x / TPR;
  const float inv_n = 1.f / (float)a.C;
  const int groups = a.P / kQ8Group;
  int slot = 0;
  Chunk<T> g[NCH];
  float2 acc[NCH][4];
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    g[j] = load_chunk<T, VEC>(static_cast<const T*>(a.gamma), col0<VEC>(w + j * W, lane), a.C);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = f2(0.f);
  }
  for (long long base = (long long)blockIdx.x * RPB; base < a.R; base += (long long)gridDim.x * RPB) {
    const long long row = base + rib;
    const bool live = row < a.R;
    const size_t rr = live ? row : 0, at = rr * a.C;
    const int C = live ? a.C : 0, P = live ? a.P : 0;
    Chunk<T> dn[NCH], hs[CK ? 1 : NCH], dh[NCH];
    uint2 hq[CK ? NCH : 1];
    uint32_t he[CK ? NCH : 1][VEC ? 1 : 2];
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int c0 = col0<VEC>(w + j * W, lane);
      dn[j] = load_chunk<T, VEC>(static_cast<const T*>(a.dn) + at, c0, C);
      if constexpr (CK) {
        hq[j] = load_bytes<VEC>(a.q + rr * a.P, c0, P);
        const int8_t* e = a.e + rr * groups;
        if constexpr (VEC) {
          he[j][0] = c0 < P ? (uint32_t)(int)e[c0 / kQ8Group] : 0u;
        } else {
          const int g0 = (w + j * W) * 8;
          he[j][0] = he[j][1] = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if ((g0 + i) * kQ8Group < P) he[j][i / 4] |= (uint32_t)(uint8_t)e[g0 + i] << (8 * (i & 3));
        }
      } else {
        hs[j] = load_chunk<T, VEC>(static_cast<const T*>(a.h) + at, c0, C);
      }
    }
    if (a.dh) {
#pragma unroll
      for (int j = 0; j < NCH; ++j)
        dh[j] = load_chunk<T, VEC>(static_cast<const T*>(a.dh) + at, col0<VEC>(w + j * W, lane), C);
    }
    const float rstd = live ? a.rstd[row] : 0.f;
    auto xhat = [&](int j, float2 (&xh)[4]) {
      if constexpr (CK) {
        biased(hq[j], xh);
        if constexpr (VEC) {
          const float s = ckpt_step((int)he[j][0]) * rstd;
#pragma unroll
          for (int i = 0; i < 4; ++i) xh[i] = mul2(add2(xh[i], f2(-kBias)), f2(s));
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float& t = i & 1 ? xh[i / 2].y : xh[i / 2].x;
            t = (t - kBias) * (ckpt_step((int8_t)(he[j][i / 4] >> (8 * (i & 3)))) * rstd);
          }
        }
      } else {
        to_pairs(hs[j], xh);
#pragma unroll
        for (int i = 0; i < 4; ++i) xh[i] = mul2(xh[i], f2(rstd));
      }
    };
    float2 dot2 = f2(0.f);
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float2 xh[4], d[4], gm[4];
      xhat(j, xh);
      to_pairs(dn[j], d);
      to_pairs(g[j], gm);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 p = mul2(d[i], xh[i]);
        if (live) acc[j][i] = add2(acc[j][i], p);
        dot2 = fma2(p, gm[i], dot2);
      }
    }
    float dot = dot2.x + dot2.y;
    uint32_t unused = 0;
    row_reduce<TPR>(dot, unused, red, slot);
    if (!live) continue;
    const float m = -dot * inv_n;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float2 xh[4], d[4], gm[4];
      xhat(j, xh);
      to_pairs(dn[j], d);
      to_pairs(g[j], gm);
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = mul2(fma2(xh[i], f2(m), mul2(d[i], gm[i])), f2(rstd));
      if (a.dh) {
        float2 r[4];
        to_pairs(dh[j], r);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = add2(d[i], r[i]);
      }
      store_chunk<T, VEC>(static_cast<T*>(a.dx) + at, col0<VEC>(w + j * W, lane), a.C, d);
    }
  }
  float* pg = a.pg + (size_t)blockIdx.x * a.C;
#pragma unroll 1
  for (int r = 0; r < RPB; ++r) {
    if (rib == r) {
#pragma unroll
      for (int j = 0; j < NCH; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = col<VEC>(col0<VEC>(w + j * W, lane), i);
          const float v = i & 1 ? acc[j][i / 2].y : acc[j][i / 2].x;
          if (c < a.C) {
            if (RPB == 1) pg[c] = v;
            else cols[c] = r ? cols[c] + v : v;
          }
        }
    }
    if (RPB > 1) __syncthreads();
  }
  if (RPB > 1)
    for (int c = threadIdx.x; c < a.C; c += TH) pg[c] = cols[c];
}

// Threads of a row, by its 256-column blocks: a warp holds two.
int rows_bwd_tpr(int C) {
  const int blocks = (q8_pitch(C) + 255) / 256;
  return blocks <= 2 ? 32 : blocks <= 8 ? 128 : 512;
}

template <typename T, bool CK, bool VEC>
cudaError_t rows_bwd(const RowsBwd& a, cudaStream_t st) {
  auto go = [&](auto k, int tpr) {
    const int th = tpr < 256 ? 256 : tpr;
    const size_t smem = tpr < 256 ? (size_t)a.C * sizeof(float) : 0;
    return launch_k(k, dim3((unsigned)rows_bwd_blocks(a.R, a.C)), dim3(th), smem, st, 1, a);
  };
  const int tpr = rows_bwd_tpr(a.C);
  if (tpr == 32) return go(k_rows_bwd<T, 32, 2, CK, VEC>, 32);
  if (tpr == 128) return go(k_rows_bwd<T, 128, 2, CK, VEC>, 128);
  if (a.P <= 8192) return go(k_rows_bwd<T, 512, 2, CK, VEC>, 512);
  return go(k_rows_bwd<T, 512, 4, CK, VEC>, 512);
}

template <typename T>
cudaError_t rows_bwd_t(const RowsBwd& a, cudaStream_t st) {
  if (rows_aligned(a.C, sizeof(T))) return a.h ? rows_bwd<T, false, true>(a, st) : rows_bwd<T, true, true>(a, st);
  return a.h ? rows_bwd<T, false, false>(a, st) : rows_bwd<T, true, false>(a, st);
}

}  // namespace

int rows_bwd_blocks(long long R, int C) {
  const int tpr = rows_bwd_tpr(C), rpb = tpr < 256 ? 256 / tpr : 1;
  const long long want = (R + rpb - 1) / rpb;
  long long most = (long long)sm_count() * (tpr < 256 ? 2 : 1);  // what is resident at once
  if (most > kRowsBwdMaxBlocks) most = kRowsBwdMaxBlocks;
  return (int)(want < most ? want : most);
}
cudaError_t launch_rows_bwd(const RowsBwd& a, cudaStream_t st) { RMX_BY_DTYPE(a.dtype, return rows_bwd_t<T>(a, st)) }

}  // namespace rmx
