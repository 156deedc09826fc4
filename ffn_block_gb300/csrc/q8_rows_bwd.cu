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

// Sum over the L lanes and W warps of a row, in a fixed order.  `red` holds two slots of a
// float per warp of the row, used in turn; the row's warps meet at a barrier of
// their own (rows of a block do not wait for one another).
template <int L>
__device__ __forceinline__ float row_sum(float s, float* red, int slot, int w, int W, int barrier) {
  s = lanes_sum<L>(s);
  if (L < 32 || W == 1) return s;
  float* r = red + slot * W;
  if ((threadIdx.x & 31) == 0) r[w] = s;
  asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(32 * W) : "memory");
  s = 0.f;
  for (int i = 0; i < W; ++i) s += r[i];
  return s;
}

// Registers of a thread with one block of a row.  Many warps with one row each
// hide the loads better than few with rows loaded ahead: 65536 rows of 1280
// 16-bit columns from a checkpoint take 120 us at 64 registers (30 warps a SM;
// 4.9 TB/s, 74% of the measured copy rate), 198 us with two rows ahead at 96 (20
// warps); at 48, 56 or 72 registers they are slower too.  What is left is latency:
// a warp issues about 217 instructions for a block of 256 columns and waits for
// its loads and the row's barrier in turn, at half of the issue rate.
constexpr int kRegs = 64;

// What a row brings, as loaded.
template <typename T, bool CK, bool VEC> struct RowIn {
  Chunk<T> dn, dh;
  Chunk<T> h;          // the stored sum
  uint2 q;             // or its checkpoint: eight int8 and their exponents
  uint2 e;             // (VEC: the lane's own in x)
};

// A row belongs to W warps (W = blocks of 256 columns, up to 16), each with
// NCH blocks of it; `rpb` rows at a time to a thread block.
template <typename T, int L, int NCH, bool CK, bool VEC>
__global__ void __maxnreg__(NCH == 1 ? kRegs : 128) k_rows_bwd(const RowsBwd a, const int W, const int rpb) {
  pdl_enter();
  __shared__ float red[64];
  extern __shared__ float cols[];  // partials of the block's sets of warps, [sets - 1][C]
  const int lane = threadIdx.x & (L - 1), part = threadIdx.x / L, rib = part / W, w = part - rib * W;
  const float inv_n = 1.f / (float)a.C;
  const int groups = a.P / kQ8Group;
  float* my_red = red + rib * 2 * W;
  auto c_of = [&](int j) { return col0<L, VEC>(w + j * W, lane); };
  auto load = [&](RowIn<T, CK, VEC>& in, long long row, int j) {
    const bool live = L == 32 || row < a.R;
    const size_t at = (size_t)(live ? row : 0) * a.C;
    const int C = live ? a.C : 0, P = live ? a.P : 0, c0 = c_of(j);
    if (!live) row = 0;
    in.dn = load_chunk<T, L, VEC>(static_cast<const T*>(a.dn) + at, c0, C);
    if (a.dh) in.dh = load_chunk<T, L, VEC>(static_cast<const T*>(a.dh) + at, c0, C);
    if constexpr (CK) {
      in.q = load_bytes<L, VEC>(a.q + (size_t)row * a.P, c0, P);
      const int8_t* e = a.e + (size_t)row * groups;
      if constexpr (VEC) in.e.x = c0 < P ? (uint32_t)(int)e[c0 / kQ8Group] : 0u;
      else in.e = load_exps<L>(e, w + j * W, groups);
    } else {
      in.h = load_chunk<T, L, VEC>(static_cast<const T*>(a.h) + at, c0, C);
    }
  };
  auto xhat = [&](const RowIn<T, CK, VEC>& in, float rstd, float2 (&xh)[4]) {
    if constexpr (CK) {
      biased(in.q, xh);
      if constexpr (VEC) {
        const float s = ckpt_step((int)in.e.x) * rstd;
#pragma unroll
        for (int i = 0; i < 4; ++i) xh[i] = mul2(add2(xh[i], f2(-kBias)), f2(s));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float& t = i & 1 ? xh[i / 2].y : xh[i / 2].x;
          t = (t - kBias) * (ckpt_step(exp_of<L>(in.e, i)) * rstd);
        }
      }
    } else {
      to_pairs(in.h, xh);
#pragma unroll
      for (int i = 0; i < 4; ++i) xh[i] = mul2(xh[i], f2(rstd));
    }
  };
  Chunk<T> g[NCH];
  float2 acc[NCH][4];
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    g[j] = load_chunk<T, L, VEC>(static_cast<const T*>(a.gamma), c_of(j), a.C);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = f2(0.f);
  }
  const long long step = (long long)gridDim.x * rpb;
  int slot = 0;
  // Every warp of a row sees the same rows, so their barriers match.
  // Parts of a warp stay in the loop together (their shuffles take every lane).
  const int first_of_warp = L == 32 ? rib : (threadIdx.x >> 5) * (32 / L);
  for (long long row = (long long)blockIdx.x * rpb + rib; row - rib + first_of_warp < a.R; row += step, slot ^= 1) {
    const bool live = L == 32 || row < a.R;
    RowIn<T, CK, VEC> in[NCH];
#pragma unroll
    for (int j = 0; j < NCH; ++j) load(in[j], row, j);
    const float rstd = live ? a.rstd[row] : 0.f;
    float2 dot2 = f2(0.f), xh[NCH][4], t[NCH][4];
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float2 gm[4];
      xhat(in[j], rstd, xh[j]);
      to_pairs(in[j].dn, t[j]);
      to_pairs(g[j], gm);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[j][i] = fma2(t[j][i], xh[j][i], acc[j][i]);
        t[j][i] = mul2(t[j][i], gm[i]);
        dot2 = fma2(t[j][i], xh[j][i], dot2);
      }
    }
    const float m = -row_sum<L>(dot2.x + dot2.y, my_red, slot, w, W, 1 + rib) * inv_n;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) t[j][i] = mul2(fma2(xh[j][i], f2(m), t[j][i]), f2(rstd));
      if (a.dh) {
        float2 r[4];
        to_pairs(in[j].dh, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) t[j][i] = add2(t[j][i], r[i]);
      }
      if (live) store_chunk<T, L, VEC>(static_cast<T*>(a.dx) + (size_t)row * a.C, c_of(j), a.C, t[j]);
    }
  }
  // The block's partials: parts of a warp in a tree of shuffles, then sets of warps
  // (a row's, or one) in order, the first set adding the others' to its own.
  // (Taking turns at one row of partials, a barrier a turn: 17 us for 3363 rows of 32,
  // 8 like this.)
  float* pg = a.pg + (size_t)blockIdx.x * a.C;
  const int sets = L == 32 ? rpb : blockDim.x / 32, set = L == 32 ? rib : threadIdx.x >> 5;
  auto each = [&](auto f) {
#pragma unroll
    for (int j = 0; j < NCH; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = col<L, VEC>(c_of(j), i);
        float& v = i & 1 ? acc[j][i / 2].y : acc[j][i / 2].x;
        f(v, c);
      }
  };
  each([&](float& v, int c) {
#pragma unroll
    for (int o = L; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (set > 0 && c < a.C) cols[(set - 1) * a.C + c] = v;
  });
  if (sets > 1) __syncthreads();
  if (set > 0) return;
#pragma unroll 1
  for (int r = 1; r < sets; ++r)
    each([&](float& v, int c) {
      if (c < a.C) v += cols[(r - 1) * a.C + c];
    });
  each([&](float& v, int c) {
    if (c < a.C) pg[c] = v;
  });
}

// How rows are spread: L lanes of W warps a row, NCH blocks of 8 * L columns
// each, rpb rows a thread block: as many as ten warps hold, eight of one warp,
// one where a row takes six warps or more.  Short rows take part of a warp:
// 1,000,000 rows of 40 columns 296 us with a warp a row, 100 with 8 lanes.  One
// block a warp where 16 warps hold the row: 65536 x 1280 in 211 us with a warp a
// row, 122 with five.  Five warps a row fill an SM best (two rows a block, 30
// warps); with one row a block and at most three blocks an SM, six and seven
// warps a row leave it 18 and 21: of as many elements, with dh, rows of 1280
// columns take 123 us, 1288 204, 1536 176, 1792 163, 2048 151, 2304 139, 2560 135.
struct Spread {
  int L, W, nch, rpb, threads;
};
Spread spread_of(int C) {
  const int P = q8_pitch(C), blocks = (P + 255) / 256;
  Spread s;
  s.L = P <= 64 ? 8 : P <= 128 ? 16 : 32;
  s.nch = blocks <= 16 ? 1 : blocks <= 32 ? 2 : 4;
  s.W = (blocks + s.nch - 1) / s.nch;
  s.rpb = s.W == 1 ? 256 / s.L : s.W < 10 ? 10 / s.W : 1;
  s.threads = s.L * s.W * s.rpb;
  return s;
}

template <typename T, bool CK, bool VEC>
cudaError_t rows_bwd(const RowsBwd& a, cudaStream_t st) {
  const Spread s = spread_of(a.C);
  const int sets = s.L == 32 ? s.rpb : s.threads / 32;
  const size_t smem = (size_t)(sets - 1) * a.C * sizeof(float);  // 9 KB at most
  auto k = s.L == 8      ? k_rows_bwd<T, 8, 1, CK, VEC>
           : s.L == 16   ? k_rows_bwd<T, 16, 1, CK, VEC>
           : s.nch == 1  ? k_rows_bwd<T, 32, 1, CK, VEC>
           : s.nch == 2  ? k_rows_bwd<T, 32, 2, CK, VEC>
                         : k_rows_bwd<T, 32, 4, CK, VEC>;
  return launch_k(k, dim3((unsigned)rows_bwd_blocks(a.R, a.C)), dim3(s.threads), smem, st, 1, a, s.W, s.rpb);
}

template <typename T>
cudaError_t rows_bwd_t(const RowsBwd& a, cudaStream_t st) {
  if (rows_aligned(a.C, sizeof(T))) return a.h ? rows_bwd<T, false, true>(a, st) : rows_bwd<T, true, true>(a, st);
  return a.h ? rows_bwd<T, false, false>(a, st) : rows_bwd<T, true, false>(a, st);
}

}  // namespace

// Blocks resident at once (at most three a SM, each with a partial row).
int rows_bwd_blocks(long long R, int C) {
  const Spread s = spread_of(C);
  const long long want = (R + s.rpb - 1) / s.rpb;
  const int fit = 65536 / (s.threads * (s.nch > 1 ? 128 : kRegs)), per_sm = fit < 3 ? fit : 3;
  long long most = (long long)sm_count() * per_sm;
  if (most > kRowsBwdMaxBlocks) most = kRowsBwdMaxBlocks;
  return (int)(want < most ? want : most);
}
cudaError_t launch_rows_bwd(const RowsBwd& a, cudaStream_t st) { RMX_BY_DTYPE(a.dtype, return rows_bwd_t<T>(a, st)) }

}  // namespace rmx
