// Zero-padded staging copies for blocks whose D or H is not a multiple of 8.
//
// The kernels address rows in whole 16-byte vectors and the tensor-core GEMM
// needs 16-byte row strides, so such a block runs on copies whose rows are
// padded with zeros to a multiple of 8 elements: x, dy and the parameters are
// gathered into padded buffers before the passes, y, dx and the gradients are
// gathered back afterwards.  The zeros are exact no-ops for the contractions
// (zero rows and columns of the weights), and the LayerNorm passes take their
// means over the real columns only.  Every destination element is written (a
// padded place with 0), so nothing needs clearing first.

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace rmx {
namespace {

// Copies of up to this many elements take an element a thread (k_pad_small), the
// others a warp a row.  A step with 32 such copies: 116 us by elements and 136 by
// rows for 8 samples of T = 8, D = 72, H = 148; 571 us and 535 for 256 samples of
// T = 10, D = 1230, H = 2460 (with the elements' form up to 2^22).  2^18 and 2^20
// measured alike.
constexpr size_t kPadSmall = 1 << 19;

// Small copies: one thread per destination element, its place from 32-bit
// divisions, so that nothing waits for the element before it.
template <typename E>
__global__ void __launch_bounds__(256) k_pad_small(const E* __restrict__ src, E* __restrict__ dst, PadMap m,
                                                   int pack, uint32_t total) {
  pdl_enter();
  const uint32_t idx = blockIdx.x * 256 + threadIdx.x;
  if (idx >= total) return;
  const uint32_t hs = m.cols / m.halves, hsp = m.cols_p / m.halves;
  const uint32_t dcols = pack ? m.cols_p : m.cols, drows = pack ? m.rows_p : m.rows;
  const uint32_t d = idx / dcols, c = idx - d * dcols, o = d / drows, r = d - o * drows;
  if (pack) {
    // padded (o, r, c) <- logical (o, r, h * hs + cc) with c = h * hsp + cc
    const uint32_t h = c / hsp, cc = c - h * hsp;
    dst[idx] = r < (uint32_t)m.rows && cc < hs ? src[(size_t)(o * m.rows + r) * m.cols + h * hs + cc] : E(0);
  } else {
    // logical (o, r, c) <- padded (o, r, h * hsp + cc) with c = h * hs + cc
    const uint32_t h = c / hs, cc = c - h * hs;
    dst[idx] = src[(size_t)(o * m.rows_p + r) * m.cols_p + h * hsp + cc];
  }
}

// Large ones: eight warps a CTA, a warp takes up to 1024 columns of one half of
// a destination row at a time (its place is worked out once), neighbouring lanes
// neighbouring columns.  8192 rows of 1001 16-bit values: 41 us an element a
// thread, 17 us like this.
template <typename E>
__global__ void __launch_bounds__(256) k_pad_copy(const E* __restrict__ src, E* __restrict__ dst, PadMap m,
                                                  int pack) {
  pdl_enter();
  const int hs = m.cols / m.halves, hsp = m.cols_p / m.halves;
  const int dcols = pack ? m.cols_p : m.cols, drows = pack ? m.rows_p : m.rows;
  const int lane = threadIdx.x & 31;
  const int W = pack ? hsp : hs, segs = (W + 1023) / 1024, per_row = m.halves * segs;
  const long long items = (long long)m.outer * drows * per_row, step = (long long)gridDim.x * 8;
  const bool narrow = items < (1ll << 31);  // one 32-bit division for the place
  for (long long it = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += step) {
    const long long d = narrow ? (long long)((uint32_t)it / (uint32_t)per_row) : it / per_row;
    const long long o = narrow ? (long long)((uint32_t)d / (uint32_t)drows) : d / drows;
    const int r = (int)(d - o * drows), part = (int)(it - d * per_row), h = part / segs;
    const int c0 = (part - h * segs) * 1024, c1 = min(W, c0 + 1024);
    E* out = dst + d * dcols + (long long)h * W;
    if (pack) {
      // padded (o, r, h * hsp + cc) <- logical (o, r, h * hs + cc)
      const E* in = src + (o * m.rows + r) * (long long)m.cols + (long long)h * hs;
#pragma unroll 8
      for (int cc = c0 + lane; cc < c1; cc += 32) out[cc] = r < m.rows && cc < hs ? in[cc] : E(0);
    } else {
      // logical (o, r, h * hs + cc) <- padded (o, r, h * hsp + cc)
      const E* in = src + (o * m.rows_p + r) * (long long)m.cols_p + (long long)h * hsp;
#pragma unroll 8
      for (int cc = c0 + lane; cc < c1; cc += 32) out[cc] = in[cc];
    }
  }
}

// dst[g][c][r] = src[g * gs + r * rs + c] for r < R, 0 for R <= r < Rp: one
// 32 x 32 tile per CTA through shared memory, reads along c and writes
// along r coalesced.
__global__ void __launch_bounds__(256) k_transpose_f32(const float* __restrict__ src, float* __restrict__ dst,
                                                       int R, int Cc, long long gs, long long rs, int Rp) {
  pdl_enter();
  __shared__ float tile[32][33];
  const int g = blockIdx.z, c0 = blockIdx.x * 32, r0 = blockIdx.y * 32;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const float* s = src + (size_t)g * gs;
#pragma unroll
  for (int k = 0; k < 32; k += 8) {
    const int r = r0 + ty + k, c = c0 + tx;
    tile[ty + k][tx] = (r < R && c < Cc) ? s[(size_t)r * rs + c] : 0.f;
  }
  __syncthreads();
  float* d = dst + (size_t)g * Cc * Rp;
#pragma unroll
  for (int k = 0; k < 32; k += 8) {
    const int c = c0 + ty + k, r = r0 + tx;
    if (c < Cc && r < Rp) d[(size_t)c * Rp + r] = tile[tx][ty + k];
  }
}

}  // namespace

cudaError_t launch_transpose_f32(const float* src, float* dst, int G, int R, int Cc, long long gs, long long rs,
                                 int Rp, cudaStream_t st) {
  if (G < 0 || R < 0 || Cc < 0 || Rp < R) return cudaErrorInvalidValue;
  if (G == 0 || Cc == 0 || Rp == 0) return cudaSuccess;
  const dim3 grid((Cc + 31) / 32, (Rp + 31) / 32, G);
  return launch_k(k_transpose_f32, grid, dim3(256), 0, st, 1, src, dst, R, Cc, gs, rs, Rp);
}

cudaError_t launch_pad_copy(const void* src, void* dst, int dtype, const PadMap& m, bool pack, cudaStream_t st) {
  if (m.outer < 0 || m.rows < 0 || m.rows > m.rows_p || m.cols > m.cols_p || m.halves < 1 ||
      m.cols % m.halves || m.cols_p % m.halves)
    return cudaErrorInvalidValue;
  const size_t total = (size_t)m.outer * (pack ? (size_t)m.rows_p * m.cols_p : (size_t)m.rows * m.cols);
  if (total == 0) return cudaSuccess;
  const int w = (pack ? m.cols_p : m.cols) / m.halves;
  const size_t items = (size_t)m.outer * (pack ? m.rows_p : m.rows) * m.halves * ((w + 1023) / 1024);
  auto go = [&](auto e) {
    using E = decltype(e);
    const E* from = static_cast<const E*>(src);
    E* to = static_cast<E*>(dst);
    if (total <= kPadSmall)
      return launch_k(k_pad_small<E>, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, st, 1, from, to, m,
                      pack ? 1 : 0, (uint32_t)total);
    const size_t want = (items + 7) / 8, most = (size_t)sm_count() * 16;
    return launch_k(k_pad_copy<E>, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, st, 1, from, to, m,
                    pack ? 1 : 0);
  };
  return dtype == 0 ? go(uint32_t{}) : go(uint16_t{});
}

}  // namespace rmx
