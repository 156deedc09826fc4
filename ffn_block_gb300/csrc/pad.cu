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
// others a warp a row.  A step with 32 such copies: 113 us by elements and 136 by
// rows for 8 samples of T = 8, D = 72, H = 148; 571 us and 535 for 256 samples of
// T = 10, D = 1230, H = 2460 (with the elements' form up to 2^22).  2^18 and 2^20
// measured alike.
constexpr size_t kPadSmall = 1 << 19;

// Destination and source as rows of dw and sw elements (a half each), dn and sn
// of them to an outer index; what the source does not have is zero.  The
// destination is written in order.
struct Run {
  int dw, sw, dn, sn;
  long long total;
};

// Small copies: one thread per destination element, its place from 32-bit
// divisions, so that nothing waits for the element before it.
template <typename E>
__global__ void __launch_bounds__(256) k_pad_small(const E* __restrict__ src, E* __restrict__ dst, const Run p) {
  pdl_enter();
  const uint32_t idx = blockIdx.x * 256 + threadIdx.x;
  if (idx >= (uint32_t)p.total) return;
  const uint32_t d = idx / (uint32_t)p.dw, c = idx - d * p.dw, o = d / (uint32_t)p.dn, r = d - o * p.dn;
  dst[idx] = r < (uint32_t)p.sn && c < (uint32_t)p.sw ? src[((size_t)o * p.sn + r) * p.sw + c] : E(0);
}

// Large ones: a warp takes up to 1024 columns of a destination row at a time (its
// place is divided out once), neighbouring lanes neighbouring columns.  8192 rows
// of 1001 16-bit values: 17 us; 41 an element a thread with 64-bit divisions, 23
// as runs of 1024 elements across rows, whose loads wait for the place.
template <typename E>
__global__ void __launch_bounds__(256) k_pad_copy(const E* __restrict__ src, E* __restrict__ dst, const Run p,
                                                  int segs, long long items) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const long long step = (long long)gridDim.x * 8;
  const bool narrow = items < (1ll << 31);  // 32-bit divisions
  for (long long it = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += step) {
    const long long d = narrow ? (long long)((uint32_t)it / (uint32_t)segs) : it / segs;
    const long long o = narrow ? (long long)((uint32_t)d / (uint32_t)p.dn) : d / p.dn;
    const int r = (int)(d - o * p.dn), c0 = (int)(it - d * segs) * 1024, c1 = min(p.dw, c0 + 1024);
    const int real = r < p.sn ? p.sw : 0;
    const E* in = src + (o * p.sn + r) * p.sw;
    E* out = dst + d * p.dw;
#pragma unroll 8
    for (int c = c0 + lane; c < c1; c += 32) out[c] = c < real ? in[c] : E(0);
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
  const int hs = m.cols / m.halves, hsp = m.cols_p / m.halves;
  Run p{hsp, hs, m.rows_p * m.halves, m.rows * m.halves, (long long)m.outer * m.rows_p * m.cols_p};
  if (!pack) p = Run{hs, hsp, m.rows * m.halves, m.rows_p * m.halves, (long long)m.outer * m.rows * m.cols};
  if (p.total == 0) return cudaSuccess;
  auto go = [&](auto e) {
    using E = decltype(e);
    const E* from = static_cast<const E*>(src);
    E* to = static_cast<E*>(dst);
    if (p.total <= (long long)kPadSmall)
      return launch_k(k_pad_small<E>, dim3((unsigned)((p.total + 255) / 256)), dim3(256), 0, st, 1, from, to, p);
    const int segs = (p.dw + 1023) / 1024;
    const long long items = p.total / p.dw * segs, want = (items + 7) / 8, most = (long long)sm_count() * 16;
    return launch_k(k_pad_copy<E>, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, st, 1, from, to, p, segs,
                    items);
  };
  return dtype == 0 ? go(uint32_t{}) : go(uint16_t{});
}

}  // namespace rmx
