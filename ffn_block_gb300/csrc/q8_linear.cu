// Product of int8 rows with scales per token and channel:
//   out[m,g,n] = (sum_k a[m,g,k] * w[g,n,k]) * sa[m,g] * sw[g,n] + bias[g,n] + resid[m,g,n]
//
// 64 x 64 output tiles, the int8 operands staged in shared memory 32 columns
// at a time, four products an instruction (dp4a) into exact int32 sums.

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "q8.h"

namespace rmx {
namespace {

template <typename T>
__global__ void __launch_bounds__(256) k_linear_q8(const LinearQ8 d) {
  pdl_enter();
  __shared__ int sa[64][9], sw[64][9];
  const int g = blockIdx.z, m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int lr = threadIdx.x >> 2, lw = (threadIdx.x & 3) * 2;  // staged row, first word
  int acc[4][4] = {};
  const bool am = m0 + lr < d.M, wn = n0 + lr < d.N;
  const int2* pa = reinterpret_cast<const int2*>(d.a + ((size_t)(am ? m0 + lr : 0) * d.G + g) * d.P) + lw / 2;
  const int2* pw = reinterpret_cast<const int2*>(d.w + ((size_t)g * d.N + (wn ? n0 + lr : 0)) * d.P) + lw / 2;
  for (int k0 = 0; k0 < d.P; k0 += 32) {
    const int2 va = am ? pa[k0 / 8] : make_int2(0, 0), vw = wn ? pw[k0 / 8] : make_int2(0, 0);
    __syncthreads();
    sa[lr][lw] = va.x;
    sa[lr][lw + 1] = va.y;
    sw[lr][lw] = vw.x;
    sw[lr][lw + 1] = vw.y;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      int x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = sa[ty + 16 * i][k];
        y[i] = sw[tx + 16 * i][k];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(x[i], y[j], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + ty + 16 * i;
    if (m >= d.M) continue;
    const float s = d.sa[(size_t)m * d.G + g];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx + 16 * j;
      if (n >= d.N) continue;
      const size_t o = ((size_t)m * d.G + g) * d.N + n;
      float v = (float)acc[i][j] * s * d.sw[(size_t)g * d.N + n];
      if (d.bias) v += to_f(static_cast<const T*>(d.bias)[(size_t)g * d.N + n]);
      if (d.resid) v += to_f(static_cast<const T*>(d.resid)[o]);
      static_cast<T*>(d.out)[o] = from_f<T>(v);
    }
  }
}

}  // namespace

cudaError_t launch_linear_q8(const LinearQ8& d, unsigned int*, cudaStream_t st) {
  const dim3 grid((d.N + 63) / 64, (d.M + 63) / 64, d.G);
  switch (d.dtype) {
    case 0: return launch_k(k_linear_q8<float>, grid, dim3(256), 0, st, 1, d);
    case 1: return launch_k(k_linear_q8<bf16>, grid, dim3(256), 0, st, 1, d);
    case 2: return launch_k(k_linear_q8<f16>, grid, dim3(256), 0, st, 1, d);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace rmx
