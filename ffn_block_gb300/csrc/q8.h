// Internal interface between the C-ABI layer (q8_api.cu, api.cu) and the
// kernels of the 8-bit operators.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace rmx {

// int8 rows are padded with zeros to a multiple of 32 bytes, so that every
// row starts on a 16-byte boundary (vector access, TMA) and holds a whole
// number of 32-column checkpoint groups.
constexpr int kQ8Group = 32;
inline int q8_pitch(int cols) { return (cols + kQ8Group - 1) / kQ8Group * kQ8Group; }

// Exponent of a checkpoint group that held an infinity or a NaN: all its
// values read back as NaN.
constexpr int kCkptNaN = 127;

// Longest row of the RMS norm and row quantisation passes: 512 threads x 4
// chunks of 8 columns, held in registers.
constexpr int kQ8MaxCols = 16384;

// RMS norm forward and / or row quantisation (norm == 0: n = x + r).
struct RowsFwd {
  long long R;
  int C, P, dtype, norm;
  float eps;
  const void *x, *r, *gamma;  // r may be null; gamma only with norm
  void *h, *y;                // x + r and the normalised row, storage type; may be null
  int8_t* q;                  // may be null (then scale too)
  float *scale, *rstd;        // rstd may be null
};
cudaError_t launch_rows_fwd(const RowsFwd& a, cudaStream_t st);

// values of int8 rows with one scale per row
cudaError_t launch_dequant_rows(long long R, int C, int dtype, const int8_t* q, const float* scale, void* x,
                                cudaStream_t st);
// 8-bit checkpoints: pack, and unpack into rows of `pitch` elements (columns
// C .. pitch-1 are written as zeros).
cudaError_t launch_ckpt_pack(long long R, int C, int dtype, const void* x, int8_t* q, int8_t* e, cudaStream_t st);
cudaError_t launch_ckpt_unpack(long long R, int C, int dtype, const int8_t* q, const int8_t* e, void* x, int pitch,
                               cudaStream_t st);

// RMS norm backward.  The sum h comes in the storage type (h) or as a
// checkpoint (q, e).  Column partials of dgamma: [rows_bwd_blocks][C].
struct RowsBwd {
  long long R;
  int C, P, dtype;
  const void *dn, *dh, *h;  // dh, h may be null
  const int8_t *q, *e;
  const float* rstd;
  const void* gamma;
  void* dx;
  float* pg;
};
constexpr int kRowsBwdMaxBlocks = 512;
int rows_bwd_blocks(long long R, int C);
cudaError_t launch_rows_bwd(const RowsBwd& a, cudaStream_t st);

// Column sums of a float32 [R][J] matrix over colpart_slices slices of its
// rows (the tensor-core products of the 16-bit types add up theirs): one slice
// writes out [J] itself, more write part [slices][J] for launch_colsums.
constexpr int kColpartMax = 64;
int colpart_slices(long long R, long long J);
cudaError_t launch_colpart(long long R, long long J, const float* x, float* part, float* out, cudaStream_t st);

// Weights [G][K][N] (storage type) -> int8 [G][N][P] (K-major, zero padded)
// with one scale per channel.
cudaError_t launch_weight_q8(int G, int K, int N, int dtype, const void* w, int8_t* q, float* scale,
                             cudaStream_t st);

// Product of int8 rows with scales per token and channel:
//   out[m,g,n] = (sum_k a[m,g,k] * w[g,n,k]) * sa[m,g] * sw[g,n] + bias[g,n] + resid[m,g,n]
struct LinearQ8 {
  int M, G, K, N, P, dtype;  // P: bytes per int8 row
  const int8_t *a, *w;
  const float *sa, *sw;
  const void *bias, *resid;  // may be null
  void* out;
};
bool linear_q8_supported(const LinearQ8& d);  // looks at the sizes only
cudaError_t launch_linear_q8(const LinearQ8& d, unsigned int* err, cudaStream_t st);

}  // namespace rmx
