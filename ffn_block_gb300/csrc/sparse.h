// Internal interface between the C-ABI layer (sparse_api.cu) and the kernels of
// the sparse layer: dropout and layer norm, routing to experts, 8-bit floating
// rows and their products.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace rmx {

// ---------------------------------------------------------------- dropout, layer norm
// Dropout as the kernels take it: an element is kept where its 16 bits are at
// least thresh, and multiplied by scale.
enum DropMode { DROP_NONE = 0, DROP_BITS = 1, DROP_ALL = 2 };
struct Drop {
  const uint64_t* state;  // device: {seed, offset}
  int mode;
  uint32_t thresh;
  float scale;
};
cudaError_t launch_dropout(long long R, int C, int dtype, const Drop& d, const void* x, const void* r, void* out,
                           cudaStream_t st);

// Longest row of the layer norm: 16 warps x 4 blocks of 256 columns.
constexpr int kLnMaxCols = 16384;
struct LnFwd {
  long long R;
  int C, dtype;
  float eps;
  Drop drop;
  const void *x, *r, *gamma, *beta;  // r, gamma, beta may be null
  void *h, *y;                       // h may be null
  float *mean, *rstd;                // may be null
};
cudaError_t launch_layer_norm(const LnFwd& a, cudaStream_t st);

// Column partials of dgamma and dbeta: [ln_bwd_blocks][C] each.
struct LnBwd {
  long long R;
  int C, dtype;
  Drop drop;
  const void *dy, *dh, *h;  // dh may be null
  const float *mean, *rstd;
  const void* gamma;        // may be null
  void *dr, *dx;            // dx may be null
  float *pg, *pb;
};
constexpr int kLnBwdMaxBlocks = 512;
int ln_bwd_rows_blocks(const LnBwd& a);
cudaError_t launch_layer_norm_bwd(const LnBwd& a, cudaStream_t st);
// dgamma, dbeta (either may be null) from the partials.
cudaError_t launch_layer_norm_params(const LnBwd& a, void* dgamma, void* dbeta, cudaStream_t st);

// ---------------------------------------------------------------- routing
constexpr int kMaxExperts = 1024;
struct Routes {
  int T, k, E, C, dtype;
  int S;  // T * k
};
// Warps that share the counting of a sort of three launches; 0: one launch sorts, of a
// CTA or a cluster.
int sort_warps(int S);
cudaError_t launch_expert_sort(const Routes& r, const int32_t* expert, int32_t* offsets, int32_t* position,
                               int32_t* source, int32_t* ws, int pass, cudaStream_t st);
cudaError_t launch_expert_gather(const Routes& r, const int32_t* source, const void* x, void* out, cudaStream_t st);
cudaError_t launch_expert_combine(const Routes& r, const int32_t* position, const float* weight, const void* y,
                                  void* out, cudaStream_t st);
cudaError_t launch_expert_combine_bwd(const Routes& r, const int32_t* position, const float* weight, const void* dout,
                                      const void* y, void* dy, float* dweight, cudaStream_t st);

// ---------------------------------------------------------------- 8-bit floating rows
constexpr int kF8Block = 128;
inline int f8_blocks(int cols) { return (cols + kF8Block - 1) / kF8Block; }
inline int f8_exps(int cols) { return (f8_blocks(cols) + 3) / 4 * 4; }
inline int f8_pitch(int cols) { return f8_blocks(cols) * kF8Block; }
// Blocks of 128 rows that M rows in G groups take at most.
inline int ragged_blocks(int M, int G) { return M / kF8Block + (G < M ? G : M); }

// source (may be null): row i is x[source[i] / k], rows with no source in [0, R)
// are left out.  out (may be null): the gathered row itself.
struct QuantRows {
  long long R;
  int C, dtype, format;
  const void* x;
  uint8_t *q, *e;
  const int32_t* source;
  int k;
  void* out;
};
cudaError_t launch_quant_f8(const QuantRows& a, cudaStream_t st);
cudaError_t launch_dequant_f8(long long R, int C, int dtype, int format, const uint8_t* q, const uint8_t* e, void* x,
                              cudaStream_t st);

struct QuantGroups {
  int M, G, C, dtype, format;
  long long row_stride, group_stride;  // elements; ragged: group_stride 0
  const int32_t* offsets;              // null: every group has M rows
  int blocks;                          // blocks of 128 rows, of all groups (ragged: at most)
  const void* x;
  uint8_t *q, *e, *qt, *et;
  long long q_row, q_group;            // rows of q between rows and groups
  int tp, tep;                         // pitches of qt and et (not with offsets)
  float* part;                         // column sums [blocks][C], may be null
  void* sums;
};
cudaError_t launch_quant_f8_groups(const QuantGroups& a, cudaStream_t st);
cudaError_t launch_quant_f8_sums(const QuantGroups& a, cudaStream_t st);

// ---------------------------------------------------------------- their product
// out[m, g, n] = sum_k t[m, g, k] * w[g, n, k] + bias + resid.  `t` rows are the
// tokens (or, for a weight gradient, the input's columns) and `w` rows the
// channels.
struct LinearF8 {
  int M, G, K, N, dtype;
  int t_format, w_format;
  const int32_t* offsets;  // null: groups of equal size
  bool wgrad;
  const uint8_t *t, *te, *w, *we;
  const void *bias, *resid;
  void* out;
};
bool linear_f8_supported(const LinearF8& d);
cudaError_t launch_linear_f8(const LinearF8& d, unsigned int* err, cudaStream_t st);

}  // namespace rmx
