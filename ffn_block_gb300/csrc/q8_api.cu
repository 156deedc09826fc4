// C-ABI layer of the 8-bit operators: argument checks, workspace layouts and
// launch sequences.  Nothing here allocates device memory or synchronises.

#include <limits.h>

#include "api.h"
#include "common.cuh"
#include "q8.h"

using namespace rmx;

namespace {

bool layer_ok(const rmx_layer* l) {
  if (!l || l->M < 0 || l->G < 1 || l->K < 1 || l->N < 1 || !storage_ok(l->dtype)) return false;
  if (l->K > (1 << 20) || l->N > (1 << 20) || l->G > 65535) return false;
  const long long G = l->G, most = 1ll << 30;
  return G * l->M <= most && G * l->K <= most && G * l->N <= most;
}
// A group's weights as the tensor maps take them: int8 [N][P] and 16-bit [K][N]
// strides below 2^40 bytes.
bool weights_fit(const rmx_layer& l) { return (long long)q8_pitch(l.K) * ((l.N + 7) / 8 * 8) < (1ll << 39); }
// Workspace of the weight gradient: the unpacked activation [M, G, Kp], and
// for rows that are not a whole number of 16-byte vectors (16-bit types)
// padded copies of dy and dw; float32: the bias gradient's column partials.
struct WgradWs {
  int Kp, Np;
  bool padded;
  size_t x, dy, dw, part, total;
};
WgradWs wgrad_ws(const rmx_layer& l) {
  WgradWs w;
  const size_t e = storage_bytes(l.dtype), rows = (size_t)l.M * l.G;
  w.padded = l.dtype != RMX_F32 && (l.K % 8 || l.N % 8);
  w.Kp = w.padded ? (l.K + 7) / 8 * 8 : l.K;
  w.Np = w.padded ? (l.N + 7) / 8 * 8 : l.N;
  size_t o = 0;
  w.x = o;
  o = up256(o + rows * w.Kp * e);
  w.dy = w.dw = o;
  if (w.padded) {
    o = up256(o + rows * w.Np * e);
    w.dw = o;
    o = up256(o + (size_t)l.G * w.Kp * w.Np * e);
  }
  w.part = o;
  if (l.dtype == RMX_F32) o += (size_t)colpart_slices(l.M, (long long)l.G * l.N) * l.G * l.N * sizeof(float);
  w.total = up256(o);
  return w;
}

char* at(void* p, size_t o) { return static_cast<char*>(p) + o; }

}  // namespace

extern "C" {

int rmx_q8_pitch(int cols) { return cols < 1 || cols > (1 << 24) ? 0 : q8_pitch(cols); }

rmx_status rmx_rms_norm_q8(const rmx_rows* shape, float eps, const void* x, const void* r, const void* gamma,
                           void* h, void* y, int8_t* q, float* scale, float* rstd, rmx_stream stream) {
  if (!rows_ok(shape) || !(eps >= 0.f)) return RMX_ERR_INVALID_ARG;
  if ((!y && !q) || (q != nullptr) != (scale != nullptr)) return RMX_ERR_INVALID_ARG;
  if (shape->cols > kQ8MaxCols) return RMX_ERR_UNSUPPORTED;
  if (shape->rows == 0) return RMX_OK;
  RMX_TRY(check_ptr(x));
  RMX_TRY(check_ptr(gamma));
  for (const void* p : {r, (const void*)h, (const void*)y, (const void*)q, (const void*)scale, (const void*)rstd})
    RMX_TRY(check_opt(p));
  if (y && (y == x || y == r || y == h)) return RMX_ERR_INVALID_ARG;
  RowsFwd a{shape->rows, shape->cols, q8_pitch(shape->cols), shape->dtype, 1, eps, x, r, gamma, h, y, q, scale, rstd};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Launch l("rms_norm_q8", st);
  return l.done(launch_rows_fwd(a, st));
}

rmx_status rmx_quant_rows_q8(const rmx_rows* shape, const void* x, int8_t* q, float* scale, rmx_stream stream) {
  if (!rows_ok(shape)) return RMX_ERR_INVALID_ARG;
  if (shape->cols > kQ8MaxCols) return RMX_ERR_UNSUPPORTED;
  if (shape->rows == 0) return RMX_OK;
  RMX_TRY(check_ptr(x));
  RMX_TRY(check_ptr(q));
  RMX_TRY(check_ptr(scale));
  RowsFwd a{shape->rows, shape->cols, q8_pitch(shape->cols), shape->dtype, 0, 0.f, x, nullptr, nullptr, nullptr,
            nullptr, q, scale, nullptr};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Launch l("quant_rows_q8", st);
  return l.done(launch_rows_fwd(a, st));
}

rmx_status rmx_dequant_rows_q8(const rmx_rows* shape, const int8_t* q, const float* scale, void* x,
                               rmx_stream stream) {
  if (!rows_ok(shape)) return RMX_ERR_INVALID_ARG;
  if (shape->rows == 0) return RMX_OK;
  RMX_TRY(check_ptr(q));
  RMX_TRY(check_ptr(scale));
  RMX_TRY(check_ptr(x));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Launch l("dequant_rows_q8", st);
  return l.done(launch_dequant_rows(shape->rows, shape->cols, shape->dtype, q, scale, x, st));
}

size_t rmx_rms_norm_backward_workspace_bytes(const rmx_rows* shape) {
  if (!rows_ok(shape) || shape->cols > kQ8MaxCols) return 0;
  return up256((size_t)kRowsBwdMaxBlocks * shape->cols * sizeof(float));
}

rmx_status rmx_rms_norm_backward(const rmx_rows* shape, const void* dn, const void* dh, const void* h,
                                 const int8_t* q, const int8_t* exps, const float* rstd, const void* gamma,
                                 void* dx, void* dgamma, void* ws, size_t ws_bytes, rmx_stream stream) {
  if (!rows_ok(shape)) return RMX_ERR_INVALID_ARG;
  if (shape->cols > kQ8MaxCols) return RMX_ERR_UNSUPPORTED;
  RMX_TRY(check_ptr(dgamma));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (shape->rows == 0)
    return cudaMemsetAsync(dgamma, 0, shape->cols * storage_bytes(shape->dtype), st) == cudaSuccess ? RMX_OK : RMX_ERR_CUDA;
  if ((h != nullptr) == (q != nullptr) || (q != nullptr) != (exps != nullptr)) return RMX_ERR_INVALID_ARG;
  for (const void* p : {dn, (const void*)rstd, gamma, (const void*)dx, (const void*)ws}) RMX_TRY(check_ptr(p));
  for (const void* p : {dh, h, (const void*)q, (const void*)exps}) RMX_TRY(check_opt(p));
  if (dx == h) return RMX_ERR_INVALID_ARG;
  if (ws_bytes < rmx_rms_norm_backward_workspace_bytes(shape)) return RMX_ERR_WORKSPACE;
  const int blocks = rows_bwd_blocks(shape->rows, shape->cols);
  RowsBwd a{shape->rows, shape->cols, q8_pitch(shape->cols), shape->dtype, dn, dh, h, q, exps, rstd, gamma, dx,
            static_cast<float*>(ws)};
  {
    Launch l("rms_norm_backward", st);
    RMX_TRY(l.done(launch_rows_bwd(a, st)));
  }
  const ColsumJob job{a.pg, dgamma, blocks, shape->cols};
  Launch l("rms_norm_dgamma", st);
  return l.done(launch_colsums(&job, 1, shape->dtype, st));
}

rmx_status rmx_weight_q8(const rmx_layer* layer, const void* w, int8_t* q, float* scale, rmx_stream stream) {
  if (!layer_ok(layer)) return RMX_ERR_INVALID_ARG;
  if (!weights_fit(*layer)) return RMX_ERR_UNSUPPORTED;
  RMX_TRY(check_ptr(w));
  RMX_TRY(check_ptr(q));
  RMX_TRY(check_ptr(scale));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Launch l("weight_q8", st);
  return l.done(launch_weight_q8(layer->G, layer->K, layer->N, layer->dtype, w, q, scale, st));
}

rmx_status rmx_linear_q8(const rmx_layer* layer, const int8_t* a, const float* a_scale, const int8_t* w,
                         const float* w_scale, const void* bias, const void* resid, void* out, rmx_stream stream) {
  if (!layer_ok(layer)) return RMX_ERR_INVALID_ARG;
  if (!weights_fit(*layer)) return RMX_ERR_UNSUPPORTED;
  if (layer->M == 0) return RMX_OK;
  for (const void* p : {(const void*)a, (const void*)a_scale, (const void*)w, (const void*)w_scale, (const void*)out})
    RMX_TRY(check_ptr(p));
  RMX_TRY(check_opt(bias));
  RMX_TRY(check_opt(resid));
  const LinearQ8 d{layer->M, layer->G, layer->K, layer->N, q8_pitch(layer->K), layer->dtype, a, w, a_scale, w_scale,
                   bias, resid, out};
  if (!linear_q8_supported(d)) return RMX_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Launch l("linear_q8", st);
  return l.done(launch_linear_q8(d, device_error_word(), st));
}

rmx_status rmx_ckpt8_pack(const rmx_rows* shape, const void* x, int8_t* q, int8_t* exps, rmx_stream stream) {
  if (!rows_ok(shape)) return RMX_ERR_INVALID_ARG;
  if (shape->rows == 0) return RMX_OK;
  RMX_TRY(check_ptr(x));
  RMX_TRY(check_ptr(q));
  RMX_TRY(check_ptr(exps));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Launch l("ckpt8_pack", st);
  return l.done(launch_ckpt_pack(shape->rows, shape->cols, shape->dtype, x, q, exps, st));
}

rmx_status rmx_ckpt8_unpack(const rmx_rows* shape, const int8_t* q, const int8_t* exps, void* x, rmx_stream stream) {
  if (!rows_ok(shape)) return RMX_ERR_INVALID_ARG;
  if (shape->rows == 0) return RMX_OK;
  RMX_TRY(check_ptr(x));
  RMX_TRY(check_ptr(q));
  RMX_TRY(check_ptr(exps));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Launch l("ckpt8_unpack", st);
  return l.done(launch_ckpt_unpack(shape->rows, shape->cols, shape->dtype, q, exps, x, shape->cols, st));
}

size_t rmx_ckpt8_wgrad_workspace_bytes(const rmx_layer* layer) {
  if (!layer_ok(layer) || !weights_fit(*layer)) return 0;
  return wgrad_ws(*layer).total;
}

rmx_status rmx_ckpt8_wgrad(const rmx_layer* layer, const int8_t* q, const int8_t* exps, const void* dy, void* dw,
                           void* db, void* ws, size_t ws_bytes, rmx_stream stream) {
  if (!layer_ok(layer)) return RMX_ERR_INVALID_ARG;
  const rmx_layer& l = *layer;
  if (!weights_fit(l)) return RMX_ERR_UNSUPPORTED;
  RMX_TRY(check_ptr(dw));
  RMX_TRY(check_opt(db));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const size_t e = storage_bytes(l.dtype);
  if (l.M == 0) {
    if (cudaMemsetAsync(dw, 0, (size_t)l.G * l.K * l.N * e, st) != cudaSuccess) return RMX_ERR_CUDA;
    if (db && cudaMemsetAsync(db, 0, (size_t)l.G * l.N * e, st) != cudaSuccess) return RMX_ERR_CUDA;
    return RMX_OK;
  }
  for (const void* p : {(const void*)q, (const void*)exps, dy, (const void*)ws}) RMX_TRY(check_ptr(p));
  const WgradWs w = wgrad_ws(l);
  if (ws_bytes < w.total) return RMX_ERR_WORKSPACE;
  const long long rows = (long long)l.M * l.G;
  {
    Launch la("ckpt8_unpack", st);
    RMX_TRY(la.done(launch_ckpt_unpack(rows, l.K, l.dtype, q, exps, at(ws, w.x), w.Kp, st)));
  }
  const void* dyp = dy;
  void* dwp = dw;
  if (w.padded) {
    dyp = at(ws, w.dy);
    dwp = at(ws, w.dw);
    const PadMap m{1, (int)rows, (int)rows, l.N, w.Np, 1};
    Launch la("pad_in", st);
    RMX_TRY(la.done(launch_pad_copy(dy, at(ws, w.dy), l.dtype, m, true, st)));
  }
  GemmDesc d{GEMM_WGRAD, EPI_STORE, l.dtype, w.Kp, w.Np, l.M, l.G, at(ws, w.x), dyp, dwp, nullptr, nullptr};
  // The tensor-core product adds up dy's columns as they pass; the strict
  // float32 one leaves them to a pass of their own.
  const bool fused = l.dtype != RMX_F32;
  if (fused) {
    d.colsum = db;
    d.colsum_n = l.N;
  }
  RMX_TRY(run_gemm("ckpt8_wgrad", d, st));
  if (w.padded) {
    const PadMap m{l.G, l.K, w.Kp, l.N, w.Np, 1};
    Launch la("pad_out", st);
    RMX_TRY(la.done(launch_pad_copy(dwp, dw, l.dtype, m, false, st)));
  }
  if (db && !fused) {
    const long long J = (long long)l.G * l.N;
    const int slices = colpart_slices(l.M, J);
    float* part = reinterpret_cast<float*>(at(ws, w.part));
    {
      Launch la("ckpt8_dbias", st);
      RMX_TRY(la.done(launch_colpart(l.M, J, static_cast<const float*>(dy), part, static_cast<float*>(db), st)));
    }
    if (slices > 1) {
      const ColsumJob job{part, db, slices, (int)J};
      Launch la("ckpt8_dbias_sum", st);
      RMX_TRY(la.done(launch_colsums(&job, 1, l.dtype, st)));
    }
  }
  return RMX_OK;
}

}  // extern "C"
