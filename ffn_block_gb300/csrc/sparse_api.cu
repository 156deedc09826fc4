// C-ABI layer of the sparse layer's operators: argument checks, workspace
// layouts and launch sequences.  Nothing here allocates device memory or
// synchronises.

#include <math.h>

#include "api.h"
#include "common.cuh"
#include "sparse.h"

using namespace rmx;

namespace {

cudaStream_t cuda_stream(rmx_stream s) { return reinterpret_cast<cudaStream_t>(s); }

// Dropout as the kernels take it; false where p or the state's pointer is bad.
// `used` false: p is looked at, the bits are not drawn.
rmx_status drop_of(const rmx_drop* d, bool used, Drop& out) {
  out = Drop{nullptr, DROP_NONE, 0, 1.f};
  if (!d) return RMX_OK;
  if (!(d->p >= 0.f && d->p <= 1.f)) return RMX_ERR_INVALID_ARG;
  if (!used) return RMX_OK;
  const long t = lrint((double)d->p * 65536.0);
  if (t == 0) return RMX_OK;
  if (t >= 65536) {
    out.mode = DROP_ALL;
    return RMX_OK;
  }
  RMX_TRY(check_ptr(d->state));
  out.state = d->state;
  out.mode = DROP_BITS;
  out.thresh = (uint32_t)t;
  out.scale = (float)(65536.0 / (65536.0 - (double)t));
  return RMX_OK;
}

bool format_ok(int f) { return f == RMX_E4M3 || f == RMX_E5M2; }

bool routes_ok(const rmx_routes* r) {
  return r && r->tokens >= 0 && r->k >= 1 && r->k <= 64 && r->experts >= 1 && r->experts <= kMaxExperts &&
         (long long)r->tokens * r->k < (1ll << 31);
}
// With the rows that are moved.
bool moved_ok(const rmx_routes* r) {
  return routes_ok(r) && r->cols >= 1 && r->cols <= 16384 && storage_ok(r->dtype);
}
Routes routes_of(const rmx_routes* r) { return Routes{r->tokens, r->k, r->experts, r->cols, r->dtype, r->tokens * r->k}; }

bool groups_ok(const rmx_groups* g) {
  if (!g || g->M < 0 || g->G < 1 || g->C < 1 || !storage_ok(g->dtype)) return false;
  const long long G = g->G, most = 1ll << 30;
  if (g->C > (1 << 24) || G * g->C > most) return false;
  if (g->order == RMX_ORDER_RAGGED) return g->G <= kMaxExperts && g->M <= most;
  return (g->order == RMX_ORDER_TOKENS || g->order == RMX_ORDER_GROUPS) && g->M <= (1 << 24) && G * g->M <= most;
}
// Blocks of 128 rows of all groups (ragged: at most).
long long group_blocks(const rmx_groups& g) {
  return g.order == RMX_ORDER_RAGGED ? ragged_blocks(g.M, g.G) : (long long)g.G * f8_blocks(g.M);
}
// One CTA a block of rows and 128 columns.
bool groups_fit(const rmx_groups& g) { return group_blocks(g) * f8_blocks(g.C) < (1ll << 31); }

bool layer_f8_ok(const rmx_layer_f8* l, bool ragged) {
  if (!l || l->M < 0 || l->G < 1 || l->K < 1 || l->N < 1 || !storage_ok(l->dtype)) return false;
  if (!format_ok(l->a_format) || !format_ok(l->b_format)) return false;
  if (l->K > (1 << 20) || l->N > (1 << 20) || l->G > 65535) return false;
  const long long G = l->G, most = 1ll << 30;
  if (G * l->K > most || G * l->N > most) return false;
  return ragged ? l->G <= kMaxExperts && l->M <= most : G * l->M <= most;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- dropout, layer norm

rmx_status rmx_dropout(const rmx_rows* shape, const rmx_drop* drop, const void* x, const void* r, void* out,
                       rmx_stream stream) {
  if (!rows_ok(shape)) return RMX_ERR_INVALID_ARG;
  Drop d;
  RMX_TRY(drop_of(drop, true, d));
  if (shape->rows == 0) return RMX_OK;
  RMX_TRY(check_ptr(x));
  RMX_TRY(check_opt(r));
  RMX_TRY(check_ptr(out));
  cudaStream_t st = cuda_stream(stream);
  Launch l("dropout", st);
  return l.done(launch_dropout(shape->rows, shape->cols, shape->dtype, d, x, r, out, st));
}

rmx_status rmx_layer_norm(const rmx_rows* shape, float eps, const rmx_drop* drop, const void* x, const void* r,
                          const void* gamma, const void* beta, void* h, void* y, float* mean, float* rstd,
                          rmx_stream stream) {
  if (!rows_ok(shape) || !(eps >= 0.f)) return RMX_ERR_INVALID_ARG;
  if (shape->cols > kLnMaxCols) return RMX_ERR_UNSUPPORTED;
  Drop d;
  RMX_TRY(drop_of(drop, true, d));
  if (shape->rows == 0) return RMX_OK;
  RMX_TRY(check_ptr(x));
  RMX_TRY(check_ptr(y));
  for (const void* p : {r, gamma, beta, (const void*)h, (const void*)mean, (const void*)rstd}) RMX_TRY(check_opt(p));
  if (y == x || y == r || y == h) return RMX_ERR_INVALID_ARG;
  const LnFwd a{shape->rows, shape->cols, shape->dtype, eps, d, x, r, gamma, beta, h, y, mean, rstd};
  cudaStream_t st = cuda_stream(stream);
  Launch l("layer_norm", st);
  return l.done(launch_layer_norm(a, st));
}

size_t rmx_layer_norm_backward_workspace_bytes(const rmx_rows* shape) {
  if (!rows_ok(shape) || shape->cols > kLnMaxCols) return 0;
  return 2 * up256((size_t)kLnBwdMaxBlocks * shape->cols * sizeof(float));
}

rmx_status rmx_layer_norm_backward(const rmx_rows* shape, const rmx_drop* drop, const void* dy, const void* dh,
                                   const void* h, const float* mean, const float* rstd, const void* gamma, void* dr,
                                   void* dx, void* dgamma, void* dbeta, void* ws, size_t ws_bytes,
                                   rmx_stream stream) {
  if (!rows_ok(shape)) return RMX_ERR_INVALID_ARG;
  if (shape->cols > kLnMaxCols) return RMX_ERR_UNSUPPORTED;
  Drop d;
  RMX_TRY(drop_of(drop, dx != nullptr && shape->rows > 0, d));
  for (const void* p : {dh, gamma, (const void*)dx, (const void*)dgamma, (const void*)dbeta}) RMX_TRY(check_opt(p));
  cudaStream_t st = cuda_stream(stream);
  if (shape->rows == 0) {
    const size_t n = shape->cols * storage_bytes(shape->dtype);
    if (dgamma && cudaMemsetAsync(dgamma, 0, n, st) != cudaSuccess) return RMX_ERR_CUDA;
    if (dbeta && cudaMemsetAsync(dbeta, 0, n, st) != cudaSuccess) return RMX_ERR_CUDA;
    return RMX_OK;
  }
  for (const void* p : {dy, h, (const void*)mean, (const void*)rstd, (const void*)dr, (const void*)ws}) RMX_TRY(check_ptr(p));
  if (dr == h || dx == h || dx == dr || (dx && (dx == dy || dx == dh))) return RMX_ERR_INVALID_ARG;
  if (ws_bytes < rmx_layer_norm_backward_workspace_bytes(shape)) return RMX_ERR_WORKSPACE;
  float* pg = static_cast<float*>(ws);
  float* pb = reinterpret_cast<float*>(static_cast<char*>(ws) +
                                       up256((size_t)kLnBwdMaxBlocks * shape->cols * sizeof(float)));
  const LnBwd a{shape->rows, shape->cols, shape->dtype, d, dy, dh, h, mean, rstd, gamma, dr, dx, pg, pb};
  {
    Launch l("layer_norm_backward", st);
    RMX_TRY(l.done(launch_layer_norm_bwd(a, st)));
  }
  if (!dgamma && !dbeta) return RMX_OK;
  Launch l("layer_norm_params", st);
  return l.done(launch_layer_norm_params(a, dgamma, dbeta, st));
}

// ---------------------------------------------------------------- routing

size_t rmx_expert_sort_workspace_bytes(const rmx_routes* routes) {
  if (!routes_ok(routes)) return 0;
  const long long warps = sort_warps(routes->tokens * routes->k);
  return up256((size_t)(warps + 1) * routes->experts * sizeof(int32_t));
}

rmx_status rmx_expert_sort(const rmx_routes* routes, const int32_t* expert, int32_t* offsets, int32_t* position,
                           int32_t* source, void* ws, size_t ws_bytes, rmx_stream stream) {
  if (!routes_ok(routes)) return RMX_ERR_INVALID_ARG;
  RMX_TRY(check_ptr(offsets));
  cudaStream_t st = cuda_stream(stream);
  if (routes->tokens == 0)
    return cudaMemsetAsync(offsets, 0, (routes->experts + 1) * sizeof(int32_t), st) == cudaSuccess ? RMX_OK : RMX_ERR_CUDA;
  for (const void* p : {(const void*)expert, (const void*)position, (const void*)source, (const void*)ws}) RMX_TRY(check_ptr(p));
  if (ws_bytes < rmx_expert_sort_workspace_bytes(routes)) return RMX_ERR_WORKSPACE;
  const Routes r = routes_of(routes);
  static const char* const kNames[3] = {"expert_count", "expert_scan", "expert_place"};
  const bool one = sort_warps(r.S) == 0;
  for (int pass = 0; pass < (one ? 1 : 3); ++pass) {
    Launch l(one ? "expert_sort" : kNames[pass], st);
    RMX_TRY(l.done(launch_expert_sort(r, expert, offsets, position, source, static_cast<int32_t*>(ws), pass, st)));
  }
  return RMX_OK;
}

rmx_status rmx_expert_gather(const rmx_routes* routes, const int32_t* source, const void* x, void* out, int format,
                             uint8_t* q, uint8_t* exps, rmx_stream stream) {
  if (!moved_ok(routes) || !format_ok(format)) return RMX_ERR_INVALID_ARG;
  if ((q != nullptr) != (exps != nullptr) || (!out && !q)) return RMX_ERR_INVALID_ARG;
  if (routes->tokens == 0) return RMX_OK;
  RMX_TRY(check_ptr(source));
  RMX_TRY(check_ptr(x));
  for (const void* p : {(const void*)out, (const void*)q, (const void*)exps}) RMX_TRY(check_opt(p));
  if (out == x) return RMX_ERR_INVALID_ARG;
  const Routes r = routes_of(routes);
  cudaStream_t st = cuda_stream(stream);
  Launch l(q ? "expert_gather_f8" : "expert_gather", st);
  if (!q) return l.done(launch_expert_gather(r, source, x, out, st));
  const QuantRows a{r.S, r.C, r.dtype, format, x, q, exps, source, r.k, out};
  return l.done(launch_quant_f8(a, st));
}

rmx_status rmx_expert_combine(const rmx_routes* routes, const int32_t* position, const float* weight, const void* y,
                              void* out, rmx_stream stream) {
  if (!moved_ok(routes)) return RMX_ERR_INVALID_ARG;
  if (routes->tokens == 0) return RMX_OK;
  for (const void* p : {(const void*)position, y, (const void*)out}) RMX_TRY(check_ptr(p));
  RMX_TRY(check_opt(weight));
  if (out == y) return RMX_ERR_INVALID_ARG;
  cudaStream_t st = cuda_stream(stream);
  Launch l("expert_combine", st);
  return l.done(launch_expert_combine(routes_of(routes), position, weight, y, out, st));
}

rmx_status rmx_expert_combine_backward(const rmx_routes* routes, const int32_t* position, const float* weight,
                                       const void* dout, const void* y, void* dy, float* dweight, rmx_stream stream) {
  if (!moved_ok(routes) || (!dy && !dweight)) return RMX_ERR_INVALID_ARG;
  if (routes->tokens == 0) return RMX_OK;
  RMX_TRY(check_ptr(position));
  RMX_TRY(check_ptr(dout));
  if (dweight) RMX_TRY(check_ptr(y));
  for (const void* p : {(const void*)weight, (const void*)dy, (const void*)dweight}) RMX_TRY(check_opt(p));
  if (dy == dout) return RMX_ERR_INVALID_ARG;
  cudaStream_t st = cuda_stream(stream);
  Launch l("expert_combine_backward", st);
  return l.done(launch_expert_combine_bwd(routes_of(routes), position, weight, dout, y, dy, dweight, st));
}

// ---------------------------------------------------------------- 8-bit floating rows

int rmx_f8_pitch(int cols) { return cols < 1 || cols > (1 << 24) ? 0 : f8_pitch(cols); }
int rmx_f8_exps(int cols) { return cols < 1 || cols > (1 << 24) ? 0 : f8_exps(cols); }
int rmx_f8_ragged_pitch(int rows, int groups) {
  if (rows < 0 || rows > (1 << 30) || groups < 1 || groups > kMaxExperts) return 0;
  return ragged_blocks(rows, groups) * kF8Block;
}

rmx_status rmx_quant_f8(const rmx_rows* shape, int format, const void* x, uint8_t* q, uint8_t* exps,
                        rmx_stream stream) {
  if (!rows_ok(shape) || !format_ok(format)) return RMX_ERR_INVALID_ARG;
  if (shape->rows == 0) return RMX_OK;
  RMX_TRY(check_ptr(x));
  RMX_TRY(check_ptr(q));
  RMX_TRY(check_ptr(exps));
  const QuantRows a{shape->rows, shape->cols, shape->dtype, format, x, q, exps, nullptr, 1, nullptr};
  cudaStream_t st = cuda_stream(stream);
  Launch l("quant_f8", st);
  return l.done(launch_quant_f8(a, st));
}

rmx_status rmx_dequant_f8(const rmx_rows* shape, int format, const uint8_t* q, const uint8_t* exps, void* x,
                          rmx_stream stream) {
  if (!rows_ok(shape) || !format_ok(format)) return RMX_ERR_INVALID_ARG;
  if (shape->rows == 0) return RMX_OK;
  RMX_TRY(check_ptr(q));
  RMX_TRY(check_ptr(exps));
  RMX_TRY(check_ptr(x));
  cudaStream_t st = cuda_stream(stream);
  Launch l("dequant_f8", st);
  return l.done(launch_dequant_f8(shape->rows, shape->cols, shape->dtype, format, q, exps, x, st));
}

size_t rmx_quant_f8_groups_workspace_bytes(const rmx_groups* groups) {
  if (!groups_ok(groups) || !groups_fit(*groups)) return 0;
  return up256((size_t)group_blocks(*groups) * groups->C * sizeof(float));
}

rmx_status rmx_quant_f8_groups(const rmx_groups* groups, int format, const int32_t* offsets, const void* x,
                               uint8_t* q, uint8_t* exps, uint8_t* qt, uint8_t* exps_t, void* sums, void* ws,
                               size_t ws_bytes, rmx_stream stream) {
  if (!groups_ok(groups) || !format_ok(format)) return RMX_ERR_INVALID_ARG;
  const rmx_groups& g = *groups;
  const bool ragged = g.order == RMX_ORDER_RAGGED;
  if (ragged != (offsets != nullptr)) return RMX_ERR_INVALID_ARG;
  if ((q != nullptr) != (exps != nullptr) || (qt != nullptr) != (exps_t != nullptr)) return RMX_ERR_INVALID_ARG;
  if (!q && !qt && !sums) return RMX_ERR_INVALID_ARG;
  if (!groups_fit(g)) return RMX_ERR_UNSUPPORTED;
  for (const void* p : {(const void*)offsets, (const void*)q, (const void*)exps, (const void*)qt, (const void*)exps_t,
                        (const void*)sums})
    RMX_TRY(check_opt(p));
  cudaStream_t st = cuda_stream(stream);
  if (g.M == 0) {
    if (sums && cudaMemsetAsync(sums, 0, (size_t)g.G * g.C * storage_bytes(g.dtype), st) != cudaSuccess) return RMX_ERR_CUDA;
    return RMX_OK;
  }
  RMX_TRY(check_ptr(x));
  if (sums) {
    RMX_TRY(check_ptr(ws));
    if (ws_bytes < rmx_quant_f8_groups_workspace_bytes(groups)) return RMX_ERR_WORKSPACE;
  }
  QuantGroups a{};
  a.M = g.M;
  a.G = g.G;
  a.C = g.C;
  a.dtype = g.dtype;
  a.format = format;
  a.offsets = offsets;
  a.blocks = (int)group_blocks(g);
  a.x = x;
  a.q = q;
  a.e = exps;
  a.qt = qt;
  a.et = exps_t;
  a.sums = sums;
  a.part = sums ? static_cast<float*>(ws) : nullptr;
  const bool tokens = g.order == RMX_ORDER_TOKENS;
  a.q_row = tokens ? g.G : 1;
  a.q_group = tokens ? 1 : ragged ? 0 : g.M;
  a.row_stride = a.q_row * g.C;
  a.group_stride = a.q_group * g.C;
  if (!ragged) {
    a.tp = f8_pitch(g.M);
    a.tep = f8_exps(g.M);
  }
  {
    Launch l("quant_f8_groups", st);
    RMX_TRY(l.done(launch_quant_f8_groups(a, st)));
  }
  if (!sums) return RMX_OK;
  Launch l("quant_f8_sums", st);
  return l.done(launch_quant_f8_sums(a, st));
}

// ---------------------------------------------------------------- their products

rmx_status rmx_linear_f8(const rmx_layer_f8* layer, const int32_t* offsets, const uint8_t* a, const uint8_t* a_exps,
                         const uint8_t* w, const uint8_t* w_exps, const void* bias, const void* resid, void* out,
                         rmx_stream stream) {
  if (!layer_f8_ok(layer, offsets != nullptr)) return RMX_ERR_INVALID_ARG;
  const rmx_layer_f8& l = *layer;
  RMX_TRY(check_opt(offsets));
  const LinearF8 d{l.M, l.G, l.K, l.N, l.dtype, l.a_format, l.b_format, offsets, false, a, a_exps, w, w_exps, bias, resid,
                   out};
  if (l.M == 0) return RMX_OK;
  if (!linear_f8_supported(d)) return RMX_ERR_UNSUPPORTED;
  for (const void* p : {(const void*)a, (const void*)a_exps, (const void*)w, (const void*)w_exps, (const void*)out})
    RMX_TRY(check_ptr(p));
  RMX_TRY(check_opt(bias));
  RMX_TRY(check_opt(resid));
  cudaStream_t st = cuda_stream(stream);
  Launch la("linear_f8", st);
  return la.done(launch_linear_f8(d, device_error_word(), st));
}

rmx_status rmx_wgrad_f8(const rmx_layer_f8* layer, const int32_t* offsets, const uint8_t* at, const uint8_t* at_exps,
                        const uint8_t* bt, const uint8_t* bt_exps, void* dw, rmx_stream stream) {
  if (!layer_f8_ok(layer, offsets != nullptr)) return RMX_ERR_INVALID_ARG;
  const rmx_layer_f8& l = *layer;
  RMX_TRY(check_opt(offsets));
  RMX_TRY(check_ptr(dw));
  const LinearF8 d{l.M, l.G, l.K, l.N, l.dtype, l.a_format, l.b_format, offsets, true, at, at_exps, bt, bt_exps, nullptr,
                   nullptr, dw};
  cudaStream_t st = cuda_stream(stream);
  if (l.M == 0)
    return cudaMemsetAsync(dw, 0, (size_t)l.G * l.K * l.N * storage_bytes(l.dtype), st) == cudaSuccess ? RMX_OK : RMX_ERR_CUDA;
  if (!linear_f8_supported(d)) return RMX_ERR_UNSUPPORTED;
  for (const void* p : {(const void*)at, (const void*)at_exps, (const void*)bt, (const void*)bt_exps}) RMX_TRY(check_ptr(p));
  Launch la("wgrad_f8", st);
  return la.done(launch_linear_f8(d, device_error_word(), st));
}

}  // extern "C"
