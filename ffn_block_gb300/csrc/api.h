// What the C-ABI files share: launch instrumentation, argument checks and the
// GEMM dispatch.
#pragma once

#include <cuda_runtime.h>

#include "../../include/rmx.h"
#include "kernels.h"

namespace rmx {

// Brackets one kernel launch: counts it and, when profiling is on (for its
// name), records events around it on its stream.
class Launch {
 public:
  Launch(const char* name, cudaStream_t st);
  rmx_status done(cudaError_t e);

 private:
  const char* name_;
  cudaStream_t st_;
  cudaEvent_t a_ = nullptr;
};

#define RMX_TRY(expr)                  \
  do {                                 \
    rmx_status s_ = (expr);            \
    if (s_ != RMX_OK) return s_;       \
  } while (0)

bool aligned16(const void* p);
rmx_status check_ptr(const void* p);  // non-null and 16-byte aligned
// Null is allowed; a pointer that is given must be aligned.
inline rmx_status check_opt(const void* p) { return p ? check_ptr(p) : RMX_OK; }

// ---- operators on dense rows of a storage type
inline bool storage_ok(int dtype) { return dtype == RMX_F32 || dtype == RMX_BF16 || dtype == RMX_F16; }
inline size_t storage_bytes(int dtype) { return dtype == RMX_F32 ? 4 : 2; }
// Rows and columns small enough that every byte offset fits 62 bits and every
// row index of a chunked pass 40.
inline bool rows_ok(const rmx_rows* s) {
  return s && s->rows >= 0 && s->rows <= (1ll << 36) && s->cols >= 1 && s->cols <= (1 << 24) && storage_ok(s->dtype);
}
inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// One grouped GEMM under a profile name: tensor cores where the contract and
// the shape allow, CUDA cores otherwise.
rmx_status run_gemm(const char* name, const GemmDesc& d, cudaStream_t st);

}  // namespace rmx
