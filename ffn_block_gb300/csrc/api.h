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

// One grouped GEMM under a profile name: tensor cores where the contract and
// the shape allow, CUDA cores otherwise.
rmx_status run_gemm(const char* name, const GemmDesc& d, cudaStream_t st);

}  // namespace rmx
