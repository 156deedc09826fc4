// Bounded waits of the tensor-core kernels with 8-bit operands, and how the CTAs
// of a pair hand data over to one another.
#pragma once

#include "tcgen05.cuh"

namespace rmx {

// What a wait that runs out needs.
struct WaitCtx {
  uint64_t limit_ns;
  unsigned int* err;
  volatile int* abort;
};
// How the CTAs of a pair hand data over.  One CTA's warps arrive on a barrier
// of the other at cluster scope, relaxed.  What they wrote to or read from TMEM
// is ordered by the tcgen05 fences on both sides (TENSOR); what they wrote to
// their shared memory by a release fence before the arrival and an acquire
// fence after the wait (MEMORY), both restricted to shared memory.  An arrival
// that itself releases at cluster scope waits for all writes of its thread,
// global ones too, about 1000 cycles: with one thread of the odd CTA passing its
// warps' arrivals on in that way, 1024 x 64 tokens 1280 -> 5120 take 1212 us, in
// this way 679 (693 with waits that acquire by themselves).
enum Order { LOCAL, TENSOR, MEMORY };
// Arrival by the lanes with pred set (one of a converged warp), on a barrier of
// this CTA (LOCAL) or of the cluster.
template <Order O> __device__ __forceinline__ void arrive_if(uint32_t bar, bool pred) {
  if (O == MEMORY) asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
  if (O == LOCAL)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar), "r"((uint32_t)pred)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar), "r"((uint32_t)pred)
        : "memory");
}
__device__ __forceinline__ bool try_wait_relaxed_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// One look at a barrier of this CTA on which LOCAL threads and copies arrive, or
// the pair's other CTA and the issuer's commits too.
template <Order O> __device__ __forceinline__ bool look(uint32_t bar, uint32_t parity) {
  return O == LOCAL ? mbar_try_wait(bar, parity) : try_wait_relaxed_cluster(bar, parity);
}
// What follows a look that succeeded.
template <Order O> __device__ __forceinline__ void seen() {
  if (O == MEMORY) asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
}
// The rest of a bounded wait, out of line: it spins, now and then looking at
// the clock and at whether another warp has given up.
template <Order O>
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, unsigned int bit, uint64_t limit_ns,
                                     unsigned int* err, volatile int* abort) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    for (int i = 0; i < 1024; ++i)
      if (look<O>(bar, parity)) {
        seen<O>();
        return true;
      }
    if (*abort) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      atomicOr(err, bit);
      *abort = 1;
      return false;
    }
  }
}
template <Order O>
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t ph, unsigned int bit, const WaitCtx& w) {
#pragma unroll 1
  for (int i = 0; i < 512; ++i)
    if (look<O>(bar, ph)) {
      seen<O>();
      return true;
    }
  return wait_on<O>(bar, ph, bit, w.limit_ns, w.err, w.abort);
}
// The same by a whole warp, which goes on or gives up together.
template <Order O>
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t ph, unsigned int bit, const WaitCtx& w) {
#pragma unroll 1
  for (int i = 0; i < 512; ++i)
    if (__all_sync(0xffffffffu, look<O>(bar, ph))) {
      seen<O>();
      return true;
    }
  return __all_sync(0xffffffffu, wait_on<O>(bar, ph, bit, w.limit_ns, w.err, w.abort));
}

}  // namespace rmx
