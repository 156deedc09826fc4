// Product of int8 rows with scales per token and channel:
//   out[m,g,n] = (sum_k a[m,g,k] * w[g,n,k]) * sa[m,g] * sw[g,n] + bias[g,n] + resid[m,g,n]
//
// The integers run on the 16-bit floating tensor cores: an int8 is exact in
// fp16, a product of two is exact in the fp32 accumulator and so is every sum
// below 2^24.  (sm_103a has no fast integer tensor path.)  The operands stay
// 8 bits wide up to the SM: TMA brings int8 tiles into shared memory, and two
// groups of warps turn them into fp16 there, the weights into tensor memory
// (the MMA's A operand) and the tokens into swizzled shared memory (its B
// operand).  An output tile is channels x tokens, so that few tokens are a
// narrow tile, not a padded one: 128 channels a CTA (256 a CTA pair) by up to
// 208 tokens.  The bound is the tensor rate from about 150 tokens on, the
// stream of the weights below.
//
// Roles (30 warps, one CTA per SM, persistent over tiles):
//   warp 0       TMA producer: 128 k of the CTA's channels and tokens a stage
//   warp 1       TMEM allocation; one thread issues the MMAs (even CTA)
//   warps 2-25   three sets, taking 64 k in turn, of four warps for the
//                weights (one channel a thread, int8 -> TMEM) and four for
//                the tokens (one token a thread, int8 -> smem)
//   warps 26-29  epilogue: a channel a thread, 16 tokens at a time
// TMEM: two accumulators of NT <= 208 columns (so that the epilogue of one
// tile overlaps the next), then the weights' stages of 32 columns.
//
// Conversion of four int8 at once: (w & 0x00ff00ff) ^ 0x64806480 is the pair
// of fp16 1024 + 128 + q for bytes 0 and 2, the same of w >> 8 for bytes 1 and
// 3, and subtracting 1152 is exact: five instructions for four values.  The
// order of k within a word changes in both operands alike, which leaves the
// sum over k what it is.

#include <cuda.h>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "q8.h"
#include "tcgen05.cuh"

namespace rmx {
namespace {

constexpr int kWWarps = 4, kTWarps = 4, kSets = 3, kEpiWarps = 4;
constexpr int kFirstConv = 2, kFirstEpi = kFirstConv + kSets * (kWWarps + kTWarps);
constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
constexpr int kRawK = 128, kConvK = 64;
constexpr int kMaxRaw = 8, kMaxConv = 6;
constexpr int kMaxNT = 208;
constexpr int kTmemCols = 512;
constexpr int kBarBytes = 512;
constexpr int kSmemMax = 227 * 1024;
constexpr uint64_t kDrainNs = 50ull * 1000ull * 1000ull;

struct Params {
  int M, G, K, N;
  int nt, ntc;            // tokens of a tile, and the share of them a CTA converts
  int raw_stages, conv_stages, raw_bytes, conv_bytes;
  int num_kb, num_raw;    // 64- and 128-column steps of K
  int tiles_m, tiles_n, num_tiles;
  uint32_t idesc;
  const float *sa, *sw;
  const void *bias, *resid;
  void* out;
  unsigned int* err;
  unsigned long long wait_ns;
};

__device__ __forceinline__ uint32_t sub1152(uint32_t u) {
  const __half2 c = __half2half2(__ushort_as_half(0x6480));  // 1152
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&u), c);
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Four int8 as two fp16 pairs, bytes (0, 2) and (1, 3).
__device__ __forceinline__ void widen(uint32_t w, uint32_t& a, uint32_t& b) {
  a = sub1152((w & 0x00ff00ffu) ^ 0x64806480u);
  b = sub1152(((w >> 8) & 0x00ff00ffu) ^ 0x64806480u);
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Waits for a phase in a loop of a few instructions, at most `kTries` tests.
constexpr uint32_t kTries = 1u << 14;
__device__ __forceinline__ bool mbar_spin(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, %3;\n\t"
      "SPIN:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.ne.u32 q, n, 0;\n\t"
      "@q bra SPIN;\n\t"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "n"(kTries)
      : "memory");
  return ok != 0;
}
// The rest of a bounded wait: now and then a look at the clock and at whether
// another warp has given up.  Out of line: it is all but never reached.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, uint64_t limit_ns, unsigned int* err,
                                     unsigned int bit, volatile int* abort) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_spin(bar, parity)) {
    if (*abort) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      atomicOr(err, bit);
      *abort = 1;
      return false;
    }
  }
  return true;
}
// Arrival by the lanes with pred set (one of a converged warp).
__device__ __forceinline__ void arrive_if(uint32_t bar, bool pred) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar), "r"((uint32_t)pred)
      : "memory");
}

template <typename T, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear_q8(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA, const Params p) {
  pdl_trigger();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const uint32_t sRaw = smem_u32(smem);
  const uint32_t sConv = sRaw + p.raw_stages * p.raw_bytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.raw_stages * p.raw_bytes + p.conv_stages * p.conv_bytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxRaw + 2 * kMaxConv + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t bar0 = smem_u32(bars);
  auto raw_full = [&](int s) { return bar0 + 8u * (uint32_t)s; };
  auto raw_empty = [&](int s) { return bar0 + 8u * (uint32_t)(kMaxRaw + s); };
  auto conv_full = [&](int s) { return bar0 + 8u * (uint32_t)(2 * kMaxRaw + s); };
  auto conv_empty = [&](int s) { return bar0 + 8u * (uint32_t)(2 * kMaxRaw + kMaxConv + s); };
  auto d_full = [&](int a) { return bar0 + 8u * (uint32_t)(2 * kMaxRaw + 2 * kMaxConv + a); };
  auto d_empty = [&](int a) { return bar0 + 8u * (uint32_t)(2 * kMaxRaw + 2 * kMaxConv + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (uint32_t)(2 * kMaxRaw + 2 * kMaxConv + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? (int)cluster_rank() : 0;
  const int first = PAIR ? (int)cluster_id_x() : (int)blockIdx.x;
  const int stride = PAIR ? (int)num_clusters_x() : (int)gridDim.x;
  constexpr int CTAS = PAIR ? 2 : 1;
  const int twarps = (p.ntc + 31) / 32;  // of each set, the warps that have tokens
  // Tile -> group, this CTA's first channel, the tile's first token.  Tiles
  // that share weights are neighbours.
  auto coords = [&](int tile, int& g, int& n0, int& m0) {
    const int tm = tile % p.tiles_m, r = tile / p.tiles_m;
    const int tn = r % p.tiles_n;
    g = r / p.tiles_n;
    n0 = tn * 128 * CTAS + rank * 128;
    m0 = tm * p.nt;
  };
  auto wait = [&](uint32_t bar, uint32_t ph, unsigned int bit) {
    return mbar_spin(bar, ph) || wait_on(bar, ph, p.wait_ns, p.err, bit, abort_flag);
  };
  // The same by a whole warp, which goes on or gives up together.
  auto wait_warp = [&](uint32_t bar, uint32_t ph, unsigned int bit) { return __all_sync(0xffffffffu, wait(bar, ph, bit)); };
  // Tiles of this CTA (or pair).
  const int my_tiles = first < p.num_tiles ? (p.num_tiles - first + stride - 1) / stride : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.raw_stages; ++s) {
      mbar_init(raw_full(s), 1);
      mbar_init(raw_empty(s), 2 * (kWWarps + twarps));  // the sets of its two halves
    }
    for (int s = 0; s < p.conv_stages; ++s) {
      mbar_init(conv_full(s), (kWWarps + twarps) * CTAS);
      mbar_init(conv_empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(d_full(a), 1);
      mbar_init(d_empty(a), kEpiWarps * CTAS);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_map(&tmW);
    prefetch_map(&tmA);
  }
  if (warp == 1) tmem_alloc<PAIR>(smem_u32(tmem_slot), kTmemCols);
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_barrier();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tmemA = tmem + 2 * p.nt;
  pdl_wait();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (elect_one()) {
      int s = 0, issued = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = first; ok && tile < p.num_tiles; tile += stride) {
        int g, n0, m0;
        coords(tile, g, n0, m0);
        for (int rk = 0; rk < p.num_raw; ++rk) {
          if (!wait(raw_empty(s), ph ^ 1u, ERRBIT_WAIT_PRODUCER)) {
            ok = false;
            break;
          }
          mbar_expect_tx(raw_full(s), (uint32_t)p.raw_bytes);
          const uint32_t dst = sRaw + s * p.raw_bytes;
          tma_load_3d(dst, &tmW, raw_full(s), rk * kRawK, n0, g);                             // {K, N, G}
          tma_load_3d(dst + 128 * kRawK, &tmA, raw_full(s), rk * kRawK, g, m0 + rank * p.ntc);  // {K, G, M}
          issued = min(issued + 1, p.raw_stages);
          if (++s == p.raw_stages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (!ok) {
        // Let the copies already issued land before the CTA can exit.
        while (issued-- > 0) {
          if (--s < 0) {
            s = p.raw_stages - 1;
            ph ^= 1;
          }
          volatile int no_abort = 0;
          mbar_wait_bounded(raw_full(s), ph, kDrainNs, p.err, ERRBIT_WAIT_DRAIN, &no_abort);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0 && elect_one()) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      const uint64_t desc0 = sw128_desc(sConv, 16, 1024);
      const uint32_t conv_step = (uint32_t)p.conv_bytes >> 4;  // descriptor addresses count 16 bytes
      for (int lt = 0; ok && lt < my_tiles; ++lt) {
        const int acc = lt & 1;
        if (!wait(d_empty(acc), ((uint32_t)(lt >> 1) & 1u) ^ 1u, ERRBIT_WAIT_MMA)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(acc * p.nt);
        uint32_t accumulate = 0;
#pragma unroll 1
        for (int kb = 0; kb < p.num_kb; ++kb) {
          if (!wait(conv_full(s), ph, ERRBIT_WAIT_MMA)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t b = desc0 + (uint32_t)s * conv_step;
          const uint32_t a = tmemA + s * (kConvK / 2);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            umma_f16_ts<PAIR>(d, a + k * 8, b + 2 * k, p.idesc, accumulate);
            accumulate = 1;
          }
          if (PAIR) umma_commit_pair(conv_empty(s));
          else umma_commit<false>(conv_empty(s));
          const bool wrap = s + 1 == p.conv_stages;
          s = wrap ? 0 : s + 1;
          ph ^= wrap ? 1u : 0u;
        }
        if (!ok) break;
        if (PAIR) umma_commit_pair(d_full(acc));
        else umma_commit<false>(d_full(acc));
      }
      if (!ok) {
        // No MMA may still be writing TMEM when it is freed.
        umma_commit<PAIR>(drain_bar);
        volatile int no_abort = 0;
        mbar_wait_bounded(drain_bar, 0, kDrainNs, p.err, ERRBIT_WAIT_DRAIN, &no_abort);
      }
    }
    __syncwarp();
  } else if (warp < kFirstEpi) {
    // ------------------------------------------------------------ converters
    // Three sets of eight warps take the 64-column halves of the raw stages in
    // turn: a half's chain of waits, loads, conversion and stores is longer
    // than its MMAs, so three are kept in flight.
    const int cw = warp - kFirstConv, set = cw >> 3;
    const bool weights = (cw & 7) < kWWarps;
    // Weights: the channel is the TMEM lane, and a warp reaches the quarter
    // warp % 4.  Tokens: rows in warp order; warps without tokens stay out.
    const int row = (weights ? (warp & 3) : (cw & 7) - kWWarps) * 32 + lane;
    const bool live = weights || row < p.ntc, one = lane == 0;
    // 16-byte chunk j of a 128-byte row sits at j ^ (row & 7): rows are 128
    // bytes aligned, so its address is (row's | swizzle) ^ (j << 4).  A lane
    // without a token reads its place in the first row and writes nothing.
    const uint32_t swz = (uint32_t)(row & 7) << 4;
    const uint32_t src0 = (sRaw + (weights ? 0 : 128 * kRawK) + (live ? (uint32_t)row * 128u : 0u)) | swz;
    const uint32_t full0 = PAIR ? mapa_shared(conv_full(0), 0) : conv_full(0);
    // Half `it` of this CTA's run is half it % 2 of raw stage it / 2, and goes
    // to conv stage it % conv_stages.
    int rs = set >> 1, s = set;
    uint32_t half = (uint32_t)(set & 1) << 6;           // bit 6 of the address: the upper 64 columns
    uint32_t src = src0 + rs * p.raw_bytes, rph = 0, ph = 1;  // parities of the next raw_full / conv_empty wait
    // 64 k of this lane's row widened to fp16 pairs; the raw stage is handed
    // back once it has been read.
    auto load = [&](uint32_t* o) {
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const uint4 v = ld_shared_v4((src ^ half) ^ (uint32_t)(j << 4));
        const uint4 w = ld_shared_v4((src ^ half) ^ (uint32_t)((j + 1) << 4));
        if (j == 2) {
          __syncwarp();
          arrive_if(raw_empty(rs), one);
        }
        uint32_t* q = o + 8 * j;
        widen(v.x, q[0], q[1]);
        widen(v.y, q[2], q[3]);
        widen(v.z, q[4], q[5]);
        widen(v.w, q[6], q[7]);
        widen(w.x, q[8], q[9]);
        widen(w.y, q[10], q[11]);
        widen(w.z, q[12], q[13]);
        widen(w.w, q[14], q[15]);
      }
      // Three halves on: one raw stage and a half.
      const int adv = half ? 2 : 1;
      const bool wrap = rs + adv >= p.raw_stages;
      rs += wrap ? adv - p.raw_stages : adv;
      src = src0 + rs * p.raw_bytes;
      rph ^= wrap ? 1u : 0u;
      half ^= 64u;
    };
    auto next = [&]() {
      __syncwarp();
      arrive_if(full0 + 8u * (uint32_t)s, one);
      const bool wrap = s + kSets >= p.conv_stages;
      s += wrap ? kSets - p.conv_stages : kSets;
      ph ^= wrap ? 1u : 0u;
    };
    const long long halves = (long long)my_tiles * p.num_kb;
    if (weights) {
      const uint32_t a0 = tmemA + ((uint32_t)((warp & 3) * 32) << 16);
#pragma unroll 1
      for (long long i = set; i < halves; i += kSets) {
        uint32_t o[32];
        if (!wait_warp(raw_full(rs), rph, ERRBIT_WAIT_ROWS)) break;
        load(o);
        if (!wait_warp(conv_empty(s), ph, ERRBIT_WAIT_ROWS)) break;
        tc_fence_after();
        tmem_st_32x32(a0 + s * (kConvK / 2), o);
        tmem_st_wait();
        tc_fence_before();
        next();
      }
    } else if (row - lane < p.ntc) {
      const uint32_t dst0 = (sConv + (uint32_t)row * 128u) | swz;
#pragma unroll 1
      for (long long i = set; i < halves; i += kSets) {
        uint32_t o[32];
        if (!wait_warp(raw_full(rs), rph, ERRBIT_WAIT_ROWS)) break;
        load(o);
        if (!wait_warp(conv_empty(s), ph, ERRBIT_WAIT_ROWS)) break;
        if (live) {
          const uint32_t dst = dst0 + s * p.conv_bytes;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            st_shared_v4(dst ^ (uint32_t)(j << 4), o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        }
        fence_proxy_async_smem();
        next();
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    int lt = 0;
    bool ok = true;
    for (int tile = first; tile < p.num_tiles; tile += stride, ++lt) {
      int g, n0, m0;
      coords(tile, g, n0, m0);
      const int acc = lt & 1;
      const int n = n0 + q * 32 + lane;
      const bool in = n < p.N;
      const int live_cols = min(p.nt, p.M - m0);
      // While the accumulator is being computed: the scales, one token a lane.
      const float sw = in ? p.sw[(size_t)g * p.N + n] : 0.f;
      const float bias = p.bias && in ? to_f(static_cast<const T*>(p.bias)[(size_t)g * p.N + n]) : 0.f;
      // Token scales 16 columns ahead, one a lane.
      auto token_scale = [&](int c0) {
        const int c = c0 + (lane & 15);
        return c < live_cols ? p.sa[(size_t)(m0 + c) * p.G + g] : 0.f;
      };
      // The residual's addition, the rounding and the store of up to 16 tokens
      // of this lane's channel (inlined twice: `cols` is 16 for all but the
      // last tokens).  out may be resid: a value is read before it is written
      // by the same thread.
      auto finish = [&](float* v, T* out, size_t step, int cols) {
        if (p.resid) {
          const T* r = static_cast<const T*>(p.resid) + (out - static_cast<T*>(p.out));
          T rv[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) rv[c] = c < cols ? r[c * step] : from_f<T>(0.f);
#pragma unroll
          for (int c = 0; c < 16; ++c) v[c] += to_f(rv[c]);
        }
#pragma unroll
        for (int c = 0; c < 16; ++c)
          if (c < cols) out[c * step] = from_f<T>(v[c]);
      };
      float next = token_scale(0);
      if (!wait_warp(d_full(acc), (uint32_t)(lt >> 1) & 1u, ERRBIT_WAIT_EPILOGUE)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const size_t step = (size_t)p.G * p.N;
      size_t o = ((size_t)m0 * p.G + g) * p.N + n;
      const uint32_t d = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * p.nt);
#pragma unroll 1
      for (int c0 = 0; c0 < live_cols; c0 += 16, o += 16 * step) {
        const float sa = next;
        next = token_scale(c0 + 16);
        float v[16];
        tmem_ld_32x16(d + c0, v);
#pragma unroll
        for (int c = 0; c < 16; ++c) v[c] = fmaf(v[c] * __shfl_sync(0xffffffffu, sa, c), sw, bias);
        T* out = static_cast<T*>(p.out) + o;
        if (live_cols - c0 >= 16) {
          if (in) finish(v, out, step, 16);
        } else {
          if (in) finish(v, out, step, live_cols - c0);
        }
      }
      tc_fence_before();
      __syncwarp();
      arrive_if(PAIR ? mapa_shared(d_empty(acc), 0) : d_empty(acc), lane == 0);
    }
    // No commit may still be on its way to this CTA's barriers at the end:
    // wait for the last use of every stage.
    if (ok && warp == kFirstEpi) {
      const long long its = (long long)lt * p.num_kb;
      for (long long j = its > p.conv_stages ? its - p.conv_stages : 0; ok && j < its; ++j)
        ok = wait_warp(conv_empty((int)(j % p.conv_stages)), (uint32_t)(j / p.conv_stages) & 1u, ERRBIT_WAIT_DRAIN);
    }
  }

  tc_fence_before();
  __syncthreads();
  // Neither CTA of a pair leaves while the other may still read its shared
  // memory or signal its barriers; TMEM is freed by both together.
  if (PAIR) cluster_barrier();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<PAIR>(tmem, kTmemCols);
  }
}

template <typename T, bool PAIR>
cudaError_t launch(const CUtensorMap& w, const CUtensorMap& a, const Params& p, cudaStream_t st) {
  auto k = k_linear_q8<T, PAIR>;
  const int smem = 1024 + p.raw_stages * p.raw_bytes + p.conv_stages * p.conv_bytes + kBarBytes;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
  if (e != cudaSuccess) return e;
  const int slots = PAIR ? sm_count() / 2 : sm_count();
  const int n = p.num_tiles < slots ? p.num_tiles : slots;
  return launch_k(k, dim3(PAIR ? 2 * n : n), dim3(kThreads), smem, st, PAIR ? 2 : 1, w, a, p);
}

}  // namespace

cudaError_t launch_linear_q8(const LinearQ8& d, unsigned int* err, cudaStream_t st) {
  Params p;
  p.M = d.M;
  p.G = d.G;
  p.K = d.K;
  p.N = d.N;
  // A CTA alone up to 128 tokens, a pair above: the pair shares the tokens'
  // conversion, which a CTA alone would do for all of them.
  const bool pair = d.M > 128 && d.N > 128;
  const int most = pair ? kMaxNT : 128;
  p.tiles_m = (d.M + most - 1) / most;
  const int even = (d.M + p.tiles_m - 1) / p.tiles_m;
  p.nt = (even + 15) / 16 * 16;
  p.ntc = pair ? p.nt / 2 : p.nt;
  p.tiles_m = (d.M + p.nt - 1) / p.nt;
  const int tn = pair ? 256 : 128;
  p.tiles_n = (d.N + tn - 1) / tn;
  const long long tiles = (long long)d.G * p.tiles_n * p.tiles_m;
  if (tiles > (1ll << 30)) return cudaErrorInvalidValue;
  p.num_tiles = (int)tiles;
  p.num_raw = (d.K + kRawK - 1) / kRawK;
  p.num_kb = p.num_raw * (kRawK / kConvK);  // columns past K are zeros
  p.conv_stages = (kTmemCols - 2 * p.nt) / (kConvK / 2);
  if (p.conv_stages > kMaxConv) p.conv_stages = kMaxConv;
  p.raw_bytes = 128 * kRawK + p.ntc * kRawK;
  p.conv_bytes = p.ntc * kConvK * 2;
  p.raw_stages = (kSmemMax - 1024 - kBarBytes - p.conv_stages * p.conv_bytes) / p.raw_bytes;
  if (p.raw_stages > kMaxRaw) p.raw_stages = kMaxRaw;
  // kind::f16, fp16 operands (type 0), fp32 accumulator, both K-major.
  p.idesc = (1u << 4) | ((uint32_t)(p.nt >> 3) << 17) | ((uint32_t)((pair ? 256 : 128) >> 4) << 24);
  p.sa = d.sa;
  p.sw = d.sw;
  p.bias = d.bias;
  p.resid = d.resid;
  p.out = d.out;
  p.err = err;
  p.wait_ns = kWaitLimitNs;
  CUtensorMap w, a;
  const uint64_t P = d.P, K = d.K, N = d.N, G = d.G, M = d.M;
  if (!make_tensor_map_rows8(&w, d.w, K, N, G, P, N * P, 128, 1) ||
      !make_tensor_map_rows8(&a, d.a, K, G, M, P, G * P, 1, (uint32_t)p.ntc))
    return cudaErrorInvalidValue;
#define RMX_LQ8(T) return pair ? launch<T, true>(w, a, p, st) : launch<T, false>(w, a, p, st)
  switch (d.dtype) {
    case 0: RMX_LQ8(float);
    case 1: RMX_LQ8(bf16);
    case 2: RMX_LQ8(f16);
    default: return cudaErrorInvalidValue;
  }
#undef RMX_LQ8
}

}  // namespace rmx
