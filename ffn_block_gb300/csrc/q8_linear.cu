// Product of int8 rows with scales per token and channel:
//   out[m,g,n] = (sum_k a[m,g,k] * w[g,n,k]) * sa[m,g] * sw[g,n] + bias[g,n] + resid[m,g,n]
//
// The integers run on the 16-bit floating tensor cores: an int8 is exact in
// fp16, a product of two is exact in the fp32 accumulator and so is the sum
// while no partial sum passes 2^24.  (sm_103a has no fast integer tensor path.)
// The operands stay 8 bits wide up to the SM: TMA brings int8 tiles into shared
// memory, and two groups of warps turn them into fp16 there, the weights into
// tensor memory (the MMA's A operand) and the tokens into swizzled shared
// memory (its B operand).  An output tile is channels x tokens, so that few
// tokens are a narrow tile, not a padded one: 128 channels a CTA (256 a CTA
// pair) by up to 192 tokens.  The bound is the tensor rate from about 150
// tokens on, the stream of the weights below.
//
// Roles (31 warps, one CTA per SM, persistent over tiles):
//   warp 0       TMA producer: 128 k of the CTA's channels and tokens a stage
//   warp 1       TMEM allocation; one thread issues the MMAs (even CTA)
//   warps 2-22   three sets, taking 64 k in turn, of four warps for the
//                weights (one channel a thread, int8 -> TMEM) and three for
//                the tokens (one token a thread, int8 -> smem)
//   warps 23-30  epilogue: a channel a thread, 16 tokens at a time
// Few tiles with many steps of k: a cluster of two or four CTAs shares a tile's
// steps and adds the sums up through distributed shared memory (split_of).
// TMEM: two accumulators of NT <= 192 columns (so that the epilogue of one
// tile overlaps the next), then the weights' stages of 32 columns.
//
// Conversion of four int8 at once: (w & 0x00ff00ff) ^ 0x64806480 is the pair
// of fp16 1024 + 128 + q for bytes 0 and 2, the same of w >> 8 for bytes 1 and
// 3, and 2 * (u - 1152) is exact: five instructions for four values.  The
// order of k within a word changes in both operands alike, which leaves the
// sum over k what it is.
//
// Measured (GB300; us for one call among others): 1024 samples x 64 tokens
// through 1280 -> 5120 664 us (1290 TFLOP/s, 67% of the measured cuBLAS bf16
// rate; 620 in short runs, 700 where the board is held at its power limit),
// 1000 x 40 through 3600 -> 1200 279 us, one sample x 64 tokens through 1280 ->
// 5120 73 us (5.8 TB/s, 87% of the measured copy rate).  The library's 16-bit
// products of these sizes take 467, 231 and 118 us: this one is for few tokens
// and for weights and activations that are 8 bits wide already.  What bounds the
// large products is the SM's instruction issue: a step of 64 k of a 256 x 176
// tile takes the tensor cores 352 cycles, and about 1440 instructions (560 of
// them the conversion itself, 260 the epilogue) at an IPC of 2.6, and the fences
// and waits of the hand-over between a pair's CTAs.  With an epilogue of 4 warps
// or tiles of 208 tokens the epilogue bounds it instead; outputs through shared
// memory and TMA cost more instructions than they save.

#include <cuda.h>

#include "common.cuh"
#include "handover.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "q8.h"
#include "tcgen05.cuh"

namespace rmx {
namespace {

constexpr int kWWarps = 4, kTWarps = 3, kSets = 3, kEpiWarps = 8;
constexpr int kSetWarps = kWWarps + kTWarps;
constexpr int kFirstConv = 2, kFirstEpi = kFirstConv + kSets * kSetWarps;
constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
constexpr int kRawK = 128, kConvK = 64;
constexpr int kMaxRaw = 8, kConv = 2 * kSets;
constexpr int kMaxNT = 192, kMaxAlone = 32 * kTWarps;
constexpr int kMaxSplit = 4;
constexpr int kTmemCols = 512, kAcols = kConvK / 2;
constexpr int kScaleBytes = kEpiWarps * 1024;  // each epilogue warp's copy of a tile's token scales
constexpr int kBarBytes = 512;
constexpr int kSmemMax = 227 * 1024;
constexpr uint64_t kDrainNs = 50ull * 1000ull * 1000ull;

struct Params {
  int M, G, K, N;
  int nt, ntc;            // tokens of a tile, and the share of them a CTA converts
  int raw_bytes, conv_bytes, raw_stages;
  int num_raw;            // 128-column steps of K
  int split;              // CTAs that share a tile's steps (SPLIT)
  int tiles_m, tiles_n, num_tiles;
  uint32_t idesc;
  const float *sa, *sw;
  const void *bias, *resid;
  void* out;
  unsigned int* err;
  unsigned long long wait_ns;
};

// 2 * (u - 1152) of a pair of fp16, exact.  The factor of two keeps this a
// fused multiply-add, which runs on another pipe than the bit operations (a
// plain addition shares theirs); each operand carries it, and the channel
// scale takes the four away again.
__device__ __forceinline__ uint32_t centre(uint32_t u) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(u), "r"(0x40004000u), "r"(0xe880e880u));  // 2, -2304
  return r;
}
// Four int8 as two fp16 pairs, bytes (0, 2) and (1, 3).
__device__ __forceinline__ void widen(uint32_t w, uint32_t& a, uint32_t& b) {
  // lop3 0x6a is (x & y) ^ z in one instruction, which the compiler does not
  // form by itself from two constants.
  uint32_t x, y;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(x) : "r"(w), "r"(0x00ff00ffu), "r"(0x64806480u));
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(y) : "r"(w >> 8), "r"(0x00ff00ffu), "r"(0x64806480u));
  a = centre(x);
  b = centre(y);
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t cluster_addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// A converter warp's run.  Half `it` (64 k) of the CTA's run is half it % 2 of
// raw stage it / 2.  Set x takes halves x, x + 3, x + 6, ...: conv stages x
// and x + 3 of the six in turn.  Tokens go to conv stage it % 6 once the MMAs
// of half it - 6 are done, weights to TMEM stage it % W once those of half
// it - W are (W is 3 where the accumulators leave room for no more); the
// barriers are those of the conv stages either way.
template <bool PAIR, int W, bool WEIGHTS>
__device__ __forceinline__ void convert(int set, int row, bool live, int halves, uint32_t src0, uint32_t raw_bytes,
                                        int raw_stages, uint32_t raw_bar, uint32_t conv_full, uint32_t conv_empty,
                                        uint32_t dst0, uint32_t conv_bytes, const WaitCtx& wc) {
  constexpr Order ORDER = !PAIR ? LOCAL : WEIGHTS ? TENSOR : MEMORY;  // tokens are handed over in shared memory
  const bool one = (threadIdx.x & 31) == 0;
  // 16-byte chunk j of a 128-byte row sits at j ^ (row & 7): rows are 128
  // bytes aligned, so its address is (row's | swizzle) ^ (j << 4).
  const uint32_t swz = (uint32_t)(row & 7) << 4;
  uint32_t dst[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
    dst[j] = WEIGHTS ? dst0 + (uint32_t)(W == 3 ? set : set + kSets * j) * kAcols
                     : (dst0 + (uint32_t)(set + kSets * j) * conv_bytes) | swz;
  const uint32_t cfull = conv_full + 8u * (uint32_t)set, cempty = conv_empty + 8u * (uint32_t)set;
  int rs = set >> 1;
  uint32_t src = ((src0 + (uint32_t)rs * raw_bytes) | swz) ^ ((uint32_t)(set & 1) << 6);  // bit 6: the upper half
  uint32_t rph = 0, lap = 0;  // parities of the raw stages' and the conv stages' laps
  // A raw stage that has been read.  The copy that fills it again is of the
  // async proxy: only a proxy fence orders the warp's reads before its writes.
  // (Without it a read that had been issued, but waited behind the epilogue's
  // stores, returned the next contents.)  CTAs alone give it back as soon as the
  // reads are issued (one sample 1280 -> 5120 73.0 us, after the conversion
  // 74.3); a pair's weights after the conversion and its tokens after their
  // stores, with the fence that these need anyway, since there the fences cost
  // more than the stage (1024 x 64 1280 -> 5120 678 us, both after the
  // conversion 686; 1024 x 16 156 us, at once 161).
  auto hand_back = [&](uint32_t bar) {
    fence_proxy_async_smem();
    __syncwarp();
    arrive_if<LOCAL>(bar, one);
  };
#pragma unroll 1
  for (int i = set; i < halves; i += 2 * kSets) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (j && i + kSets >= halves) return;
      const uint32_t rbar = raw_bar + 8u * (uint32_t)rs;
      if (!wait_warp<LOCAL>(rbar, rph, ERRBIT_WAIT_ROWS, wc)) return;
      uint32_t o[32];
#pragma unroll
      for (int c = 0; c < 4; c += 2) {
        const uint4 v = ld_shared_v4(src ^ (uint32_t)(c << 4));
        const uint4 w = ld_shared_v4(src ^ (uint32_t)((c + 1) << 4));
        if (c == 2 && !PAIR) hand_back(rbar + 8u * kMaxRaw);
        uint32_t* q = o + 8 * c;
        widen(v.x, q[0], q[1]);
        widen(v.y, q[2], q[3]);
        widen(v.z, q[4], q[5]);
        widen(v.w, q[6], q[7]);
        widen(w.x, q[8], q[9]);
        widen(w.y, q[10], q[11]);
        widen(w.z, q[12], q[13]);
        widen(w.w, q[14], q[15]);
      }
      if (PAIR && WEIGHTS) hand_back(rbar + 8u * kMaxRaw);
      // The half whose MMAs free this place: six back (this conv stage, the
      // lap before), or three (the other one of this set).
      constexpr bool kThree = WEIGHTS && W == 3;
      const uint32_t e = cempty + (((j & 1) != 0) != kThree ? 8u * kSets : 0u);
      const uint32_t eph = kThree && (j & 1) ? lap : lap ^ 1u;
      if (!wait_warp<ORDER>(e, eph, ERRBIT_WAIT_ROWS, wc)) return;
      if (WEIGHTS) {
        tc_fence_after();
        tmem_st_32x32(dst[j], o);
        tmem_st_wait();
        tc_fence_before();
      } else {
        if (live) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            st_shared_v4(dst[j] ^ (uint32_t)(c << 4), o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      arrive_if<ORDER>(cfull + (j ? 8u * kSets : 0u), one);
      if (PAIR && !WEIGHTS) arrive_if<LOCAL>(rbar + 8u * kMaxRaw, one);
      if (j) lap ^= 1u;
      // Three halves on: one raw stage and a half.
      const int adv = ((set + j) & 1) ? 2 : 1;
      const bool wrap = rs + adv >= raw_stages;
      rs += wrap ? adv - raw_stages : adv;
      src = (src ^ 64u) + (uint32_t)(wrap ? adv - raw_stages : adv) * raw_bytes;
      rph ^= wrap ? 1u : 0u;
    }
  }
}

// SPLIT: the CTAs of a cluster each take a share of one tile's steps of K and
// leave their sums in shared memory; then each adds up every p.split-th token's,
// in the order of the shares, and stores them.  A cluster has one tile.
template <typename T, bool PAIR, int W, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear_q8(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA, const Params p) {
  pdl_trigger();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const uint32_t sRaw = smem_u32(smem);
  const uint32_t sConv = sRaw + p.raw_stages * p.raw_bytes, sScale = sConv + kConv * p.conv_bytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.raw_stages * p.raw_bytes + kConv * p.conv_bytes + kScaleBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxRaw + 2 * kConv + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t bar0 = smem_u32(bars);
  auto raw_full = [&](int s) { return bar0 + 8u * (uint32_t)s; };
  auto raw_empty = [&](int s) { return bar0 + 8u * (uint32_t)(kMaxRaw + s); };
  auto conv_full = [&](int s) { return bar0 + 8u * (uint32_t)(2 * kMaxRaw + s); };
  auto conv_empty = [&](int s) { return bar0 + 8u * (uint32_t)(2 * kMaxRaw + kConv + s); };
  auto d_full = [&](int a) { return bar0 + 8u * (uint32_t)(2 * kMaxRaw + 2 * kConv + a); };
  auto d_empty = [&](int a) { return bar0 + 8u * (uint32_t)(2 * kMaxRaw + 2 * kConv + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (uint32_t)(2 * kMaxRaw + 2 * kConv + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? (int)cluster_rank() : 0;
  const int first = PAIR || SPLIT ? (int)cluster_id_x() : (int)blockIdx.x;
  const int stride = PAIR || SPLIT ? (int)num_clusters_x() : (int)gridDim.x;
  const int share = SPLIT ? (int)cluster_rank() : 0;
  const int raw0 = SPLIT ? p.num_raw * share / p.split : 0;
  const int num_raw = SPLIT ? p.num_raw * (share + 1) / p.split - raw0 : p.num_raw;
  constexpr int CTAS = PAIR ? 2 : 1;
  constexpr Order CROSS = PAIR ? TENSOR : LOCAL;
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
  const WaitCtx wc{p.wait_ns, p.err, abort_flag};
  float sum_sw = 0.f, sum_bias = 0.f;  // SPLIT: this lane's channel's, for the last pass
  // Tiles of this CTA (or pair).
  const int my_tiles = first < p.num_tiles ? (p.num_tiles - first + stride - 1) / stride : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.raw_stages; ++s) {
      mbar_init(raw_full(s), 1);
      mbar_init(raw_empty(s), 2 * (kWWarps + twarps));  // the sets of its two halves
    }
    for (int s = 0; s < kConv; ++s) {
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
        for (int rk = raw0; rk < raw0 + num_raw; ++rk) {
          if (!wait_one<LOCAL>(raw_empty(s), ph ^ 1u, ERRBIT_WAIT_PRODUCER, wc)) {
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
        if (!wait_one<CROSS>(d_empty(acc), ((uint32_t)(lt >> 1) & 1u) ^ 1u, ERRBIT_WAIT_MMA, wc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(acc * p.nt);
        uint32_t accumulate = 0;
#pragma unroll 1
        for (int rk = 0; ok && rk < num_raw; ++rk) {
          // The two halves of a raw stage.
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!wait_one<PAIR ? MEMORY : LOCAL>(conv_full(s), ph, ERRBIT_WAIT_MMA, wc)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t b = desc0 + (uint32_t)s * conv_step;
            const uint32_t a = tmemA + (uint32_t)(W == 3 && s >= 3 ? s - 3 : s) * kAcols;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              umma_f16_ts<PAIR>(d, a + k * 8, b + 2 * k, p.idesc, accumulate);
              accumulate = 1;
            }
            if (PAIR) umma_commit_pair(conv_empty(s));
            else umma_commit<false>(conv_empty(s));
            const bool wrap = s == kConv - 1;
            s = wrap ? 0 : s + 1;
            ph ^= wrap ? 1u : 0u;
          }
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
    const int cw = warp - kFirstConv, set = cw / kSetWarps, role = cw - set * kSetWarps;
    const uint32_t full0 = PAIR ? mapa_shared(conv_full(0), 0) : conv_full(0);
    const int halves = 2 * my_tiles * num_raw;  // the launch keeps this below 2^31
    if (role < kWWarps) {
      // The channel is the TMEM lane, and a warp reaches the quarter warp % 4.
      const int row = (warp & 3) * 32 + lane;
      convert<PAIR, W, true>(set, row, true, halves, sRaw + (uint32_t)row * 128u, p.raw_bytes, p.raw_stages,
                             raw_full(0), full0, conv_empty(0), tmemA + ((uint32_t)((warp & 3) * 32) << 16), 0, wc);
    } else {
      // Warps without tokens stay out; a lane without a token reads the first
      // token's place and writes nothing.
      const int row = (role - kWWarps) * 32 + lane;
      const bool live = row < p.ntc;
      if (row - lane < p.ntc)
        convert<PAIR, W, false>(set, row, live, halves, sRaw + 128 * kRawK + (live ? (uint32_t)row * 128u : 0u),
                                p.raw_bytes, p.raw_stages, raw_full(0), full0, conv_empty(0),
                                sConv + (uint32_t)row * 128u, p.conv_bytes, wc);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    // Two warps a lane quarter, taking 16 tokens in turn.
    const int q = warp & 3, odd = (warp - kFirstEpi) >> 2;
    const uint32_t scales = sScale + (uint32_t)(warp - kFirstEpi) * 1024u;
    int lt = 0;
    bool ok = true;
    for (int tile = first; tile < p.num_tiles; tile += stride, ++lt) {
      int g, n0, m0;
      coords(tile, g, n0, m0);
      const int acc = lt & 1;
      const int n = n0 + q * 32 + lane;
      const bool in = n < p.N;
      const int live_cols = min(p.nt, p.M - m0);
      // While the accumulator is being computed: the scales.  (0.25: the
      // factor of two in each operand.)
      const float sw = in ? 0.25f * p.sw[(size_t)g * p.N + n] : 0.f;
      const float bias = p.bias && in ? to_f(static_cast<const T*>(p.bias)[(size_t)g * p.N + n]) : 0.f;
      for (int c = lane; c < p.nt; c += 32)
        st_shared_f32(scales + 4u * (uint32_t)c, c < live_cols ? p.sa[(size_t)(m0 + c) * p.G + g] : 0.f);
      __syncwarp();
      if (!wait_warp<CROSS>(d_full(acc), (uint32_t)(lt >> 1) & 1u, ERRBIT_WAIT_EPILOGUE, wc)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if constexpr (SPLIT) {
        // Sums [token][128 channels], where the raw stages were: every copy has
        // landed and been converted once the MMAs are done.
#pragma unroll 1
        for (int c0 = 16 * odd; c0 < live_cols; c0 += 32) {
          float v[16];
          tmem_ld_32x16(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)c0, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) st_shared_f32(sRaw + (uint32_t)((c0 + i) * 512 + (q * 32 + lane) * 4), v[i]);
        }
        sum_sw = sw;
        sum_bias = bias;
        continue;
      }
      const uint32_t d = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * p.nt);
      const float2 sw2 = f2(sw), bias2 = f2(bias);
      const size_t step = (size_t)p.G * p.N;
      size_t at = ((size_t)(m0 + 16 * odd) * p.G + g) * p.N + n;
      // Up to 16 tokens of this lane's channel (inlined twice: `cols` is 16
      // for all but the last).  Neighbouring lanes write neighbouring
      // channels.  out may be resid: a value is read before the same thread
      // writes it.
      auto finish = [&](float2* v, int cols) {
        if (p.resid) {
          const T* r = static_cast<const T*>(p.resid) + at;
          T rv[16];
#pragma unroll
          for (int c = 0; c < 16; ++c, r += step) rv[c] = c < cols ? *r : from_f<T>(0.f);
#pragma unroll
          for (int c = 0; c < 8; ++c) v[c] = add2(v[c], make_float2(to_f(rv[2 * c]), to_f(rv[2 * c + 1])));
        }
        T* out = static_cast<T*>(p.out) + at;
#pragma unroll
        for (int c = 0; c < 16; ++c, out += step)
          if (c < cols) *out = from_f<T>(c & 1 ? v[c / 2].y : v[c / 2].x);
      };
#pragma unroll 1
      for (int c0 = 16 * odd; c0 < live_cols; c0 += 32, at += 32 * step) {
        float2 v[8];
        tmem_ld_32x16(d + c0, reinterpret_cast<float*>(v));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 sa = ld_shared_f4(scales + 4u * (uint32_t)(c0 + 4 * i));
          v[2 * i] = fma2(mul2(v[2 * i], make_float2(sa.x, sa.y)), sw2, bias2);
          v[2 * i + 1] = fma2(mul2(v[2 * i + 1], make_float2(sa.z, sa.w)), sw2, bias2);
        }
        if (live_cols - c0 >= 16) {
          if (in) finish(v, 16);
        } else {
          if (in) finish(v, live_cols - c0);
        }
      }
      tc_fence_before();
      __syncwarp();
      arrive_if<CROSS>(PAIR ? mapa_shared(d_empty(acc), 0) : d_empty(acc), lane == 0);
    }
    // No commit may still be on its way to this CTA's barriers at the end:
    // wait for the last use of every stage.
    if (ok && warp == kFirstEpi) {
      const long long its = 2ll * lt * num_raw;
      for (long long j = its > kConv ? its - kConv : 0; ok && j < its; ++j)
        ok = wait_warp<CROSS>(conv_empty((int)(j % kConv)), (uint32_t)(j / kConv) & 1u, ERRBIT_WAIT_DRAIN, wc);
    }
  }

  tc_fence_before();
  __syncthreads();
  // Neither CTA of a pair leaves while the other may still read its shared
  // memory or signal its barriers; TMEM is freed by both together.
  if (PAIR || SPLIT) cluster_barrier();
  if constexpr (SPLIT) {
    if (warp >= kFirstEpi) {
      int g, n0, m0;
      coords(first, g, n0, m0);
      const int ch = (warp & 3) * 32 + lane, odd = (warp - kFirstEpi) >> 2, n = n0 + ch;
      const int live_cols = min(p.nt, p.M - m0);
      const uint32_t scales = sScale + (uint32_t)(warp - kFirstEpi) * 1024u;
      uint32_t sums[kMaxSplit];  // this channel's of each share
#pragma unroll
      for (int k = 0; k < kMaxSplit; ++k) sums[k] = mapa_shared(sRaw + 4u * (uint32_t)ch, k < p.split ? (uint32_t)k : 0u);
      if (n < p.N) {
        // Four tokens at a time: all their shares' loads are in flight.
#pragma unroll 1
        for (int c0 = share + p.split * odd; c0 < live_cols; c0 += 8 * p.split) {
          float x[4][kMaxSplit];
          const size_t step = (size_t)2 * p.split * p.G * p.N;
          const size_t at = ((size_t)(m0 + c0) * p.G + g) * p.N + n;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = c0 + 2 * i * p.split;
#pragma unroll
            for (int k = 0; k < kMaxSplit; ++k) {
              x[i][k] = 0.f;
              if (k < p.split && c < live_cols) x[i][k] = ld_cluster_f32(sums[k] + (uint32_t)c * 512u);
            }
          }
          T r[4];
          if (p.resid) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              r[i] = c0 + 2 * i * p.split < live_cols ? static_cast<const T*>(p.resid)[at + i * step] : from_f<T>(0.f);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = c0 + 2 * i * p.split;
            if (c >= live_cols) break;
            float v = x[i][0];
#pragma unroll
            for (int k = 1; k < kMaxSplit; ++k) v += x[i][k];
            v = fmaf(v * ld_shared_f32(scales + 4u * (uint32_t)c), sum_sw, sum_bias);
            if (p.resid) v += to_f(r[i]);
            static_cast<T*>(p.out)[at + i * step] = from_f<T>(v);
          }
        }
      }
    }
    __syncwarp();
    cluster_barrier();  // the others may still be reading this CTA's sums
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<PAIR>(tmem, kTmemCols);
  }
}

template <typename T, bool PAIR, int W, bool SPLIT>
cudaError_t launch(const CUtensorMap& w, const CUtensorMap& a, const Params& p, cudaStream_t st) {
  auto k = k_linear_q8<T, PAIR, W, SPLIT>;
  const int smem = 1024 + p.raw_stages * p.raw_bytes + kConv * p.conv_bytes + kScaleBytes + kBarBytes;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
  if (e != cudaSuccess) return e;
  const int cluster = SPLIT ? p.split : PAIR ? 2 : 1;
  const int slots = SPLIT ? p.num_tiles : sm_count() / cluster;
  const int n = p.num_tiles < slots ? p.num_tiles : slots;
  return launch_k(k, dim3(cluster * n), dim3(kThreads), smem, st, cluster, w, a, p);
}

// The accumulators of a CTA alone (up to 96 tokens) leave TMEM room for six
// stages of weights, those of a pair for three.
template <typename T>
cudaError_t dispatch(const CUtensorMap& w, const CUtensorMap& a, const Params& p, bool pair, cudaStream_t st) {
  return pair          ? launch<T, true, 3, false>(w, a, p, st)
         : p.split > 1 ? launch<T, false, 6, true>(w, a, p, st)
                       : launch<T, false, 6, false>(w, a, p, st);
}

// CTAs to a tile of nt tokens and num_raw steps (CTAs alone).  Few tiles leave
// most SMs idle; sharing a tile's steps costs two cluster barriers and the sums'
// way through shared memory.  36 clusters of four and 76 of two fit the GPU at
// once.  us, one CTA / two / four to a tile:
//   30 tiles of 16 tokens: 8 steps 7.0 / 7.1 / 6.9, 12 steps 8.4 / 7.8 / 7.1,
//   30 steps 15.0 / 11.1 / 8.9; of 96: 10 steps 9.3 / 10.8 / 9.2, 12 steps
//   10.2 / 11.4 / 9.3, 30 steps 17.9 / 15.6 / 11.6
//   70 tiles of 16 tokens: 10 steps 7.8 / 7.9, 12 steps 8.6 / 8.3, 30 steps
//   15.1 / 11.6; of 96: 16 steps 12.0 / 12.7, 30 steps 18.1 / 16.1
// Eight to a tile gain little more (15 tiles of 30 steps 8.1 against 8.5) and lose
// where no more than 15 such clusters fit (16 tiles 14.9).
int split_of(long long tiles, int nt, int num_raw) {
  if (tiles <= 36) return num_raw >= 8 + nt / 48 ? 4 : 1;
  return tiles <= 72 && num_raw >= 10 + nt / 10 ? 2 : 1;
}

// The sizes, tiles and stages of a product.  False where the kernel's counters
// would not hold it.
bool plan(const LinearQ8& d, Params& p, bool& pair) {
  p.M = d.M;
  p.G = d.G;
  p.K = d.K;
  p.N = d.N;
  // A CTA alone up to 96 tokens (what three warps convert), a pair above: the
  // pair shares the tokens' conversion, which a CTA alone would do for all of
  // them.  16 groups of 1280 -> 5120, us alone / as a pair: 64 tokens 29.5 /
  // 30.0, 96 33.0 / 33.8, 97 47 / 34.6, 192 52 / 39, 1024 242 / 158.  But alone
  // while there is an SM for every tile: they are narrower, and can be shared
  // (pair / alone: 706 x 2 tokens, 2979 -> 214, 18.3 / 10.7; 490 x 5, 2147 -> 357,
  // 14.9 / 12.7; 192 x 8, 256 -> 1024, 7.4 / 5.4).
  const long long alone = (long long)d.G * ((d.N + 127) / 128) * ((d.M + kMaxAlone - 1) / kMaxAlone);
  pair = d.M > kMaxAlone && d.N > 128 && alone > sm_count();
  const int most = pair ? kMaxNT : kMaxAlone;
  p.tiles_m = (d.M + most - 1) / most;
  const int even = (d.M + p.tiles_m - 1) / p.tiles_m;
  p.nt = (even + 15) / 16 * 16;
  p.ntc = pair ? p.nt / 2 : p.nt;
  p.tiles_m = (d.M + p.nt - 1) / p.nt;
  const int tn = pair ? 256 : 128;
  p.tiles_n = (d.N + tn - 1) / tn;
  const long long tiles = (long long)d.G * p.tiles_n * p.tiles_m;
  if (tiles > (1ll << 30)) return false;
  p.num_tiles = (int)tiles;
  p.num_raw = (d.K + kRawK - 1) / kRawK;  // columns past K are zeros
  p.raw_bytes = 128 * kRawK + p.ntc * kRawK;
  p.conv_bytes = p.ntc * kConvK * 2;
  p.raw_stages = (kSmemMax - 1024 - kScaleBytes - kBarBytes - kConv * p.conv_bytes) / p.raw_bytes;
  if (p.raw_stages > kMaxRaw) p.raw_stages = kMaxRaw;
  p.split = pair ? 1 : split_of(tiles, p.nt, p.num_raw);
  const int at_once = pair ? sm_count() / 2 : sm_count();
  const long long rounds = at_once > 0 ? (tiles + at_once - 1) / at_once : tiles;
  return rounds * p.num_raw < (1ll << 30);  // past that: more than 10^19 operations
}

}  // namespace

bool linear_q8_supported(const LinearQ8& d) {
  Params p;
  bool pair;
  return plan(d, p, pair);
}

cudaError_t launch_linear_q8(const LinearQ8& d, unsigned int* err, cudaStream_t st) {
  Params p;
  bool pair;
  if (!plan(d, p, pair)) return cudaErrorInvalidValue;
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
  switch (d.dtype) {
    case 0: return dispatch<float>(w, a, p, pair, st);
    case 1: return dispatch<bf16>(w, a, p, pair, st);
    case 2: return dispatch<f16>(w, a, p, pair, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace rmx
