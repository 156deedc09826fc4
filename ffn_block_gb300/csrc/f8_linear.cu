// Product of 8-bit floating rows, and the weight gradient from 8-bit columns:
//   out[m,g,n] = sum_k t[m,g,k] * w[g,n,k] + bias[g,n] + resid[m,g,n]
// with one power-of-two exponent per 128 k of a row of either operand.
//
// The tensor cores take both exponents themselves (block-scaled MMA: an exponent
// byte for each row and 32 k, here the same byte four times), so the sum over all
// of K stays in the float32 accumulator in tensor memory and the epilogue runs
// once a tile.  An output tile is channels x tokens (as in the int8 product): few
// tokens are a narrow tile, not a padded one; 128 channels a CTA (256 a CTA pair)
// by up to 224 tokens.
//
// Roles (16 warps, one CTA an SM, persistent over tiles):
//   warp 0      TMA producer: 128 k of the CTA's channels and tokens a stage
//   warp 1      TMEM allocation; one thread issues the MMAs (even CTA of a pair)
//   warps 4-7   exponents: 512 k of them at a time from global into tensor
//               memory, a warp to each quarter of its lanes
//   warps 8-15  epilogue: a channel a thread, 16 tokens at a time
// Few tiles with many steps of k: a cluster of two, four or eight CTAs shares a tile's
// steps and adds the sums up through distributed shared memory (split_of).
// TMEM: two accumulators of up to 224 columns (the epilogue of one tile overlaps
// the next), then four places of 12 columns for exponents.
//
// Exponents in tensor memory: a 32-bit word holds a row's for four blocks of k,
// byte i for block 4 j + i; the word of row r is in lane r % 32 (the same in all four
// quarters), column r / 32.  The instruction names the byte.
//
// Groups are tokens of a per-token layer, or experts with rows given by offsets in
// device memory; the weight gradient contracts over a group's rows, whose columns
// then lie in blocks of 128 rows, each group's from a block of its own on.
//
// Measured (GB300): 8192 tokens through 4096 -> 4096 74 us (3.7 PFLOP/s), 1024 x 64
// tokens through 1280 -> 5120 371 us (2.3 PFLOP/s), 32,768 rows of 32 experts through
// 1280 -> 2560 80 us (2.7), the weight gradient of that 93 us (2.3), one sample x 64
// tokens through 1280 -> 5120 66 us (6.3 TB/s, 95% of the copy rate).  A tile of N
// tokens takes as long as N + 118 columns would at the tensor cores' best, so tiles
// are as wide as tensor memory allows (32,768 rows as above: 224 tokens 85 us, 192
// 86, 160 95, 128 107).  Products of few k are bound by their outputs: a plain fill
// writes 3.5 to 4.0 TB/s (16,384 tokens 256 -> 2560 27 us, of which 25 for 84 MB).
// Not kept: outputs in 16-byte pieces of eight tokens (the 371 us 434), through
// shared memory as whole rows (447), more epilogue warps (366 to 377), the next
// tile's operands prefetched to L2 (372).

#include <cuda.h>

#include "common.cuh"
#include "handover.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ragged.cuh"
#include "sparse.h"
#include "tcgen05.cuh"

namespace rmx {
namespace {

constexpr int kFirstExp = 4, kFirstEpi = 8, kEpiWarps = 8, kThreads = 32 * (kFirstEpi + kEpiWarps);
constexpr int kK = 128;                // k of a stage: a block of exponents, a 128-byte row
constexpr int kMaxStages = 8, kSlots = 4, kSlotCols = 12;
constexpr int kMaxNT = 224, kMaxSplit = 8;
constexpr int kTmemCols = 512, kAccCols = kMaxNT, kExpCol0 = 2 * kAccCols;
constexpr int kBarBytes = 256;
constexpr int kSmemMax = 226 * 1024;  // and a little static shared memory
constexpr uint64_t kDrainNs = 50ull * 1000ull * 1000ull;
static_assert(kExpCol0 + kSlots * kSlotCols <= kTmemCols, "tensor memory");

struct Params {
  int M, G, N;                 // rows (tokens, or K of a weight gradient), groups, channels
  int nkb;                     // blocks of k (weight gradient with offsets: by group)
  int nt, ntc;                 // tokens of a tile, and a CTA's share
  int stage_bytes, stages;
  int split;                   // CTAs that share a tile's blocks of k (SPLIT)
  int tiles_m, tiles_n, num_tiles;  // (tiles_m, num_tiles: without offsets, or weight gradient)
  int rows_end;                // last row + 1 of the token operand, for the exponents
  uint32_t idesc;
  const int32_t* offsets;
  int Mcap;                    // rows that offsets may reach
  const uint8_t *te, *we;
  long long te_row, te_group, we_row, we_group;  // bytes between rows and groups
  long long te_word, we_word;                    // and from four blocks' exponents to the next four's
  long long out_row, out_group;                  // elements
  const void *bias, *resid;
  void* out;
  unsigned int* err;
  unsigned long long wait_ns;
};
enum Mode { EQUAL = 0, RAGGED = 1, WGRAD = 2, WGRAD_RAGGED = 3 };

// D[tmem] (+)= A[smem] * B[smem]^T of 8-bit floats, each row of either scaled by
// an exponent in tensor memory.
template <bool PAIR>
__device__ __forceinline__ void umma_mxf8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t ea, uint32_t eb,
                                          uint32_t accumulate) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(ea), "r"(eb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(ea), "r"(eb), "r"(accumulate)
        : "memory");
}
// N words per lane to N consecutive columns; complete after tmem_st_wait().
__device__ __forceinline__ void tmem_st_32x4(uint32_t addr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void tmem_st_32x8(uint32_t addr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t cluster_addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// SPLIT: the CTAs of a cluster each take a share of one tile's blocks of k and leave
// their sums in shared memory; then each adds up every p.split-th token's, in the
// order of the shares, and stores them.  A cluster has one tile.
template <typename T, bool PAIR, int MODE, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear_f8(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmT, const Params p) {
  pdl_trigger();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const uint32_t sRing = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.stages * p.stage_bytes);
  constexpr int NBARS = 2 * kMaxStages + 2 * kSlots + 5;
  static_assert(NBARS * 8 + 8 <= kBarBytes, "barriers");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* first = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + kBarBytes);  // offsets: [G + 1] each
  int* before = first + p.G + 1;
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * (uint32_t)s; };
  auto empty = [&](int s) { return bar0 + 8u * (uint32_t)(kMaxStages + s); };
  auto exp_full = [&](int s) { return bar0 + 8u * (uint32_t)(2 * kMaxStages + s); };
  auto exp_empty = [&](int s) { return bar0 + 8u * (uint32_t)(2 * kMaxStages + kSlots + s); };
  auto d_full = [&](int a) { return bar0 + 8u * (uint32_t)(2 * kMaxStages + 2 * kSlots + a); };
  auto d_empty = [&](int a) { return bar0 + 8u * (uint32_t)(2 * kMaxStages + 2 * kSlots + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (uint32_t)(2 * kMaxStages + 2 * kSlots + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? (int)cluster_rank() : 0;
  const int tile0 = PAIR || SPLIT ? (int)cluster_id_x() : (int)blockIdx.x;
  const int stride = PAIR || SPLIT ? (int)num_clusters_x() : (int)gridDim.x;
  const int share = SPLIT ? (int)cluster_rank() : 0;
  constexpr int CTAS = PAIR ? 2 : 1;
  constexpr Order CROSS = PAIR ? TENSOR : LOCAL;
  constexpr bool OFFSETS = MODE == RAGGED || MODE == WGRAD_RAGGED;
  const WaitCtx wc{p.wait_ns, p.err, abort_flag};

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(exp_full(s), 4 * CTAS);
      mbar_init(exp_empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(d_full(a), 1);
      mbar_init(d_empty(a), kEpiWarps * CTAS);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_map(&tmW);
    prefetch_map(&tmT);
  }
  if (warp == 1) tmem_alloc<PAIR>(smem_u32(tmem_slot), kTmemCols);
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_barrier();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  if (OFFSETS) ragged_scan<kThreads>(p.offsets, p.G, p.Mcap, MODE == RAGGED ? p.nt : kK, first, before);
  const int num_tiles = MODE == RAGGED ? before[p.G] * p.tiles_n : p.num_tiles;

  // A tile: its group, this CTA's first channel, the first token (of all rows
  // where they lie by expert), the tokens it has, its blocks of k and the first
  // of them.  Tiles that share weights are neighbours.
  struct Tile {
    int g, n0, m0, live, nkb, kb0;
  };
  auto tile_of = [&](int tile) {
    Tile t;
    int tn, tm;
    if (MODE == RAGGED) {
      // before[g] * tiles_n <= tile < before[g + 1] * tiles_n
      t.g = ragged_group(before, p.G, tile / p.tiles_n);
      const int mt = before[t.g + 1] - before[t.g], r = tile - before[t.g] * p.tiles_n;
      tn = r / mt;
      tm = r - tn * mt;
      t.m0 = first[t.g] + tm * p.nt;
      t.live = min(p.nt, first[t.g + 1] - t.m0);
    } else {
      tm = tile % p.tiles_m;
      const int r = tile / p.tiles_m;
      tn = r % p.tiles_n;
      t.g = r / p.tiles_n;
      t.m0 = tm * p.nt;
      t.live = min(p.nt, p.M - t.m0);
    }
    t.n0 = tn * 128 * CTAS + rank * 128;
    t.kb0 = MODE == WGRAD_RAGGED ? before[t.g] : 0;
    t.nkb = MODE == WGRAD_RAGGED ? before[t.g + 1] - before[t.g] : p.nkb;
    if (SPLIT) {
      const int k0 = (int)((long long)t.nkb * share / p.split);
      t.nkb = (int)((long long)t.nkb * (share + 1) / p.split) - k0;
      t.kb0 += k0;
    }
    return t;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (elect_one()) {
      int s = 0, issued = 0;
      uint32_t ph = 0;
      bool ok = true;
      const uint32_t full0 = PAIR ? mapa_shared(full(0), 0) : full(0);
      for (int tile = tile0; ok && tile < num_tiles; tile += stride) {
        const Tile t = tile_of(tile);
        const int mr = t.m0 + rank * p.ntc;
        for (int kb = 0; kb < t.nkb; ++kb) {
          if (!wait_one<CROSS>(empty(s), ph ^ 1u, ERRBIT_WAIT_PRODUCER, wc)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_expect_tx(full(s), (uint32_t)(p.stage_bytes * CTAS));
          const uint32_t dst = sRing + (uint32_t)(s * p.stage_bytes), fb = full0 + 8u * (uint32_t)s;
          // Channels {k, N, G}; tokens {k, G, M}, or {k, K, G} of a weight gradient;
          // by expert its operands lie block by block, {128, N or K, block}.
          const int x = MODE == WGRAD_RAGGED ? 0 : (t.kb0 + kb) * kK, wg = MODE == WGRAD_RAGGED ? t.kb0 + kb : t.g;
          const int c1 = MODE == EQUAL ? t.g : MODE == RAGGED ? 0 : mr, c2 = MODE == WGRAD || MODE == WGRAD_RAGGED ? wg : mr;
          if (PAIR) {
            tma_load_3d_pair(dst, &tmW, fb, x, t.n0, wg);
            tma_load_3d_pair(dst + 128 * kK, &tmT, fb, x, c1, c2);
          } else {
            tma_load_3d(dst, &tmW, fb, x, t.n0, wg);
            tma_load_3d(dst + 128 * kK, &tmT, fb, x, c1, c2);
          }
          issued = min(issued + 1, p.stages);
          if (++s == p.stages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // The last use of every stage: the MMAs' commits have arrived here (and no
      // longer travel to this CTA's barriers when it ends).  After a wait that
      // gave up: the copies already issued have landed (a pair's are counted at
      // the even CTA).
      for (; issued > 0; --issued) {
        if (--s < 0) {
          s = p.stages - 1;
          ph ^= 1u;
        }
        volatile int no_abort = 0;
        if (ok) ok = wait_one<CROSS>(empty(s), ph, ERRBIT_WAIT_DRAIN, wc);
        else if (rank == 0) mbar_wait_bounded(full(s), ph, kDrainNs, p.err, ERRBIT_WAIT_DRAIN, &no_abort);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0 && elect_one()) {
      int s = 0, slot = 0, lt = 0;
      uint32_t ph = 0, eph = 0;
      bool ok = true;
      const uint64_t desc0 = sw128_desc(sRing, 16, 1024);
      const uint32_t step = (uint32_t)p.stage_bytes >> 4;  // descriptor addresses count 16 bytes
      for (int tile = tile0; ok && tile < num_tiles; tile += stride, ++lt) {
        const Tile t = tile_of(tile);
        const int acc = lt & 1;
        if (!wait_one<CROSS>(d_empty(acc), ((uint32_t)(lt >> 1) & 1u) ^ 1u, ERRBIT_WAIT_MMA, wc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(acc * kAccCols);
        uint32_t accumulate = 0;
#pragma unroll 1
        for (int kb = 0; kb < t.nkb; ++kb) {
          const uint32_t byte = (uint32_t)(t.kb0 + kb) & 3u;
          if ((byte == 0 || kb == 0) && !wait_one<CROSS>(exp_full(slot), eph, ERRBIT_WAIT_MMA, wc)) {
            ok = false;
            break;
          }
          if (!wait_one<LOCAL>(full(s), ph, ERRBIT_WAIT_MMA, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t a = desc0 + (uint32_t)s * step, b = a + ((128 * kK) >> 4);
          const uint32_t ea = tmem + (uint32_t)(kExpCol0 + slot * kSlotCols), eb = ea + 4;
          const uint32_t idesc = p.idesc | byte << 4 | byte << 29;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            umma_mxf8<PAIR>(d, a + 2 * k, b + 2 * k, idesc, ea, eb, accumulate);
            accumulate = 1;
          }
          if (PAIR) umma_commit_pair(empty(s));
          else umma_commit<false>(empty(s));
          if (byte == 3 || kb == t.nkb - 1) {
            if (PAIR) umma_commit_pair(exp_empty(slot));
            else umma_commit<false>(exp_empty(slot));
            slot = slot == kSlots - 1 ? 0 : slot + 1;
            eph ^= slot == 0 ? 1u : 0u;
          }
          s = s == p.stages - 1 ? 0 : s + 1;
          ph ^= s == 0 ? 1u : 0u;
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
  } else if (warp >= kFirstExp && warp < kFirstEpi) {
    // ------------------------------------------------------------ exponents
    // A word of each row for every four blocks of k: the next four's are on
    // their way while these wait for their place.
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kExpCol0;
    const uint32_t full0 = PAIR ? mapa_shared(exp_full(0), 0) : exp_full(0);
    int slot = 0, used = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int tile = tile0; ok && tile < num_tiles; tile += stride) {
      const Tile t = tile_of(tile);
      // Rows past the end take the last one's: their products are not stored.
      const uint8_t* row[12];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        row[c] = p.we + (MODE == WGRAD_RAGGED ? 0 : (size_t)t.g * p.we_group) + (size_t)min(t.n0 + 32 * c + lane, p.N - 1) * p.we_row;
#pragma unroll
      for (int c = 0; c < 8; ++c)
        row[4 + c] = p.te + (MODE == WGRAD_RAGGED ? 0 : (size_t)t.g * p.te_group) +
                     (size_t)min(t.m0 + 32 * c + lane, p.rows_end - 1) * p.te_row;
      const int q0 = t.kb0 >> 2, q1 = t.nkb > 0 ? (t.kb0 + t.nkb + 3) >> 2 : q0;
      auto load = [&](int q, uint32_t (&w)[12]) {
#pragma unroll
        for (int c = 0; c < 12; ++c)
          w[c] = c < 4 || 32 * (c - 4) < p.nt
                     ? *reinterpret_cast<const uint32_t*>(row[c] + (size_t)q * (c < 4 ? p.we_word : p.te_word))
                     : 0u;
      };
      uint32_t w[12], next[12];
      if (q0 < q1) load(q0, w);
      for (int q = q0; q < q1; ++q) {
        if (q + 1 < q1) load(q + 1, next);
        if (!wait_warp<CROSS>(exp_empty(slot), ph ^ 1u, ERRBIT_WAIT_ROWS, wc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        tmem_st_32x4(lanes + (uint32_t)(slot * kSlotCols), w);
        tmem_st_32x8(lanes + (uint32_t)(slot * kSlotCols + 4), w + 4);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        arrive_if<CROSS>(full0 + 8u * (uint32_t)slot, lane == 0);
        used = min(used + 1, kSlots);
        if (++slot == kSlots) {
          slot = 0;
          ph ^= 1u;
        }
#pragma unroll
        for (int c = 0; c < 12; ++c) w[c] = next[c];
      }
    }
    if (warp == kFirstExp) {
      // The last use of every place, as for the stages.
      for (; ok && used > 0; --used) {
        if (--slot < 0) {
          slot = kSlots - 1;
          ph ^= 1u;
        }
        ok = wait_warp<CROSS>(exp_empty(slot), ph, ERRBIT_WAIT_DRAIN, wc);
      }
    }
  } else if (warp >= kFirstEpi) {
    // ------------------------------------------------------------ epilogue
    // Two warps a lane quarter, taking 16 tokens in turn.
    const int q = warp & 3, odd = (warp - kFirstEpi) >> 2;
    int lt = 0;
    for (int tile = tile0; tile < num_tiles; tile += stride, ++lt) {
      const Tile t = tile_of(tile);
      const int acc = lt & 1, n = t.n0 + q * 32 + lane;
      const bool in = n < p.N;
      const float bias = p.bias && in ? to_f(static_cast<const T*>(p.bias)[(size_t)t.g * p.N + n]) : 0.f;
      if (!wait_warp<CROSS>(d_full(acc), (uint32_t)(lt >> 1) & 1u, ERRBIT_WAIT_EPILOGUE, wc)) break;
      tc_fence_after();
      const uint32_t d = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kAccCols);
      if constexpr (SPLIT) {
        // Sums [token][128 channels], where the ring was: every copy has landed and
        // been multiplied once the MMAs are done.
#pragma unroll 1
        for (int c0 = 16 * odd; c0 < t.live; c0 += 32) {
          float v[16];
          tmem_ld_32x16(d + c0, v);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(sRing + (uint32_t)((c0 + i) * 512 + (q * 32 + lane) * 4)),
                         "f"(t.nkb == 0 ? 0.f : v[i])
                         : "memory");
        }
        continue;
      }
      const size_t step = (size_t)p.out_row;
      size_t at = (size_t)(t.m0 + 16 * odd) * step + (MODE == RAGGED ? 0 : (size_t)t.g * p.out_group) + n;
      // Up to 16 tokens of this lane's channel (inlined twice: `cols` is 16 for
      // all but the last).  Neighbouring lanes write neighbouring channels.  out
      // may be resid: a value is read before the same thread writes it.
      auto finish = [&](float* v, int cols) {
        if (p.resid) {
          const T* r = static_cast<const T*>(p.resid) + at;
          T rv[16];
#pragma unroll
          for (int c = 0; c < 16; ++c, r += step) rv[c] = c < cols ? *r : from_f<T>(0.f);
#pragma unroll
          for (int c = 0; c < 16; ++c) v[c] += to_f(rv[c]);
        }
        T* out = static_cast<T*>(p.out) + at;
#pragma unroll
        for (int c = 0; c < 16; ++c, out += step)
          if (c < cols) *out = from_f<T>(v[c]);
      };
#pragma unroll 1
      for (int c0 = 16 * odd; c0 < t.live; c0 += 32, at += 32 * step) {
        float v[16];
        tmem_ld_32x16(d + c0, v);
        // (A group without rows has had no MMA.)
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = MODE == WGRAD_RAGGED && t.nkb == 0 ? 0.f : v[i] + bias;
        if (t.live - c0 >= 16) {
          if (in) finish(v, 16);
        } else {
          if (in) finish(v, t.live - c0);
        }
      }
      tc_fence_before();
      __syncwarp();
      arrive_if<CROSS>(PAIR ? mapa_shared(d_empty(acc), 0) : d_empty(acc), lane == 0);
    }
  }

  tc_fence_before();
  __syncthreads();
  // Neither CTA of a pair leaves while the other may still read its shared
  // memory or signal its barriers; TMEM is freed by both together.
  if (PAIR || SPLIT) cluster_barrier();
  if constexpr (SPLIT) {
    if (warp >= kFirstEpi) {
      const Tile t = tile_of(tile0);
      const int ch = (warp & 3) * 32 + lane, odd = (warp - kFirstEpi) >> 2, n = t.n0 + ch;
      if (n < p.N) {
        const float bias = p.bias ? to_f(static_cast<const T*>(p.bias)[(size_t)t.g * p.N + n]) : 0.f;
        const size_t at = (size_t)t.m0 * p.out_row + (size_t)t.g * p.out_group + n;
        uint32_t sums[kMaxSplit];  // this channel's of each share
#pragma unroll
        for (int k = 0; k < kMaxSplit; ++k) sums[k] = mapa_shared(sRing + 4u * (uint32_t)ch, k < p.split ? (uint32_t)k : 0u);
        // Two tokens at a time (eight: a microsecond more for one token).
        constexpr int TOK = 2;
#pragma unroll 1
        for (int c0 = share + p.split * odd; c0 < t.live; c0 += 2 * TOK * p.split) {
          float x[TOK][kMaxSplit];
#pragma unroll
          for (int i = 0; i < TOK; ++i) {
            const int c = c0 + 2 * i * p.split;
#pragma unroll
            for (int k = 0; k < kMaxSplit; ++k) {
              x[i][k] = 0.f;
              if (k < p.split && c < t.live) x[i][k] = ld_cluster_f32(sums[k] + (uint32_t)c * 512u);
            }
          }
#pragma unroll
          for (int i = 0; i < TOK; ++i) {
            const int c = c0 + 2 * i * p.split;
            if (c >= t.live) break;
            float v = x[i][0];
#pragma unroll
            for (int k = 1; k < kMaxSplit; ++k) v += x[i][k];
            v += bias;
            const size_t o = at + (size_t)c * p.out_row;
            if (p.resid) v += to_f(static_cast<const T*>(p.resid)[o]);
            static_cast<T*>(p.out)[o] = from_f<T>(v);
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

template <typename T, bool PAIR, int MODE, bool SPLIT>
cudaError_t launch(const CUtensorMap& w, const CUtensorMap& t, const Params& p, long long tiles, cudaStream_t st) {
  auto k = k_linear_f8<T, PAIR, MODE, SPLIT>;
  const int extra = kBarBytes + (MODE == RAGGED || MODE == WGRAD_RAGGED ? 2 * (p.G + 1) * (int)sizeof(int) : 0);
  const int smem = 1024 + p.stages * p.stage_bytes + extra;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
  if (e != cudaSuccess) return e;
  const int cluster = SPLIT ? p.split : PAIR ? 2 : 1;
  const long long slots = SPLIT ? tiles : sm_count() / cluster;
  const int n = (int)(tiles < slots ? tiles : slots);
  return launch_k(k, dim3(cluster * n), dim3(kThreads), smem, st, cluster, w, t, p);
}
template <typename T, int MODE>
cudaError_t by_size(bool pair, const CUtensorMap& w, const CUtensorMap& t, const Params& p, long long tiles, cudaStream_t st) {
  if (pair) return launch<T, true, MODE, false>(w, t, p, tiles, st);
  if constexpr (MODE != RAGGED) {
    if (p.split > 1) return launch<T, false, MODE, true>(w, t, p, tiles, st);
  }
  return launch<T, false, MODE, false>(w, t, p, tiles, st);
}
template <typename T>
cudaError_t dispatch(bool pair, int mode, const CUtensorMap& w, const CUtensorMap& t, const Params& p, long long tiles,
                     cudaStream_t st) {
  switch (mode) {
    case EQUAL: return by_size<T, EQUAL>(pair, w, t, p, tiles, st);
    case RAGGED: return by_size<T, RAGGED>(pair, w, t, p, tiles, st);
    case WGRAD: return by_size<T, WGRAD>(pair, w, t, p, tiles, st);
    default: return by_size<T, WGRAD_RAGGED>(pair, w, t, p, tiles, st);
  }
}

// CTAs to a tile of nt tokens and `steps` blocks of k (CTAs alone).  Few tiles leave
// most SMs idle; a step takes about 0.23 us, and sharing costs about 0.6 us and, for
// each token, 0.035, 0.022 or 0.016 us with two, four or eight CTAs (two cluster
// barriers, and the sums' way through distributed shared memory).  36 clusters of
// four, 76 of two and 15 of eight fit the GPU at once; two are taken up to 72 tiles,
// about what was measured.  us, one CTA / two / four / eight to a tile:
//   15 tiles: 1 token 4096 -> 1920 11.4 / 9.2 / 7.5 / 6.2, 224 tokens 1024 -> 1920
//   6.4 / 14.0 / 10.5 / 9.1, 4096 -> 1920 13.1 / 17.6 / 13.0 / 10.5
//   32 tiles: 8 tokens 4096 -> 4096 11.3 / 9.3 / 7.8, 200 tokens 12.8 / 17.0 / 12.6
//   71 tiles: 1 token 4096 -> 9088 11.4 / 9.4, 1024 -> 9088 5.8 / 6.1
//   weight gradients: 23,770 rows, 1701 x 212 77 / 46 / 29, 65,536 rows, 224 x 1280
//   282 / 131 / 67 / 38
int split_of(long long tiles, int nt, long long steps) {
  for (int s = kMaxSplit; s > 1; s /= 2) {
    const long long fit = s == 8 ? 15 : s == 4 ? 36 : 72;
    if (tiles <= fit && steps * 23 * (s - 1) > 60 * s + (long long)nt * (s + 5)) return s;
  }
  return 1;
}

int mode_of(const LinearF8& d) {
  return d.wgrad ? (d.offsets ? WGRAD_RAGGED : WGRAD) : (d.offsets ? RAGGED : EQUAL);
}

// The sizes, tiles and stages of a product.  False where the kernel's counters
// would not hold it.  `tiles`: how many there are (with offsets: at most).
bool plan(const LinearF8& d, Params& p, bool& pair, long long& tiles) {
  const int mode = mode_of(d);
  p = Params{};
  p.M = d.wgrad ? d.K : d.M;
  p.G = d.G;
  p.N = d.N;
  p.Mcap = d.M;
  p.nkb = d.wgrad ? f8_blocks(d.M) : f8_blocks(d.K);
  // Rows of a tile's operand: with offsets, an expert's share of the rows.
  const long long rows = mode == RAGGED ? (d.M + (long long)d.G - 1) / d.G : p.M;
  const long long alone = (long long)d.G * ((d.N + 127) / 128) * ((rows + 127) / 128);
  pair = rows > 128 && d.N > 128 && alone > sm_count();
  const int unit = pair ? 32 : 16;
  long long tm = (rows + kMaxNT - 1) / kMaxNT;
  const long long even = (rows + tm - 1) / tm;
  p.nt = (int)((even + unit - 1) / unit * unit);
  p.ntc = pair ? p.nt / 2 : p.nt;
  const int tn = pair ? 256 : 128;
  p.tiles_n = (d.N + tn - 1) / tn;
  p.tiles_m = (int)((rows + p.nt - 1) / p.nt);
  // With offsets each expert may end inside a tile.
  const long long mt = mode == RAGGED ? d.M / p.nt + (long long)(d.G < d.M ? d.G : d.M) : (long long)d.G * p.tiles_m;
  tiles = mt * p.tiles_n;
  if (tiles > (1ll << 30)) return false;
  p.num_tiles = (int)tiles;
  // Blocks of k of a tile: a group's share of them where they go by expert.
  const long long steps = mode == WGRAD_RAGGED ? (f8_blocks(d.M) + d.G - 1) / d.G : p.nkb;
  p.split = pair || mode == RAGGED ? 1 : split_of(tiles, p.nt, steps);
  // Strides of a tensor map: below 2^40 bytes.
  const long long pitch = mode == WGRAD_RAGGED ? kK : (long long)p.nkb * kK;
  const long long most = d.K > d.N && d.wgrad ? d.K : d.N;
  if (pitch > (1ll << 30) || pitch * most >= (1ll << 39) || pitch * d.G >= (1ll << 39)) return false;
  p.stage_bytes = (128 + p.ntc) * kK;
  const int extra = 1024 + kBarBytes + (d.offsets ? 2 * (d.G + 1) * (int)sizeof(int) : 0);
  p.stages = (kSmemMax - extra) / p.stage_bytes;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  return true;
}

}  // namespace

bool linear_f8_supported(const LinearF8& d) {
  Params p;
  bool pair;
  long long tiles;
  return plan(d, p, pair, tiles);
}

cudaError_t launch_linear_f8(const LinearF8& d, unsigned int* err, cudaStream_t st) {
  Params p;
  bool pair;
  long long tiles;
  if (!plan(d, p, pair, tiles)) return cudaErrorInvalidValue;
  const int mode = mode_of(d);
  // Block-scaled 8-bit MMA, exponents of 8 bits, both operands K-major; A is
  // the channels, B the tokens.
  p.idesc = (uint32_t)d.w_format << 7 | (uint32_t)d.t_format << 10 | (uint32_t)(p.nt >> 3) << 17 | 1u << 23 |
            (uint32_t)((pair ? 256 : 128) >> 4) << 24;
  p.offsets = d.offsets;
  p.te = d.te;
  p.we = d.we;
  p.bias = d.bias;
  p.resid = d.resid;
  p.out = d.out;
  p.err = err;
  p.wait_ns = kWaitLimitNs;
  const uint64_t M = d.M, G = d.G, K = d.K, N = d.N;
  // Bytes of a row of either operand, and how many matrices of rows there are.
  const bool blocks = mode == WGRAD_RAGGED;
  const uint64_t pitch = blocks ? kF8Block : f8_pitch(d.wgrad ? d.M : d.K), exps = f8_exps(d.wgrad ? d.M : d.K);
  const uint64_t mats = blocks ? ragged_blocks(d.M, d.G) : G;
  CUtensorMap w, t;
  bool ok = make_tensor_map_rows8(&w, d.w, pitch, N, mats, pitch, N * pitch, 128, 1);
  p.we_row = p.te_row = (long long)exps;
  p.we_word = p.te_word = 4;
  p.we_group = (long long)(N * exps);
  p.rows_end = p.M;
  p.out_row = (long long)N;
  switch (mode) {
    case EQUAL:
      ok = ok && make_tensor_map_rows8(&t, d.t, pitch, G, M, pitch, G * pitch, 1, (uint32_t)p.ntc);
      p.te_row = (long long)(G * exps);
      p.te_group = (long long)exps;
      p.out_row = (long long)(G * N);
      p.out_group = (long long)N;
      break;
    case RAGGED:
      ok = ok && make_tensor_map_rows8(&t, d.t, pitch, 1, M, pitch, pitch, 1, (uint32_t)p.ntc);
      break;
    case WGRAD:
      ok = ok && make_tensor_map_rows8(&t, d.t, pitch, K, G, pitch, K * pitch, (uint32_t)p.ntc, 1);
      p.te_group = (long long)(K * exps);
      p.out_group = (long long)(K * N);
      break;
    default:
      ok = ok && make_tensor_map_rows8(&t, d.t, pitch, K, mats, pitch, K * pitch, (uint32_t)p.ntc, 1);
      p.we_row = p.te_row = 4;
      p.we_word = (long long)(4 * N);
      p.te_word = (long long)(4 * K);
      p.out_group = (long long)(K * N);
  }
  if (!ok) return cudaErrorInvalidValue;
  switch (d.dtype) {
    case 0: return dispatch<float>(pair, mode, w, t, p, tiles, st);
    case 1: return dispatch<bf16>(pair, mode, w, t, p, tiles, st);
    case 2: return dispatch<f16>(pair, mode, w, t, p, tiles, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace rmx
