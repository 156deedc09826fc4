// Routing rows to experts: slots sorted by expert, rows gathered in that order,
// experts' rows added up at their tokens, and the backward of that.
//
// The sort counts.  A warp takes its slots in order, 32 at a time: lanes with
// the same expert find one another by votes, so a slot's place among them is a
// population count, and the first of them moves the warp's own counter on.  No
// atomics: the order is the slots' own.  Up to 2048 slots are sorted by one CTA, up
// to 49,152 by a cluster of eight, whose CTAs read one another's counts, in one
// launch; more by three launches: each warp counts its share, each expert's counts
// are summed over the warps, and each warp places its share.
//
// The rows are bound by HBM.  65,536 tokens to two of 64 experts, 1280 bf16 columns:
// sort 13 us, gather 95 us (336 MB written: 84 us at the rate of pure writes, 4.0
// TB/s), combination 76 us (6.6 TB/s), its backward 139 us (6.0 TB/s).

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "q8_rows.cuh"
#include "sparse.h"
#include "tcgen05.cuh"

namespace rmx {
namespace {

__device__ __forceinline__ uint32_t lanes_below() {
  uint32_t m;
  asm("mov.u32 %0, %%lanemask_lt;" : "=r"(m));
  return m;
}
__device__ __forceinline__ int expert_of(const int32_t* expert, long long slot, long long end, int E) {
  const int e = slot < end ? expert[slot] : -1;
  return (uint32_t)e < (uint32_t)E ? e : -1;
}
// The lanes with this lane's expert (of 2^bits), one vote a bit: 131,072 slots to 64
// experts, cold: 33 us with the match instruction, 25 with votes.
__device__ __forceinline__ uint32_t same_expert(int e, int bits) {
  uint32_t same = __ballot_sync(0xffffffffu, e >= 0);
  for (int b = 0; b < bits; ++b) {
    const bool one = (e >> b) & 1;
    const uint32_t ones = __ballot_sync(0xffffffffu, one);
    same &= one ? ones : ~ones;
  }
  return same;  // (of no meaning where e < 0)
}
__device__ __forceinline__ int expert_bits(int E) { return 32 - __clz(E - 1); }
// Loads of a warp in flight at a time.
constexpr int kAhead = 4;
// Slots [begin, end) of a warp (32 at a time, all lanes together) counted into
// its own hist[E].
__device__ __forceinline__ void count_slots(const int32_t* expert, long long begin, long long end, int E, int* hist) {
  const int lane = threadIdx.x & 31, bits = expert_bits(E);
  for (long long s0 = begin; s0 < end; s0 += 32 * kAhead) {
    int id[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) id[i] = expert_of(expert, s0 + 32 * i + lane, end, E);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const uint32_t same = same_expert(id[i], bits);
      if (id[i] >= 0 && (same & lanes_below()) == 0) hist[id[i]] += __popc(same);
      __syncwarp();
    }
  }
}
// The same slots given their places: hist[e] is the warp's next place of expert e.
__device__ __forceinline__ void place_slots(const int32_t* expert, long long begin, long long end, int E, int* hist,
                                            int32_t* position, int32_t* source) {
  const int lane = threadIdx.x & 31, bits = expert_bits(E);
  for (long long s0 = begin; s0 < end; s0 += 32 * kAhead) {
    int id[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) id[i] = expert_of(expert, s0 + 32 * i + lane, end, E);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const long long slot = s0 + 32 * i + lane;
      const int e = id[i];
      const uint32_t same = same_expert(e, bits);
      const uint32_t below = same & lanes_below();
      const int first = e >= 0 ? hist[e] : 0;
      __syncwarp();
      if (e >= 0 && below == 0) hist[e] = first + __popc(same);
      __syncwarp();
      if (slot < end) {
        const int at = e >= 0 ? first + __popc(below) : -1;
        position[slot] = at;
        if (e >= 0) source[at] = (int32_t)slot;
      }
    }
  }
}
// Exclusive prefix over the block's threads of v; `total` gets the sum.  tmp: 33
// ints.  blockDim.x is a multiple of 32.
__device__ __forceinline__ int block_prefix(int v, int* tmp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) tmp[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const int mine = lane < warps ? tmp[lane] : 0;
    int s = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    if (lane < warps) tmp[lane] = s - mine;
    if (lane == 31) tmp[32] = s;
  }
  __syncthreads();
  total = tmp[32];
  return tmp[warp] + inc - v;
}

constexpr int kWarps = 32;             // of a CTA that sorts, at most
// Slots that one CTA sorts by itself, and that a cluster does.  us for 64 experts, a
// CTA / a cluster / three launches: 2048 slots 7.1 / - / -, 8192 11.9 / 7.8 / -,
// 32,768 - / 8.6 / 10.8, 65,536 - / 12.9 / 11.7, 131,072 - / 21.4 / 13.1.
constexpr int kOneSlots = 2048, kCluster = 8, kClusterSlots = 49152;

__device__ __forceinline__ int ld_cluster_s32(uint32_t cluster_addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// CTAS: 1, or a cluster of kCluster, each CTA with the next kWarps shares.
// blockDim.x >= E, and at least 32 * warps.
template <int CTAS>
__global__ void __launch_bounds__(32 * kWarps) k_sort(int S, int E, int warps, int share, const int32_t* expert,
                                                      int32_t* offsets, int32_t* position, int32_t* source) {
  pdl_enter();
  extern __shared__ int hist[];  // [warps][E], then this CTA's count of each expert [E]
  __shared__ int tmp[33];
  int* mine = hist + warps * E;
  const int warp = threadIdx.x >> 5, rank = CTAS > 1 ? (int)cluster_rank() : 0;
  for (int i = threadIdx.x; i < warps * E; i += blockDim.x) hist[i] = 0;
  __syncthreads();
  const long long begin = min((long long)S, (long long)(rank * warps + warp) * share), end = min((long long)S, begin + share);
  if (warp < warps) count_slots(expert, begin, end, E, hist + warp * E);
  __syncthreads();
  int n = 0;
  const int e = threadIdx.x;
  if (e < E) {
    for (int w = 0; w < warps; ++w) {
      const int c = hist[w * E + e];
      hist[w * E + e] = n;
      n += c;
    }
    mine[e] = n;
  }
  int all = n, base = 0;
  if (CTAS > 1) {
    cluster_barrier();
    if (e < E) {
      const uint32_t at = smem_u32(mine + e);
      all = 0;
#pragma unroll
      for (int r = 0; r < CTAS; ++r) {
        const int c = ld_cluster_s32(mapa_shared(at, (uint32_t)r));
        base += r < rank ? c : 0;
        all += c;
      }
    }
    cluster_barrier();  // none leaves, or goes on to count, while another reads
  }
  int total;
  const int off = block_prefix(e < E ? all : 0, tmp, total);
  if (e < E) {
    if (rank == 0) offsets[e] = off;
    for (int w = 0; w < warps; ++w) hist[w * E + e] += off + base;
  }
  if (rank == 0 && threadIdx.x == 0) offsets[E] = total;
  __syncthreads();
  if (warp < warps) place_slots(expert, begin, end, E, hist + warp * E, position, source);
  for (long long i = total + (long long)rank * blockDim.x + threadIdx.x; i < S; i += CTAS * blockDim.x) source[i] = -1;
}

// ws: counts [warps][E], then totals [E].
constexpr int kManyWarps = 8;
__global__ void __launch_bounds__(32 * kManyWarps) k_sort_count(int S, int E, int share, int warps, const int32_t* expert,
                                                                int32_t* counts) {
  pdl_enter();
  extern __shared__ int hist[];
  const int warp = threadIdx.x >> 5, gw = blockIdx.x * kManyWarps + warp;
  for (int i = threadIdx.x; i < kManyWarps * E; i += 32 * kManyWarps) hist[i] = 0;
  __syncthreads();
  const long long begin = min((long long)S, (long long)gw * share), end = min((long long)S, begin + share);
  count_slots(expert, begin, end, E, hist + warp * E);
  __syncthreads();
  const int rows = min(kManyWarps, warps - (int)blockIdx.x * kManyWarps);
  int32_t* out = counts + (size_t)blockIdx.x * kManyWarps * E;
  for (int i = threadIdx.x; i < rows * E; i += 32 * kManyWarps) out[i] = hist[i];
}
// counts become, per expert, the sums over the warps before; a CTA takes 32
// experts, a warp of it a range of the rows.
__global__ void __launch_bounds__(1024) k_sort_scan(int E, int warps, int32_t* counts, int32_t* totals) {
  pdl_enter();
  __shared__ int sums[32][33];
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
  const int share = (warps + 31) / 32, begin = min(warps, part * share), end = min(warps, begin + share);
  int n = 0;
  if (e < E)
    for (int w = begin; w < end; ++w) n += counts[(size_t)w * E + e];
  sums[part][lane] = n;
  __syncthreads();
  int before = 0;
  for (int p = 0; p < part; ++p) before += sums[p][lane];
  if (e < E) {
    if (part == 31) totals[e] = before + n;
    for (int w = begin; w < end; ++w) {
      const int c = counts[(size_t)w * E + e];
      counts[(size_t)w * E + e] = before;
      before += c;
    }
  }
}
__global__ void __launch_bounds__(32 * kManyWarps) k_sort_place(int S, int E, int share, int warps, const int32_t* expert,
                                                                const int32_t* counts, const int32_t* totals,
                                                                int32_t* offsets, int32_t* position, int32_t* source) {
  pdl_enter();
  extern __shared__ int hist[];  // [8][E], then offsets [E]
  __shared__ int tmp[33];
  int* off = hist + kManyWarps * E;
  int run = 0;
  for (int e0 = 0; e0 < E; e0 += 32 * kManyWarps) {
    const int e = e0 + threadIdx.x;
    int total;
    const int before = block_prefix(e < E ? totals[e] : 0, tmp, total);
    if (e < E) off[e] = run + before;
    run += total;
    __syncthreads();
  }
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e < E; e += 32 * kManyWarps) offsets[e] = off[e];
    if (threadIdx.x == 0) offsets[E] = run;
  }
  const int rows = min(kManyWarps, warps - (int)blockIdx.x * kManyWarps);
  const int32_t* in = counts + (size_t)blockIdx.x * kManyWarps * E;
  for (int i = threadIdx.x; i < rows * E; i += 32 * kManyWarps) hist[i] = in[i] + off[i % E];
  __syncthreads();
  const int warp = threadIdx.x >> 5, gw = blockIdx.x * kManyWarps + warp;
  const long long begin = min((long long)S, (long long)gw * share), end = min((long long)S, begin + share);
  if (begin < end) place_slots(expert, begin, end, E, hist + warp * E, position, source);
  for (long long i = run + (long long)blockIdx.x * blockDim.x + threadIdx.x; i < S; i += (long long)gridDim.x * blockDim.x)
    source[i] = -1;
}
// A warp's share of the slots: 256 (128 or 512: 131,072 slots in 14.6 and 15.8 us, not
// 13.1), or what keeps the warps at 4096.
int share_of(int S) {
  const int least = (int)(((long long)S + 4095) / 4096);
  return least <= 256 ? 256 : (least + 31) / 32 * 32;
}

// ---------------------------------------------------------------- rows
// A unit is a block of 8 * L columns of a row.
struct Units {
  int bpr;
  long long total;
};
template <int L> Units units_of(long long rows, int C) {
  Units u;
  u.bpr = (C + 8 * L - 1) / (8 * L);
  u.total = rows * u.bpr;
  return u;
}
__device__ __forceinline__ long long row_of(const Units& u, long long i, int& blk) {
  const long long r = u.total < (1ll << 31) ? (long long)((uint32_t)i / (uint32_t)u.bpr) : i / u.bpr;
  blk = (int)(i - r * u.bpr);
  return r;
}

constexpr int kBatch = 4;
template <typename T, int L, bool VEC>
__global__ void __launch_bounds__(256) k_gather(const Units u, int S, int k, int C, const bool stream, const int32_t* source,
                                                const T* x, T* out) {
  pdl_enter();
  constexpr int PER = 256 / L;
  const int lane = threadIdx.x & (L - 1);
  const long long step = (long long)gridDim.x * PER * kBatch;
  for (long long u0 = (long long)blockIdx.x * PER * kBatch + threadIdx.x / L; u0 < u.total; u0 += step) {
    Chunk<T> c[kBatch];
    long long row[kBatch];
    int c0[kBatch], src[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const long long i = u0 + j * PER;
      int blk = 0;
      row[j] = i < u.total ? row_of(u, i, blk) : -1;
      c0[j] = col0<L, VEC>(blk, lane);
      src[j] = row[j] >= 0 ? source[row[j]] : -1;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if ((uint32_t)src[j] < (uint32_t)S) c[j] = load_chunk<T, L, VEC>(x + (size_t)((uint32_t)src[j] / (uint32_t)k) * C, c0[j], C);
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if ((uint32_t)src[j] < (uint32_t)S) {
        T* o = out + (size_t)row[j] * C;
        if constexpr (VEC) {
          constexpr int V = 16 / (int)sizeof(T);
          const uint4* s = reinterpret_cast<const uint4*>(&c[j]);
#pragma unroll
          for (int i = 0; i < 8 / V; ++i)
            if (c0[j] + i * V < C) {
              uint4* q = reinterpret_cast<uint4*>(o + c0[j]) + i;
              if (stream) __stcs(q, s[i]);
              else *q = s[i];
            }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (col<L, VEC>(c0[j], i) < C) o[col<L, VEC>(c0[j], i)] = c[j].v[i];
        }
      }
  }
}

template <typename T, int L, bool VEC>
__global__ void __launch_bounds__(256) k_combine(const Units u, int S, int k, int C, const int32_t* position,
                                                 const float* weight, const T* y, T* out) {
  pdl_enter();
  constexpr int PER = 256 / L;
  const int lane = threadIdx.x & (L - 1);
  const long long step = (long long)gridDim.x * PER;
  for (long long i = (long long)blockIdx.x * PER + threadIdx.x / L; i < u.total; i += step) {
    int blk;
    const long long t = row_of(u, i, blk);
    const int c0 = col0<L, VEC>(blk, lane);
    const int32_t* pos = position + t * k;
    const float* w = weight ? weight + t * k : nullptr;
    float2 acc[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = f2(0.f);
    for (int j0 = 0; j0 < k; j0 += 4) {
      Chunk<T> c[4];
      int p[4];
      float f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[j] = j0 + j < k ? pos[j0 + j] : -1;
        f[j] = j0 + j < k && w ? w[j0 + j] : 1.f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((uint32_t)p[j] < (uint32_t)S) c[j] = load_chunk<T, L, VEC>(y + (size_t)p[j] * C, c0, C);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((uint32_t)p[j] < (uint32_t)S) {
          float2 v[4];
          to_pairs(c[j], v);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] = fma2(v[e], f2(f[j]), acc[e]);
        }
    }
    store_chunk<T, L, VEC>(out + (size_t)t * C, c0, C, acc);
  }
}

// The same for rows of more than 512 columns: a warp has a segment of NCH blocks of
// a token's row and two experts' rows of it on their way at a time, and knows the
// next token's rows before it is done with this one.
template <typename T, int NCH, bool VEC>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1)
    k_combine_rows(int tokens, int S, int k, int C, const int segs, const int32_t* position, const float* weight, const T* y,
                   T* out) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const uint32_t units = (uint32_t)tokens * (uint32_t)segs;  // segments of 1.5 KB and more: far below 2^31
  const uint32_t step = gridDim.x * 8;
  uint32_t u = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (u >= units) return;
  struct Slot {
    int p;
    float w;
  };
  auto slot = [&](uint32_t t, int j) {
    Slot s{-1, 1.f};
    if (j < k) {
      s.p = position[(size_t)t * k + j];
      if (weight) s.w = weight[(size_t)t * k + j];
    }
    return s;
  };
  uint32_t t = u / (uint32_t)segs;
  Slot a = slot(t, 0), b = slot(t, 1);
  while (true) {
    const int seg0 = (int)(u - t * (uint32_t)segs) * NCH;
    const uint32_t nu = u + step, nt = nu < units ? nu / (uint32_t)segs : 0;
    float2 acc[NCH][4];
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = f2(0.f);
    for (int j = 0; j < k; j += 2) {
      Chunk<T> ca[NCH], cb[NCH];
      const bool la = (uint32_t)a.p < (uint32_t)S, lb = (uint32_t)b.p < (uint32_t)S;
      if (la) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) ca[i] = load_chunk<T, 32, VEC>(y + (size_t)a.p * C, col0<32, VEC>(seg0 + i, lane), C);
      }
      if (lb) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) cb[i] = load_chunk<T, 32, VEC>(y + (size_t)b.p * C, col0<32, VEC>(seg0 + i, lane), C);
      }
      const float wa = a.w, wb = b.w;
      if (j + 2 < k) {
        a = slot(t, j + 2);
        b = slot(t, j + 3);
      } else if (nu < units) {
        a = slot(nt, 0);
        b = slot(nt, 1);
      }
      auto add = [&](const Chunk<T> (&c)[NCH], float w) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          float2 v[4];
          to_pairs(c[i], v);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][e] = fma2(v[e], f2(w), acc[i][e]);
        }
      };
      if (la) add(ca, wa);
      if (lb) add(cb, wb);
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i) store_chunk<T, 32, VEC>(out + (size_t)t * C, col0<32, VEC>(seg0 + i, lane), C, acc[i]);
    if (nu >= units) return;
    u = nu;
    t = nt;
  }
}

// A token belongs to L lanes of W warps with NCH blocks each, dout's row in
// registers while its k rows of y pass.
template <typename T, int L, int NCH, bool VEC>
__global__ void __launch_bounds__(512) k_combine_bwd(int tokens, int S, int k, int C, const int W, const int rpb,
                                                     const int32_t* position, const float* weight, const T* dout,
                                                     const T* y, T* dy, float* dweight) {
  pdl_enter();
  __shared__ float red[64];
  const int lane = threadIdx.x & (L - 1), part = threadIdx.x / L, rib = part / W, w = part - rib * W;
  float* my_red = red + rib * 2 * W;
  auto c_of = [&](int j) { return col0<L, VEC>(w + j * W, lane); };
  const long long step = (long long)gridDim.x * rpb;
  const int first_of_warp = L == 32 ? rib : (threadIdx.x >> 5) * (32 / L);
  int slot = 0;
  for (long long t = (long long)blockIdx.x * rpb + rib; t - rib + first_of_warp < tokens; t += step) {
    const bool live = L == 32 || t < tokens;
    Chunk<T> cd[NCH];
#pragma unroll
    for (int j = 0; j < NCH; ++j) cd[j] = load_chunk<T, L, VEC>(dout + (size_t)(live ? t : 0) * C, c_of(j), live ? C : 0);
    for (int i = 0; i < k; ++i) {
      const int p = live ? position[t * k + i] : -1;
      const bool in = (uint32_t)p < (uint32_t)S;
      const float f = in && weight ? weight[t * k + i] : 1.f;
      const size_t at = (size_t)(in ? p : 0) * C;
      Chunk<T> cy[NCH];
      if (dweight) {
#pragma unroll
        for (int j = 0; j < NCH; ++j) cy[j] = load_chunk<T, L, VEC>(y + at, c_of(j), in ? C : 0);
      }
      float2 dot = f2(0.f);
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        float2 d[4], v[4];
        to_pairs(cd[j], d);
        if (dweight) {
          to_pairs(cy[j], v);
#pragma unroll
          for (int e = 0; e < 4; ++e) dot = fma2(d[e], v[e], dot);
        }
        if (dy) {
#pragma unroll
          for (int e = 0; e < 4; ++e) d[e] = mul2(d[e], f2(f));
          if (in) store_chunk<T, L, VEC>(dy + at, c_of(j), C, d);
        }
      }
      if (dweight) {
        float s = lanes_sum<L>(dot.x + dot.y);
        if (L == 32 && W > 1) {
          float* r = my_red + slot * W;
          if (lane == 0) r[w] = s;
          asm volatile("bar.sync %0, %1;" ::"r"(1 + rib), "r"(32 * W) : "memory");
          s = 0.f;
          for (int q = 0; q < W; ++q) s += r[q];
          slot ^= 1;
        }
        if (live && w == 0 && lane == 0) dweight[t * k + i] = in ? s : 0.f;
      }
    }
  }
}

unsigned grid_of(long long units, int per_block) {
  const long long want = (units + per_block - 1) / per_block, most = (long long)sm_count() * 64;
  return (unsigned)(want < most ? want : most);
}

template <typename T, bool VEC>
cudaError_t gather(const Routes& r, const int32_t* source, const void* x, void* out, cudaStream_t st) {
  auto go = [&](auto k, const Units& u, int per) {
    // A token's row is read again for its next expert: outputs that would push it out
    // of L2 leave first (65536 x 2 rows of 1280 16-bit columns 105 us, 95 like this).
    const bool stream = (long long)r.S * r.C * (int)sizeof(T) > (64ll << 20);
    return launch_k(k, dim3(grid_of(u.total, per * kBatch)), dim3(256), 0, st, 1, u, r.S, r.k, r.C, stream, source, (const T*)x,
                    (T*)out);
  };
  if (r.C <= 64) return go(k_gather<T, 8, VEC>, units_of<8>(r.S, r.C), 32);
  if (r.C <= 128) return go(k_gather<T, 16, VEC>, units_of<16>(r.S, r.C), 16);
  return go(k_gather<T, 32, VEC>, units_of<32>(r.S, r.C), 8);
}
template <typename T, bool VEC>
cudaError_t combine(const Routes& r, const int32_t* position, const float* weight, const void* y, void* out,
                    cudaStream_t st) {
  auto go = [&](auto k, const Units& u, int per) {
    return launch_k(k, dim3(grid_of(u.total, per)), dim3(256), 0, st, 1, u, r.S, r.k, r.C, position, weight, (const T*)y,
                    (T*)out);
  };
  if (r.C <= 64) return go(k_combine<T, 8, VEC>, units_of<8>(r.T, r.C), 32);
  if (r.C <= 128) return go(k_combine<T, 16, VEC>, units_of<16>(r.T, r.C), 16);
  const int blocks = (r.C + 255) / 256;
  if (blocks > 2) {
    const int segs = (blocks + 4) / 5, nch = (blocks + segs - 1) / segs;
    auto k = nch == 3 ? k_combine_rows<T, 3, VEC> : nch == 4 ? k_combine_rows<T, 4, VEC> : k_combine_rows<T, 5, VEC>;
    const long long want = ((long long)r.T * segs + 7) / 8, fit = (sizeof(T) == 2 ? 2ll : 1ll) * sm_count();
    return launch_k(k, dim3((unsigned)(want < fit ? want : fit)), dim3(256), 0, st, 1, r.T, r.S, r.k, r.C, segs, position,
                    weight, (const T*)y, (T*)out);
  }
  return go(k_combine<T, 32, VEC>, units_of<32>(r.T, r.C), 8);
}
// Blocks of 256 columns that a warp of k_combine_bwd takes of a token's row of `blocks`
// of them, more than one.  16-bit types: as few warps as five blocks each allow, the
// blocks shared evenly (us, 240 MB of experts' rows, four a warp / like this: 512
// columns 176 / 103, 600 166 / 109, 1536 148 / 98, 2560 133 / 106, 8192 129 / 122; 1280
// as two warps of three 105, as one of five 103; 64 tokens 4 in all of them).  Float32:
// four, but five where the row is then one warp's (1280 columns, 23,437 tokens 103 / 89;
// 64 tokens 3.8 / 5.6).  Fewer blocks or five elsewhere win and lose there: two for
// 512 columns 58,593 tokens 107 / 93, 2000 tokens 4.8 / 6.6; five for 2560 columns
// 11,718 tokens 105 / 90, 64 tokens 3.9 / 5.8.
template <typename T> int bwd_blocks(int blocks) {
  if (sizeof(T) == 4) return blocks == 5 ? 5 : 4;
  const int warps = (blocks + 4) / 5;
  return (blocks + warps - 1) / warps;
}
template <typename T, bool VEC>
cudaError_t combine_bwd(const Routes& r, const int32_t* position, const float* weight, const void* dout, const void* y,
                        void* dy, float* dweight, cudaStream_t st) {
  const int blocks = (r.C + 255) / 256;
  auto go = [&](auto k, int L, int nch) {
    const int W = L < 32 ? 1 : (blocks + nch - 1) / nch;
    const int rpb = W == 1 ? 256 / L : W < 8 ? 8 / W : 1;
    const long long want = ((long long)r.T + rpb - 1) / rpb, most = (long long)sm_count() * 16;
    return launch_k(k, dim3((unsigned)(want < most ? want : most)), dim3(L * W * rpb), 0, st, 1, r.T, r.S, r.k, r.C, W, rpb,
                    position, weight, (const T*)dout, (const T*)y, (T*)dy, dweight);
  };
  if (r.C <= 64) return go(k_combine_bwd<T, 8, 1, VEC>, 8, 1);
  if (r.C <= 128) return go(k_combine_bwd<T, 16, 1, VEC>, 16, 1);
  if (blocks <= 1) return go(k_combine_bwd<T, 32, 1, VEC>, 32, 1);
  const int nch = bwd_blocks<T>(blocks);
  if constexpr (sizeof(T) == 2) {
    if (nch == 2) return go(k_combine_bwd<T, 32, 2, VEC>, 32, 2);
    if (nch == 3) return go(k_combine_bwd<T, 32, 3, VEC>, 32, 3);
  }
  if (nch == 4) return go(k_combine_bwd<T, 32, 4, VEC>, 32, 4);
  return go(k_combine_bwd<T, 32, 5, VEC>, 32, 5);
}

}  // namespace

int sort_warps(int S) {
  if (S <= kClusterSlots) return 0;
  const int share = share_of(S);
  return (int)(((long long)S + share - 1) / share);
}

cudaError_t launch_expert_sort(const Routes& r, const int32_t* expert, int32_t* offsets, int32_t* position,
                               int32_t* source, int32_t* ws, int pass, cudaStream_t st) {
  const int warps = sort_warps(r.S), E = r.E;
  if (warps == 0) {
    const bool one = r.S <= kOneSlots;
    // A warp to every 32 slots, up to what the CTAs have.
    const int most = (r.S + 31) / 32, nw = !one ? kWarps : most < 1 ? 1 : most < kWarps ? most : kWarps;
    const int all = one ? nw : kCluster * kWarps, share = ((r.S + all - 1) / all + 31) / 32 * 32;
    const int threads = 32 * nw > (E + 31) / 32 * 32 ? 32 * nw : (E + 31) / 32 * 32;
    const int smem = (nw + 1) * E * (int)sizeof(int);  // 132 KB at most
    auto k = one ? k_sort<1> : k_sort<kCluster>;
    cudaError_t e = allow_smem(k, smem, (kWarps + 1) * kMaxExperts * (int)sizeof(int));
    if (e != cudaSuccess) return e;
    return launch_k(k, dim3(one ? 1 : kCluster), dim3(threads), smem, st, one ? 1 : kCluster, r.S, E, nw, share, expert, offsets,
                    position, source);
  }
  const int share = share_of(r.S), ctas = (warps + kManyWarps - 1) / kManyWarps;
  int32_t* totals = ws + (size_t)warps * E;
  const int hist = kManyWarps * E * (int)sizeof(int);
  if (pass == 0) return launch_k(k_sort_count, dim3(ctas), dim3(32 * kManyWarps), hist, st, 1, r.S, E, share, warps, expert, ws);
  if (pass == 1) return launch_k(k_sort_scan, dim3((E + 31) / 32), dim3(1024), 0, st, 1, E, warps, ws, totals);
  return launch_k(k_sort_place, dim3(ctas), dim3(32 * kManyWarps), hist + E * (int)sizeof(int), st, 1, r.S, E, share, warps,
                  expert, (const int32_t*)ws, (const int32_t*)totals, offsets, position, source);
}

cudaError_t launch_expert_gather(const Routes& r, const int32_t* source, const void* x, void* out, cudaStream_t st) {
  RMX_BY_DTYPE(r.dtype,
               return rows_aligned(r.C, sizeof(T)) ? gather<T, true>(r, source, x, out, st) : gather<T, false>(r, source, x, out, st))
}
cudaError_t launch_expert_combine(const Routes& r, const int32_t* position, const float* weight, const void* y,
                                  void* out, cudaStream_t st) {
  RMX_BY_DTYPE(r.dtype, return rows_aligned(r.C, sizeof(T)) ? combine<T, true>(r, position, weight, y, out, st)
                                                            : combine<T, false>(r, position, weight, y, out, st))
}
cudaError_t launch_expert_combine_bwd(const Routes& r, const int32_t* position, const float* weight, const void* dout,
                                      const void* y, void* dy, float* dweight, cudaStream_t st) {
  RMX_BY_DTYPE(r.dtype, return rows_aligned(r.C, sizeof(T))
                                   ? combine_bwd<T, true>(r, position, weight, dout, y, dy, dweight, st)
                                   : combine_bwd<T, false>(r, position, weight, dout, y, dy, dweight, st))
}

}  // namespace rmx
