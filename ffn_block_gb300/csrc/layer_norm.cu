// Layer norm with dropout and the residual before it, its backward, and dropout
// by itself.
//
//   h = drop(x) + r;  y = (h - mean) * rstd * gamma + beta
//   dr = rstd * (t - mean(t) - xh * mean(t * xh)) + dh,  t = dy * gamma, xh = (h - mean) * rstd
//
// Bound by HBM: one pass over the data each, the row in registers between its
// moments and its output.  The moments are taken in two steps (mean, then the
// squared deviations), and both directions subtract the mean before they multiply, so
// a row far from zero loses no more than its mean's rounding.  (Float32 rows of mean 1000
// and deviation 1: with h * rstd - mean * rstd in one operation the backward's xh was off
// by up to 6e-5, like this by 2e-7.)
// The backward's outputs take two operations an element, with rstd in the row's means.
//
// Measured (GB300, 65,536 rows of 1280 bf16 columns, dropout and residual; a copy
// moves 6.68 TB/s): forward 108 us (6.2 TB/s), backward 142 us with its column sums
// (5.9 TB/s), dropout alone 76 us with a residual (6.6 TB/s) and 63 without (5.3:
// there the generator's integer operations bound it).

#include "common.cuh"
#include "dropout.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "q8_rows.cuh"
#include "sparse.h"
#include "tcgen05.cuh"

namespace rmx {
namespace {

// Sums of N values over the L lanes and W warps of a row, in a fixed order.
// `red` holds two slots of N floats a warp, used in turn; the row's warps meet
// at a barrier of their own.
template <int L, int N>
__device__ __forceinline__ void row_sums(float (&s)[N], float* red, int slot, int w, int W, int barrier) {
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = lanes_sum<L>(s[i]);
  if (L < 32 || W == 1) return;
  float* r = red + slot * N * W;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) r[N * w + i] = s[i];
  }
  asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(32 * W) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = 0.f;
  for (int j = 0; j < W; ++j) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += r[N * j + i];
  }
}

// Zeroes the elements past the row's end.
template <int L, bool VEC> __device__ __forceinline__ void mask_end(float2 (&v)[4], int c0, int C) {
  if (col<L, VEC>(c0, 7) < C) return;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (col<L, VEC>(c0, i) >= C) (i & 1 ? v[i / 2].y : v[i / 2].x) = 0.f;
}

// A lane's eight column sums to a row of partials (rows of it start anywhere).
template <int L, bool VEC> __device__ __forceinline__ void store_partial(float* row, int c0, int C, const float2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (col<L, VEC>(c0, i) < C) row[col<L, VEC>(c0, i)] = i & 1 ? v[i / 2].y : v[i / 2].x;
}

// ---------------------------------------------------------------- dropout
// A unit is a block of 8 * L columns of a row, a lane takes eight of them;
// kUnits units at a time, so that their loads are in flight together.  (The units'
// generators round by round, sharing the keys: 96 us for 65,536 x 1280 with a
// residual, one after the other 76.)
constexpr int kUnits = 4;
template <typename T, int L, bool VEC>
__global__ void __launch_bounds__(256) k_dropout(long long row0, uint32_t units, int bpr, int step_row, int step_blk, int C,
                                                 const Drop d, const T* x, const T* r, T* out) {
  pdl_enter();
  const int lane = threadIdx.x & (L - 1);
  const DropBits bits = drop_bits(d);
  constexpr int PER = 256 / L;
  const uint32_t u0 = blockIdx.x * (PER * kUnits) + threadIdx.x / L;
  Chunk<T> cx[kUnits], cr[kUnits];
  long long row[kUnits];
  int c0[kUnits];
  bool live[kUnits];
  // One division; from unit to unit PER blocks on.
  uint32_t ur = u0 / (uint32_t)bpr, blk = u0 - ur * (uint32_t)bpr;
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    live[j] = u0 + (uint32_t)(j * PER) < units;
    row[j] = live[j] ? row0 + ur : row0;
    c0[j] = col0<L, VEC>(live[j] ? (int)blk : 0, lane);
    blk += (uint32_t)step_blk;
    ur += (uint32_t)step_row + (blk >= (uint32_t)bpr ? 1u : 0u);
    blk -= blk >= (uint32_t)bpr ? (uint32_t)bpr : 0u;
    const int end = live[j] ? C : 0;
    cx[j] = load_chunk<T, L, VEC>(x + (size_t)row[j] * C, c0[j], end);
    if (r) cr[j] = load_chunk<T, L, VEC>(r + (size_t)row[j] * C, c0[j], end);
  }
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    float2 v[4];
    to_pairs(cx[j], v);
    drop_values<L, VEC>(bits, d.scale, row[j], c0[j], v);
    if (r) {
      float2 w[4];
      to_pairs(cr[j], w);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = add2(v[i], w[i]);
    }
    if (live[j]) store_chunk<T, L, VEC>(out + (size_t)row[j] * C, c0[j], C, v);
  }
}

template <typename T, int L, bool VEC>
cudaError_t dropout(long long R, int C, const Drop& d, const void* x, const void* r, void* out, cudaStream_t st) {
  const int bpr = (C + 8 * L - 1) / (8 * L);
  // 32-bit unit numbers: the largest tensors go in ranges of rows.
  const long long most = (1ll << 30) / bpr;
  for (long long row0 = 0; row0 < R; row0 += most) {
    const long long rows = R - row0 < most ? R - row0 : most;
    const uint32_t units = (uint32_t)(rows * bpr);
    const uint32_t per = 256 / L * kUnits;
    cudaError_t e = launch_k(k_dropout<T, L, VEC>, dim3((units + per - 1) / per), dim3(256), 0, st, 1, row0, units, bpr,
                             256 / L / bpr, 256 / L % bpr, C, d, (const T*)x, (const T*)r, (T*)out);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}
template <typename T>
cudaError_t dropout_t(long long R, int C, const Drop& d, const void* x, const void* r, void* out, cudaStream_t st) {
  const bool vec = rows_aligned(C, sizeof(T));
  if (C <= 64) return vec ? dropout<T, 8, true>(R, C, d, x, r, out, st) : dropout<T, 8, false>(R, C, d, x, r, out, st);
  if (C <= 128) return vec ? dropout<T, 16, true>(R, C, d, x, r, out, st) : dropout<T, 16, false>(R, C, d, x, r, out, st);
  return vec ? dropout<T, 32, true>(R, C, d, x, r, out, st) : dropout<T, 32, false>(R, C, d, x, r, out, st);
}

// ---------------------------------------------------------------- rows through shared memory
// Rows longer than 512 columns.  A warp has a segment of NCH blocks of 256 columns
// of a row (rows of up to 1280 columns belong to one warp) and brings its rows in
// with bulk copies into shared memory of its own, `depth` rows ahead: what is in
// flight takes no registers, which hold the row's values and (backward) the column
// sums, 16 a block.  Warps meet only where a row has several.
//
// VEC: rows start on 16-byte boundaries.  Else a copy brings the 16-byte vectors
// that a segment lies in, and the segment starts inside the first of them; of the
// tensor's last vector, where it is not a whole one, the elements are loaded one
// by one.
constexpr int kRingSmem = 200 * 1024, kRingParams = 24 * 1024;  // forward
constexpr int kBwdRingSmem = 220 * 1024, kRingMaxDepth = 3;
constexpr uint64_t kDrainNs = 50ull * 1000ull * 1000ull;
template <typename T, bool VEC> constexpr int ring_pitch(int nch) { return nch * 256 + (VEC ? 0 : 32 / (int)sizeof(T)); }
template <typename T, int NCH, bool VEC> struct RowRing {
  static constexpr int SEG = NCH * 256, PITCH = ring_pitch<T, VEC>(NCH);
  T* base;            // [depth][nt][PITCH]
  uint32_t bar0;      // depth barriers
  const T* src[3];
  int nt, depth, seg0, seg, C;
  long long R, step;
  int s;              // the stage of the row at hand, and its parity
  uint32_t ph;
  bool failed;

  // The bytes of a segment that copies bring, from its first vector on; 0 where the
  // segment lies in the tensor's last vector and that is not a whole one.
  __device__ __forceinline__ void range(long long row, size_t& from, uint32_t& bytes) const {
    const size_t b0 = ((size_t)row * C + seg0) * sizeof(T), b1 = b0 + (size_t)seg * sizeof(T);
    from = VEC ? b0 : b0 & ~(size_t)15;
    const size_t all = (size_t)R * C * sizeof(T) & ~(size_t)15, up = (b1 + 15) & ~(size_t)15;
    bytes = (uint32_t)((VEC ? b1 : up < all ? up : all) - from);
  }
  __device__ __forceinline__ void issue(long long row, int stage) const {
    if ((threadIdx.x & 31) != 0 || row >= R) return;
    const uint32_t bar = bar0 + 8u * (uint32_t)stage, dst = smem_u32(base + (size_t)stage * nt * PITCH);
    size_t from;
    uint32_t bytes;
    range(row, from, bytes);
    if (!VEC && bytes == 0) {  // a segment inside the tensor's last vector, where that is not a whole one
      mbar_arrive(bar);
      return;
    }
    mbar_arrive_expect_tx(bar, bytes * (uint32_t)nt);
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < nt)
        bulk_g2s(dst + (uint32_t)(i * PITCH * (int)sizeof(T)), reinterpret_cast<const char*>(src[i]) + from, bytes, bar);
  }
  // Eight values of a tensor of the row at hand, block j of the segment; zeros past
  // its end (VEC: written once, by init).
  __device__ __forceinline__ Chunk<T> load(const T* row, int tensor, int j) const {
    const int lane = threadIdx.x & 31;
    const T* p = row + tensor * PITCH;
    if constexpr (VEC) return whole(p + j * 256 + lane * 8);
    else return load_chunk<T, 32, false>(p, j * 256 + lane, seg);
  }
  static __device__ __forceinline__ Chunk<T> whole(const T* p) {
    Chunk<T> k;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(&k)[i] = reinterpret_cast<const uint4*>(p)[i];
    return k;
  }
  // The warp's barriers; before the block meets.
  __device__ __forceinline__ void init() {
    if (VEC)
      for (int i = 0; i < depth * nt; ++i)
        for (int c = seg + (int)(threadIdx.x & 31); c < SEG; c += 32) base[i * PITCH + c] = from_f<T>(0.f);
    if ((threadIdx.x & 31) == 0) {
      for (int i = 0; i < depth; ++i) mbar_init(bar0 + 8u * (uint32_t)i, 1);
      fence_mbar_init();
    }
    s = 0;
    ph = 0;
    failed = false;
  }
  __device__ __forceinline__ void start(long long row0) const {
    for (int i = 0; i < depth; ++i) issue(row0 + i * step, i);
  }
  // Waits for the row at hand, and returns where its segment starts.  A wait that
  // gives up leaves the block's barriers in step: the warp goes on (with what it
  // finds), waits no more and issues nothing.
  __device__ __forceinline__ const T* wait(long long row, unsigned long long limit, unsigned int* err, volatile int* abort) {
    if (!failed) {
      const bool ok = mbar_wait_bounded(bar0 + 8u * (uint32_t)s, ph, limit, err, ERRBIT_WAIT_ROWS, abort);
      failed = !__all_sync(0xffffffffu, ok);
    }
    T* stage = base + (size_t)s * nt * PITCH;
    if constexpr (VEC) return stage;
    size_t from;
    uint32_t bytes;
    range(row, from, bytes);
    const size_t b0 = ((size_t)row * C + seg0) * sizeof(T);
    T* in = stage + (b0 - from) / sizeof(T);
    // The elements that copies have brought (none where bytes is 0: from is then at most b0).
    const int there = bytes == 0 ? 0 : (int)((from + bytes - b0) / sizeof(T)), lane = threadIdx.x & 31;
    if (there < seg) {
      if (there + lane < seg) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (i < nt) in[i * PITCH + there + lane] = src[i][b0 / sizeof(T) + there + lane];
      }
      __syncwarp();
    }
    return in;
  }
  // The row has been read: its stage takes the one `depth` rows on.  The copy is of
  // the async proxy: a proxy fence orders the warp's reads before its writes.
  __device__ __forceinline__ void next(long long row) {
    fence_proxy_async_smem();
    __syncwarp();
    if (failed) return;
    issue(row + depth * step, s);
    if (++s == depth) {
      s = 0;
      ph ^= 1u;
    }
  }
  // After a wait that gave up (s, ph have stayed at that row): copies still on
  // their way land before the shared memory is used again or the block ends.
  __device__ __forceinline__ void drain(long long gave_up, unsigned int* err) {
    if (!failed) return;
    volatile int no_abort = 0;
    for (int i = 0; i < depth && gave_up + i * step < R; ++i) {
      mbar_wait_bounded(bar0 + 8u * (uint32_t)s, ph, kDrainNs, err, ERRBIT_WAIT_DRAIN, &no_abort);
      if (++s == depth) {
        s = 0;
        ph ^= 1u;
      }
    }
  }
};
// W warps to a row, rpb rows at a time, as many as shared memory and `threads`
// hold; deeper where there is room.
struct RingSpread {
  int W, nch, rpb, depth, smem;
};
// `few`: the number of blocks to stay at as long as a warp has no second row (0: no
// such wish).
RingSpread ring_spread(long long R, int C, int dtype, int nt, int threads, int smem, long long few = 0) {
  RingSpread s;
  const int blocks = (C + 255) / 256;
  s.W = (blocks + 4) / 5;
  s.nch = (blocks + s.W - 1) / s.W;
  const int e = dtype == 0 ? 4 : 2, row_bytes = nt * (s.nch * 256 * e + (rows_aligned(C, e) ? 0 : 32));
  int warps = smem / (2 * row_bytes);
  if (warps > threads / 32) warps = threads / 32;
  s.rpb = warps / s.W;
  // Few rows: on as many SMs as there are.
  const long long on = few && R <= few * s.rpb ? few : sm_count(), share = (R + on - 1) / on;
  if (s.rpb > share) s.rpb = (int)share;
  s.depth = s.rpb > 0 ? smem / (s.rpb * s.W * row_bytes) : 0;
  if (s.depth > kRingMaxDepth) s.depth = kRingMaxDepth;
  // No deeper than a warp has rows: with less shared memory a small launch starts sooner.
  const long long at_once = (long long)sm_count() * s.rpb, rows = at_once > 0 ? (R + at_once - 1) / at_once : 0;
  if (s.depth > rows) s.depth = (int)rows;
  s.smem = s.rpb * s.W * s.depth * row_bytes;
  // The backward's partials take the ring's place at the end.
  const int partials = (s.rpb - 1) * 2 * s.W * s.nch * 256 * (int)sizeof(float);
  if (few && s.smem < partials) s.smem = partials;
  return s;
}

// ---------------------------------------------------------------- forward
// Forward: 16 warps of 128 registers two rows deep, gamma and beta in shared memory:
// 108 us for 65,536 x 1280, when the choice was made 117 (12 warps with them in
// registers 124, 20 or 24 warps, which spill, 160 and 165; without a ring 130 to
// 200).  Backward: 8 warps of 255 registers, a row's values kept from its sums to its
// output: 142 us, then 145 (12 warps that work them out again 176, without a ring 350).
constexpr int kFwdRingThreads = 512, kBwdRingThreads = 256;
template <typename T, int NCH, bool VEC>
__global__ void __launch_bounds__(kFwdRingThreads, 1)
    k_layer_norm_ring(const LnFwd a, const int W, const int rpb, const int depth, const bool staged, unsigned int* err,
                      const unsigned long long limit) {
  pdl_trigger();
  constexpr int SEG = NCH * 256;
  extern __shared__ uint4 ring_smem[];
  __shared__ float red[64];
  __shared__ uint64_t bars[kRingMaxDepth * (kFwdRingThreads / 32)];
  __shared__ int abort_flag;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rib = warp / W, w = warp - rib * W;
  const int seg0 = w * SEG, seg = min(SEG, a.C - seg0);
  RowRing<T, NCH, VEC> ring;
  ring.nt = a.r ? 2 : 1;
  ring.depth = depth;
  ring.base = reinterpret_cast<T*>(ring_smem) + (size_t)warp * (depth * ring.nt * ring.PITCH);
  ring.bar0 = smem_u32(bars + kRingMaxDepth * warp);
  ring.src[0] = static_cast<const T*>(a.x);
  ring.src[1] = static_cast<const T*>(a.r);
  ring.src[2] = nullptr;
  ring.seg0 = seg0;
  ring.C = a.C;
  ring.seg = seg;
  ring.R = a.R;
  ring.step = (long long)gridDim.x * rpb;
  ring.init();
  if (threadIdx.x == 0) abort_flag = 0;
  __syncthreads();
  pdl_wait();
  const long long row0 = (long long)blockIdx.x * rpb + rib;
  ring.start(row0);
  const DropBits bits = drop_bits(a.drop);
  const float inv_n = 1.f / (float)a.C;
  float* my_red = red + rib * 2 * W;
  // gamma and beta in shared memory behind the ring, where they fit.
  T* const held = reinterpret_cast<T*>(ring_smem) + (size_t)rpb * W * (depth * ring.nt * ring.PITCH);
  const int pitch = W * SEG;
  if (staged) {
    constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;
    using U = typename std::conditional<VEC, uint4, T>::type;
    for (int c = V * (int)threadIdx.x; c < a.C; c += V * (int)blockDim.x) {
      if (a.gamma) *reinterpret_cast<U*>(held + c) = *reinterpret_cast<const U*>(static_cast<const T*>(a.gamma) + c);
      if (a.beta) *reinterpret_cast<U*>(held + pitch + c) = *reinterpret_cast<const U*>(static_cast<const T*>(a.beta) + c);
    }
    __syncthreads();
  }
  auto param = [&](const void* p, int i, int c) {
    return load_chunk<T, 32, VEC>(staged ? held + i * pitch : static_cast<const T*>(p), c, a.C);
  };
  long long gave_up = row0;
  for (long long row = row0; row < a.R; row += ring.step) {
    const T* in = ring.wait(row, limit, err, &abort_flag);
    if (!ring.failed) gave_up = row + ring.step;
    const size_t at = (size_t)row * a.C;
    float2 v[NCH][4], s2 = f2(0.f);
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int c0 = seg0 + col0<32, VEC>(j, lane);
      to_pairs(ring.load(in, 0, j), v[j]);
      drop_values<32, VEC>(bits, a.drop.scale, row, c0, v[j]);
      if (a.r) {
        float2 r[4];
        to_pairs(ring.load(in, 1, j), r);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = add2(v[j][i], r[i]);
      }
      if (a.h) store_chunk<T, 32, VEC>(static_cast<T*>(a.h) + at, c0, a.C, v[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) s2 = add2(s2, v[j][i]);
    }
    ring.next(row);
    float s[1] = {s2.x + s2.y};
    row_sums<32, 1>(s, my_red, 0, w, W, 1 + rib);
    const float mean = s[0] * inv_n;
    s2 = f2(0.f);
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = add2(v[j][i], f2(-mean));
      if (seg != SEG) mask_end<32, VEC>(v[j], seg0 + col0<32, VEC>(j, lane), a.C);
#pragma unroll
      for (int i = 0; i < 4; ++i) s2 = fma2(v[j][i], v[j][i], s2);
    }
    s[0] = s2.x + s2.y;
    row_sums<32, 1>(s, my_red, 1, w, W, 1 + rib);
    const float rstd = 1.f / sqrtf(s[0] * inv_n + a.eps);
    if (w == 0 && lane == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = mul2(v[j][i], f2(rstd));
      float2 g[4], b[4];
      if (a.gamma) {
        to_pairs(param(a.gamma, 0, seg0 + col0<32, VEC>(j, lane)), g);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = mul2(v[j][i], g[i]);
      }
      if (a.beta) {
        to_pairs(param(a.beta, 1, seg0 + col0<32, VEC>(j, lane)), b);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = add2(v[j][i], b[i]);
      }
      store_chunk<T, 32, VEC>(static_cast<T*>(a.y) + at, seg0 + col0<32, VEC>(j, lane), a.C, v[j]);
    }
  }
  ring.drain(gave_up, err);
}
template <typename T, bool VEC> cudaError_t layer_norm_ring(const LnFwd& a, const RingSpread& s, cudaStream_t st) {
  auto k = s.nch == 3 ? k_layer_norm_ring<T, 3, VEC> : s.nch == 4 ? k_layer_norm_ring<T, 4, VEC> : k_layer_norm_ring<T, 5, VEC>;
  const int params = 2 * s.W * s.nch * 256 * (int)sizeof(T);
  // (Worth its wait where a warp has several rows.)
  const bool staged = (a.gamma || a.beta) && params <= kRingParams && a.R > 4ll * s.rpb * sm_count();
  const size_t smem = s.smem + (staged ? params : 0);
  cudaError_t e = allow_smem(k, smem, kRingSmem + kRingParams);
  if (e != cudaSuccess) return e;
  const long long want = (a.R + s.rpb - 1) / s.rpb;
  return launch_k(k, dim3((unsigned)(want < sm_count() ? want : sm_count())), dim3(32 * s.W * s.rpb),
                  smem, st, 1, a, s.W, s.rpb, s.depth, staged, device_error_word(), (unsigned long long)kWaitLimitNs);
}

// Other rows: a row belongs to L lanes of W warps (W > 1 only with L = 32), with
// NCH blocks of 8 * L columns each; rpb rows at a time to a thread block, RB of
// them to each thread (W = 1), whose loads and shuffles are in flight together.
// One block after another on an SM's resident ones would start each with its loads
// exposed: the grid is what fits at once, and blocks go through the rows.
constexpr int kFwdBlocks = 2;  // an SM (three, four or six of them spill and are slower)
template <typename T, int L, int NCH, int RB, bool VEC, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? kFwdBlocks : 1) k_layer_norm(const LnFwd a, const int W, const int rpb) {
  pdl_enter();
  __shared__ float red[64];
  const int lane = threadIdx.x & (L - 1), part = threadIdx.x / L, rib = part / W, w = part - rib * W;
  const DropBits bits = drop_bits(a.drop);
  const float inv_n = 1.f / (float)a.C;
  float* my_red = red + rib * 2 * RB * W;
  const long long step = (long long)gridDim.x * rpb;
  auto c_of = [&](int j) { return col0<L, VEC>(w + j * W, lane); };
  // Parts of a warp stay in the loop together (their shuffles take every lane).
  const int first_of_warp = L == 32 ? rib : (threadIdx.x >> 5) * (32 / L);
  for (long long row0 = (long long)blockIdx.x * rpb + rib; row0 - rib + first_of_warp < a.R; row0 += RB * step) {
    Chunk<T> cx[RB][NCH], cr[RB][NCH];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const long long row = row0 + r * step;
      const bool live = row < a.R;
      const size_t at = (size_t)(live ? row : 0) * a.C;
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        cx[r][j] = load_chunk<T, L, VEC>(static_cast<const T*>(a.x) + at, c_of(j), live ? a.C : 0);
        if (a.r) cr[r][j] = load_chunk<T, L, VEC>(static_cast<const T*>(a.r) + at, c_of(j), live ? a.C : 0);
      }
    }
    float2 v[RB][NCH][4];
    float s[RB], mean[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const long long row = row0 + r * step;
      float2 s2 = f2(0.f);
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        float2(&u)[4] = v[r][j];
        to_pairs(cx[r][j], u);
        drop_values<L, VEC>(bits, a.drop.scale, row, c_of(j), u);
        if (a.r) {
          float2 t[4];
          to_pairs(cr[r][j], t);
#pragma unroll
          for (int i = 0; i < 4; ++i) u[i] = add2(u[i], t[i]);
        }
        if (a.h && row < a.R) store_chunk<T, L, VEC>(static_cast<T*>(a.h) + (size_t)row * a.C, c_of(j), a.C, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) s2 = add2(s2, u[i]);
      }
      s[r] = s2.x + s2.y;
    }
    row_sums<L, RB>(s, my_red, 0, w, W, 1 + rib);
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      mean[r] = s[r] * inv_n;
      float2 s2 = f2(0.f);
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        float2(&u)[4] = v[r][j];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = add2(u[i], f2(-mean[r]));
        mask_end<L, VEC>(u, c_of(j), a.C);
#pragma unroll
        for (int i = 0; i < 4; ++i) s2 = fma2(u[i], u[i], s2);
      }
      s[r] = s2.x + s2.y;
    }
    row_sums<L, RB>(s, my_red, 1, w, W, 1 + rib);
    float rstd[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const long long row = row0 + r * step;
      rstd[r] = 1.f / sqrtf(s[r] * inv_n + a.eps);
      if (row < a.R && w == 0 && lane == 0) {
        if (a.mean) a.mean[row] = mean[r];
        if (a.rstd) a.rstd[row] = rstd[r];
      }
    }
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float2 g[4], b[4];
      if (a.gamma) to_pairs(load_chunk<T, L, VEC>(static_cast<const T*>(a.gamma), c_of(j), a.C), g);
      if (a.beta) to_pairs(load_chunk<T, L, VEC>(static_cast<const T*>(a.beta), c_of(j), a.C), b);
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        const long long row = row0 + r * step;
        float2(&u)[4] = v[r][j];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u[i] = mul2(u[i], f2(rstd[r]));
          if (a.gamma) u[i] = mul2(u[i], g[i]);
          if (a.beta) u[i] = add2(u[i], b[i]);
        }
        if (row < a.R) store_chunk<T, L, VEC>(static_cast<T*>(a.y) + (size_t)row * a.C, c_of(j), a.C, u);
      }
    }
  }
}

struct Spread {
  int L, W, nch, rpb, threads;
};
// Up to 512 columns a warp (or a part of it) has the row to itself, without a
// barrier; above (the rows that the rings do not hold), warps with four blocks each.
Spread fwd_spread(int C) {
  Spread s;
  const int blocks = (C + 255) / 256;
  s.L = C <= 64 ? 8 : C <= 128 ? 16 : 32;
  s.nch = blocks <= 2 ? blocks : 4;
  s.W = (blocks + s.nch - 1) / s.nch;
  s.rpb = s.W == 1 ? 256 / s.L : s.W < 8 ? 8 / s.W : 1;
  s.threads = s.L * s.W * s.rpb;
  return s;
}
template <typename T, bool VEC> cudaError_t layer_norm(const LnFwd& a, cudaStream_t st) {
  if (a.C > 512) {
    const RingSpread r = ring_spread(a.R, a.C, a.dtype, a.r ? 2 : 1, kFwdRingThreads, kRingSmem);
    if (r.rpb >= 1) return layer_norm_ring<T, VEC>(a, r, st);
  }
  const Spread s = fwd_spread(a.C);
  auto go = [&](auto k, int rb) {
    const long long share = (long long)s.rpb * rb, want = (a.R + share - 1) / share, most = (long long)sm_count() * kFwdBlocks;
    // Few rows: as many blocks as there are rows to give them.
    const long long few = (a.R + s.rpb - 1) / s.rpb, least = few < sm_count() ? few : sm_count();
    const long long grid = want < least ? least : want < most ? want : most;
    return launch_k(k, dim3((unsigned)grid), dim3(s.threads), 0, st, 1, a, s.W, s.rpb);
  };
  if (s.L == 8) return go(k_layer_norm<T, 8, 1, 4, VEC, 256>, 4);
  if (s.L == 16) return go(k_layer_norm<T, 16, 1, 4, VEC, 256>, 4);
  if (s.nch == 1) return go(k_layer_norm<T, 32, 1, 4, VEC, 256>, 4);
  if (s.nch == 2) return go(k_layer_norm<T, 32, 2, 2, VEC, 256>, 2);
  return go(k_layer_norm<T, 32, 4, 1, VEC, 512>, 1);
}

// ---------------------------------------------------------------- backward
// Other rows, as in the forward.
template <typename T, int L, int NCH, int RB, bool VEC, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 2 : 1) k_layer_norm_bwd(const LnBwd a, const int W, const int rpb) {
  pdl_enter();
  __shared__ float red[64];
  extern __shared__ float cols[];  // partials of the block's sets of warps
  const int lane = threadIdx.x & (L - 1), part = threadIdx.x / L, rib = part / W, w = part - rib * W;
  const DropBits bits = drop_bits(a.drop);
  const float inv_n = 1.f / (float)a.C;
  float* my_red = red + rib * 4 * RB * W;
  auto c_of = [&](int j) { return col0<L, VEC>(w + j * W, lane); };
  float2 ag[NCH][4], ab[NCH][4];
  Chunk<T> gm[NCH];
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    if (a.gamma) gm[j] = load_chunk<T, L, VEC>(static_cast<const T*>(a.gamma), c_of(j), a.C);
#pragma unroll
    for (int i = 0; i < 4; ++i) ag[j][i] = ab[j][i] = f2(0.f);
  }
  const long long step = (long long)gridDim.x * rpb;
  int slot = 0;
  const int first_of_warp = L == 32 ? rib : (threadIdx.x >> 5) * (32 / L);
  for (long long row0 = (long long)blockIdx.x * rpb + rib; row0 - rib + first_of_warp < a.R; row0 += RB * step, slot ^= 1) {
    Chunk<T> cy[RB][NCH], ch[RB][NCH], cd[RB][NCH];
    float rstd[RB], mean[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const long long row = row0 + r * step;
      const bool live = row < a.R;
      const size_t at = (size_t)(live ? row : 0) * a.C;
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        cy[r][j] = load_chunk<T, L, VEC>(static_cast<const T*>(a.dy) + at, c_of(j), live ? a.C : 0);
        ch[r][j] = load_chunk<T, L, VEC>(static_cast<const T*>(a.h) + at, c_of(j), live ? a.C : 0);
        if (a.dh) cd[r][j] = load_chunk<T, L, VEC>(static_cast<const T*>(a.dh) + at, c_of(j), live ? a.C : 0);
      }
      rstd[r] = live ? a.rstd[row] : 0.f;
      mean[r] = live ? a.mean[row] : 0.f;
    }
    auto both = [&](int r, int j, float2 (&xh)[4], float2 (&t)[4]) {
      to_pairs(ch[r][j], xh);
      to_pairs(cy[r][j], t);
#pragma unroll
      for (int i = 0; i < 4; ++i) xh[i] = mul2(add2(xh[i], f2(-mean[r])), f2(rstd[r]));
    };
    auto weigh = [&](int j, float2 (&t)[4]) {
      if (!a.gamma) return;
      float2 g[4];
      to_pairs(gm[j], g);
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = mul2(t[i], g[i]);
    };
    float m[2 * RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      float2 m1 = f2(0.f), m2 = f2(0.f);
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        float2 xh[4], t[4];
        both(r, j, xh, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ag[j][i] = fma2(t[i], xh[i], ag[j][i]);
          ab[j][i] = add2(t[i], ab[j][i]);
        }
        weigh(j, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          m1 = add2(m1, t[i]);
          m2 = fma2(t[i], xh[i], m2);
        }
      }
      m[2 * r] = m1.x + m1.y;
      m[2 * r + 1] = m2.x + m2.y;
    }
    row_sums<L, 2 * RB>(m, my_red, slot, w, W, 1 + rib);
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const long long row = row0 + r * step;
      const bool live = row < a.R;
      const size_t at = (size_t)(live ? row : 0) * a.C;
      const float2 rs = f2(rstd[r]), c1 = f2(-m[2 * r] * inv_n * rstd[r]), c2 = f2(-m[2 * r + 1] * inv_n * rstd[r]);
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        float2 xh[4], t[4];
        both(r, j, xh, t);
        weigh(j, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = fma2(t[i], rs, fma2(xh[i], c2, c1));
        if (a.dh) {
          float2 d[4];
          to_pairs(cd[r][j], d);
#pragma unroll
          for (int i = 0; i < 4; ++i) t[i] = add2(t[i], d[i]);
        }
        if (live) store_chunk<T, L, VEC>(static_cast<T*>(a.dr) + at, c_of(j), a.C, t);
        if (a.dx) {
          drop_values<L, VEC>(bits, a.drop.scale, row, c_of(j), t);
          if (live) store_chunk<T, L, VEC>(static_cast<T*>(a.dx) + at, c_of(j), a.C, t);
        }
      }
    }
  }
  // The block's partials: parts of a warp in a tree of shuffles, then the sets
  // of warps in order, the first adding the others' to its own.
  const int sets = L == 32 ? rpb : blockDim.x / 32, set = L == 32 ? rib : threadIdx.x >> 5;
  const int set_size = 2 * W * NCH * 8 * L;  // [2][W][NCH][8][L]
  float* mine = cols + w * (NCH * 8 * L) + lane;
  auto each = [&](auto f) {
#pragma unroll
    for (int j = 0; j < NCH; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        f(i & 1 ? ag[j][i / 2].y : ag[j][i / 2].x, i & 1 ? ab[j][i / 2].y : ab[j][i / 2].x, (j * 8 + i) * L);
  };
  each([&](float& g, float& b, int at) {
#pragma unroll
    for (int o = L; o < 32; o <<= 1) {
      g += __shfl_xor_sync(0xffffffffu, g, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (set > 0) {  // (the parts of a warp write the same values)
      mine[(set - 1) * set_size + at] = g;
      mine[(set - 1) * set_size + set_size / 2 + at] = b;
    }
  });
  if (sets > 1) __syncthreads();
  if (set > 0) return;
#pragma unroll 1
  for (int r = 0; r < sets - 1; ++r)
    each([&](float& g, float& b, int at) {
      g += mine[r * set_size + at];
      b += mine[r * set_size + set_size / 2 + at];
    });
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    store_partial<L, VEC>(a.pg + (size_t)blockIdx.x * a.C, c_of(j), a.C, ag[j]);
    store_partial<L, VEC>(a.pb + (size_t)blockIdx.x * a.C, c_of(j), a.C, ab[j]);
  }
}

template <typename T, int NCH, bool VEC>
__global__ void __launch_bounds__(kBwdRingThreads, 1)
    k_layer_norm_bwd_ring(const LnBwd a, const int W, const int rpb, const int depth, unsigned int* err,
                          const unsigned long long limit) {
  pdl_trigger();
  constexpr int SEG = NCH * 256;
  extern __shared__ uint4 ring_smem[];
  __shared__ float red[64];
  __shared__ uint64_t bars[kRingMaxDepth * (kBwdRingThreads / 32)];
  __shared__ int abort_flag;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rib = warp / W, w = warp - rib * W;
  const int seg0 = w * SEG, seg = min(SEG, a.C - seg0);
  RowRing<T, NCH, VEC> ring;
  ring.nt = a.dh ? 3 : 2;
  ring.depth = depth;
  ring.base = reinterpret_cast<T*>(ring_smem) + (size_t)warp * (depth * ring.nt * ring.PITCH);
  ring.bar0 = smem_u32(bars + kRingMaxDepth * warp);
  ring.src[0] = static_cast<const T*>(a.dy);
  ring.src[1] = static_cast<const T*>(a.h);
  ring.src[2] = static_cast<const T*>(a.dh);
  ring.seg0 = seg0;
  ring.C = a.C;
  ring.seg = seg;
  ring.R = a.R;
  ring.step = (long long)gridDim.x * rpb;
  ring.init();
  if (threadIdx.x == 0) abort_flag = 0;
  __syncthreads();
  pdl_wait();
  const long long row0 = (long long)blockIdx.x * rpb + rib;
  ring.start(row0);
  const DropBits bits = drop_bits(a.drop);
  const float inv_n = 1.f / (float)a.C;
  float* my_red = red + rib * 4 * W;
  Chunk<T> gm[NCH];
  if (a.gamma) {
#pragma unroll
    for (int j = 0; j < NCH; ++j) gm[j] = load_chunk<T, 32, VEC>(static_cast<const T*>(a.gamma), seg0 + col0<32, VEC>(j, lane), a.C);
  }
  float2 ag[NCH][4], ab[NCH][4];
#pragma unroll
  for (int j = 0; j < NCH; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) ag[j][i] = ab[j][i] = f2(0.f);
  long long gave_up = row0;
  int slot = 0;
  float next_rstd = row0 < a.R ? a.rstd[row0] : 0.f, next_mean = row0 < a.R ? a.mean[row0] : 0.f;
  for (long long row = row0; row < a.R; row += ring.step, slot ^= 1) {
    const float rstd = next_rstd, mean = next_mean;
    if (row + ring.step < a.R) {
      next_rstd = a.rstd[row + ring.step];
      next_mean = a.mean[row + ring.step];
    }
    const T* in = ring.wait(row, limit, err, &abort_flag);
    if (!ring.failed) gave_up = row + ring.step;
    float2 m1 = f2(0.f), m2 = f2(0.f), xh[NCH][4], t[NCH][4];
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      to_pairs(ring.load(in, 0, j), t[j]);
      to_pairs(ring.load(in, 1, j), xh[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xh[j][i] = mul2(add2(xh[j][i], f2(-mean)), f2(rstd));
        ag[j][i] = fma2(t[j][i], xh[j][i], ag[j][i]);
        ab[j][i] = add2(t[j][i], ab[j][i]);
      }
      if (a.gamma) {
        float2 g[4];
        to_pairs(gm[j], g);
#pragma unroll
        for (int i = 0; i < 4; ++i) t[j][i] = mul2(t[j][i], g[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m1 = add2(m1, t[j][i]);
        m2 = fma2(t[j][i], xh[j][i], m2);
      }
    }
    float m[2] = {m1.x + m1.y, m2.x + m2.y};
    row_sums<32, 2>(m, my_red, slot, w, W, 1 + rib);
    const float2 rs = f2(rstd), c1 = f2(-m[0] * inv_n * rstd), c2 = f2(-m[1] * inv_n * rstd);
    const size_t at = (size_t)row * a.C;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int c0 = seg0 + col0<32, VEC>(j, lane);
#pragma unroll
      for (int i = 0; i < 4; ++i) t[j][i] = fma2(t[j][i], rs, fma2(xh[j][i], c2, c1));
      if (a.dh) {
        float2 d[4];
        to_pairs(ring.load(in, 2, j), d);
#pragma unroll
        for (int i = 0; i < 4; ++i) t[j][i] = add2(t[j][i], d[i]);
      }
      store_chunk<T, 32, VEC>(static_cast<T*>(a.dr) + at, c0, a.C, t[j]);
      if (a.dx) {
        drop_values<32, VEC>(bits, a.drop.scale, row, c0, t[j]);
        store_chunk<T, 32, VEC>(static_cast<T*>(a.dx) + at, c0, a.C, t[j]);
      }
    }
    ring.next(row);
  }
  ring.drain(gave_up, err);
  __syncthreads();
  // The block's partials: the rows' sets of warps in order, the first adding the
  // others' to its own.  Each lane's values lie with its neighbours' (in the order of
  // the columns, eight a lane, they would share banks: 500 rows of 1280 14.6 us, like
  // this 10.0.)
  float* cols = reinterpret_cast<float*>(ring_smem);  // [rpb - 1][2][W][NCH][8][32]
  const int set_size = 2 * W * SEG;
  float* mine = cols + w * SEG + lane;
  auto each = [&](auto f) {
#pragma unroll
    for (int j = 0; j < NCH; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        f(i & 1 ? ag[j][i / 2].y : ag[j][i / 2].x, i & 1 ? ab[j][i / 2].y : ab[j][i / 2].x, (j * 8 + i) * 32);
  };
  if (rib > 0)
    each([&](float& g, float& b, int at) {
      mine[(rib - 1) * set_size + at] = g;
      mine[(rib - 1) * set_size + W * SEG + at] = b;
    });
  __syncthreads();
  if (rib > 0) return;
#pragma unroll 1
  for (int r = 0; r < rpb - 1; ++r)
    each([&](float& g, float& b, int at) {
      g += mine[r * set_size + at];
      b += mine[r * set_size + W * SEG + at];
    });
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    const int c0 = seg0 + col0<32, VEC>(j, lane);
    store_partial<32, VEC>(a.pg + (size_t)blockIdx.x * a.C, c0, a.C, ag[j]);
    store_partial<32, VEC>(a.pb + (size_t)blockIdx.x * a.C, c0, a.C, ab[j]);
  }
}

// As long as a warp has no second row, the partials stay at this many rows.
constexpr long long kFewBlocks = 64;
RingSpread bwd_ring_spread(const LnBwd& a) {
  return ring_spread(a.R, a.C, a.dtype, a.dh ? 3 : 2, kBwdRingThreads, kBwdRingSmem, kFewBlocks);
}
template <typename T, bool VEC> cudaError_t layer_norm_bwd_ring(const LnBwd& a, cudaStream_t st) {
  const RingSpread s = bwd_ring_spread(a);
  auto k = s.nch == 3   ? k_layer_norm_bwd_ring<T, 3, VEC>
           : s.nch == 4 ? k_layer_norm_bwd_ring<T, 4, VEC>
                        : k_layer_norm_bwd_ring<T, 5, VEC>;
  cudaError_t e = allow_smem(k, s.smem, kBwdRingSmem);
  if (e != cudaSuccess) return e;
  return launch_k(k, dim3((unsigned)ln_bwd_rows_blocks(a)), dim3(32 * s.W * s.rpb), s.smem, st, 1, a, s.W, s.rpb, s.depth,
                  device_error_word(), (unsigned long long)kWaitLimitNs);
}
// The longest rows need more warps than share a block's registers.
bool ring_takes(const LnBwd& a) {
  return a.C > 512 && bwd_ring_spread(a).rpb >= 1;
}

template <typename T> constexpr int kBwdRows = sizeof(T) == 2 ? 4 : 2;  // rows of one block at a time
Spread bwd_spread(int C) {
  Spread s;
  const int blocks = (C + 255) / 256;
  s.L = C <= 64 ? 8 : C <= 128 ? 16 : 32;
  s.nch = blocks <= 2 ? blocks : 4;
  s.W = (blocks + s.nch - 1) / s.nch;
  s.rpb = s.W == 1 ? 256 / s.L : s.W < 8 ? 8 / s.W : 1;
  s.threads = s.L * s.W * s.rpb;
  return s;
}
template <typename T, bool VEC> cudaError_t layer_norm_bwd(const LnBwd& a, cudaStream_t st) {
  if (ring_takes(a)) return layer_norm_bwd_ring<T, VEC>(a, st);
  const Spread s = bwd_spread(a.C);
  const int sets = s.L == 32 ? s.rpb : s.threads / 32;
  const size_t smem = (size_t)(sets - 1) * 2 * s.W * s.nch * 8 * s.L * sizeof(float);  // 28 KB at most
  constexpr int RB = kBwdRows<T>;
  auto k = s.L == 8     ? k_layer_norm_bwd<T, 8, 1, RB, VEC, 256>
           : s.L == 16  ? k_layer_norm_bwd<T, 16, 1, RB, VEC, 256>
           : s.nch == 1 ? k_layer_norm_bwd<T, 32, 1, RB, VEC, 256>
           : s.nch == 2 ? k_layer_norm_bwd<T, 32, 2, RB / 2, VEC, 256>
                        : k_layer_norm_bwd<T, 32, 4, 1, VEC, 512>;
  return launch_k(k, dim3((unsigned)ln_bwd_rows_blocks(a)), dim3(s.threads), smem, st, 1, a, s.W, s.rpb);
}

// ---------------------------------------------------------------- parameters
// dgamma and dbeta from the blocks' partials: 32 columns a block, 16 warps each adding
// up every 16th row of partials, then in order.
constexpr int kParamWarps = 16;
template <typename T>
__global__ void __launch_bounds__(32 * kParamWarps) k_layer_norm_params(int P, int C, const float* pg, const float* pb, T* dgamma,
                                                                        T* dbeta) {
  pdl_enter();
  __shared__ float sums[kParamWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  T* out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  const float* p = (blockIdx.y ? pb : pg) + c;
  float s = 0.f;
  if (c < C) {
#pragma unroll 8
    for (int r = warp; r < P; r += kParamWarps) s += p[(size_t)r * C];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp > 0 || c >= C) return;
#pragma unroll
  for (int w = 1; w < kParamWarps; ++w) s += sums[w][lane];
  out[c] = from_f<T>(s);
}

}  // namespace

cudaError_t launch_layer_norm_params(const LnBwd& a, void* dgamma, void* dbeta, cudaStream_t st) {
  RMX_BY_DTYPE(a.dtype, return launch_k(k_layer_norm_params<T>, dim3((a.C + 31) / 32, 2), dim3(32 * kParamWarps), 0, st, 1,
                                        ln_bwd_rows_blocks(a), a.C, (const float*)a.pg, (const float*)a.pb, (T*)dgamma, (T*)dbeta))
}
cudaError_t launch_dropout(long long R, int C, int dtype, const Drop& d, const void* x, const void* r, void* out,
                           cudaStream_t st) {
  RMX_BY_DTYPE(dtype, return dropout_t<T>(R, C, d, x, r, out, st))
}
cudaError_t launch_layer_norm(const LnFwd& a, cudaStream_t st) {
  RMX_BY_DTYPE(a.dtype, return rows_aligned(a.C, sizeof(T)) ? layer_norm<T, true>(a, st) : layer_norm<T, false>(a, st))
}
int ln_bwd_rows_blocks(const LnBwd& a) {
  auto at_most = [](long long want, long long most) {
    if (most > kLnBwdMaxBlocks) most = kLnBwdMaxBlocks;
    return (int)(want < most ? want : most);
  };
  if (ring_takes(a)) {
    const int rpb = bwd_ring_spread(a).rpb;
    return at_most((a.R + rpb - 1) / rpb, sm_count());
  }
  // As many as are resident at once (two an SM, one where the row has 16 warps);
  // few rows: as many as there are.
  const Spread s = bwd_spread(a.C);
  const int rows = s.nch == 4 ? 1 : (a.dtype == 0 ? 2 : 4) / s.nch;  // of a thread at a time
  const long long all = (a.R + s.rpb - 1) / s.rpb;
  if (all > kFewBlocks && a.R <= kFewBlocks * s.rpb * rows) return (int)kFewBlocks;
  return at_most(all, (long long)sm_count() * (s.threads > 256 ? 1 : 2));
}
cudaError_t launch_layer_norm_bwd(const LnBwd& a, cudaStream_t st) {
  RMX_BY_DTYPE(a.dtype,
               return rows_aligned(a.C, sizeof(T)) ? layer_norm_bwd<T, true>(a, st) : layer_norm_bwd<T, false>(a, st))
}

}  // namespace rmx
