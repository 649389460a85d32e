// Products of few rows:  out = act(x W^T + bias) + residual  where the tiles of mk_experts.cu would leave most SMs idle.
//
// A tile is 128 outputs (the M side of the tcgen05 products) by up to 128 rows of x (the N side, in steps of 16); its k is cut
// into as many slices as there are SMs for, and a cluster has a tile, a CTA a slice.  Reading the weights bounds it (all of them
// once, from every SM), and below that a chain: launch, the first copies, products, the slices' sums.  The slices meet in shared
// memory: each CTA owns a part of the tile's rows, gets every other CTA's sums for them, adds them in the order of the slices and
// writes its part with the epilogue: nothing but results goes to memory, and equal calls give equal bits.
//
// Measured in a graph: 5 rows, 1024 -> 1536 3.3 us, 128 rows, 4096 -> 2048 with a residual 7.8 us (of them weights stream for 2.5, at 7
// TB/s; 0.6 until the first are there, 0.4 for the last products and reading the sums, 0.7 the exchange, ~1 the epilogue, the rest
// launch, setup and the end); 4096 -> 2048 without: 1 row 5.8 us, 64 7.3, 256 11.0, 512 15.1, 1024 20.8, the last two in one slice: the tiles'
// copies out of L2 bound them, 13 TB/s (with a quarter of the products 2 to 7 % less).
#include <algorithm>

#include "mk_linear.cuh"

namespace mk {
namespace {

constexpr int kSplitThreads = 192;  // producer, product issue, four epilogue warps
constexpr int kSplitW = 128;        // outputs of a tile
constexpr int kSplitRows = 128;     // ... and rows at most
constexpr int kSplitK = 64;         // columns of a stage: one 128-byte swizzle span
constexpr int kSplitStages = 12;
constexpr int kSplitBytesW = kSplitW * kSplitK * 2;
// Stages of an accumulator of float32 results.  The products drop what lies below its last bit, so that a sum is off by more the longer it
// is (2-norm: 512 columns 4.7e-7, 2048 2.1e-6, 16384 1.9e-5): sums of 512 columns are added up in registers, from two accumulators in
// turn.  A kernel of its own (LONG), which it slows down (float32, 4096 -> 2048: 64 rows 7.3 -> 7.7 us, 128 8.2 ->
// 8.7, 512 15.1 -> 17.3, 1024 20.8 -> 21.5; with the sums in shared memory the same to 1 %).
constexpr int kSegment = 8;
constexpr int kAccCols = 128;  // from one to the other

struct SplitShared {
  uint32_t tmem;
  int abort;
  unsigned long long bars[2 * kSplitStages + 5];
};
constexpr int kSplitSmem = 232448 - 1024;  // (SplitShared fits the rest)

__device__ __forceinline__ uint32_t split_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void split_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// No CTA leaves before its copies have arrived: each says when it has got its own.  (A release behind the last stores, and waited for,
// was 1.7 of 8.5 us at 128 rows, 4096 -> 2048.)
__device__ __forceinline__ void split_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void split_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* tm, int x, int y, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar)
               : "memory");
}

template <bool WIDE, bool LONG>
__global__ void __launch_bounds__(kSplitThreads, 1)
    split_kernel(const __grid_constant__ SplitParams p, const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw) {
  extern __shared__ uint8_t raw[];
  __shared__ SplitShared sh;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = split_rank();
  const int tile = (int)blockIdx.x / p.slices, wt = tile % p.w_tiles, rt = tile / p.w_tiles;
  const int w0 = wt * kSplitW, r0 = rt * p.rows, rows = min(p.rows, p.m - r0);
  const int k0 = (int)((long long)rank * p.chunks / p.slices), k1 = (int)((long long)(rank + 1) * p.chunks / p.slices);
  const uint32_t stage_bytes = kSplitBytesW + p.box * kSplitK * 2, stages = p.stages;
  const uint32_t sums = base + p.ring;  // [slice][owned row][kSplitW]
  float* const sums_g = reinterpret_cast<float*>(raw + (sums - smem_u32(raw)));
  const int own = (p.box + p.slices - 1) / p.slices;  // rows that a CTA owns of the tile
  const uint32_t bars = smem_u32(sh.bars), got = bars + 8 * 2 * kSplitStages;
  const uint32_t part = own * kSplitW * 4;  // bytes of a slice's sums for a CTA
  auto full = [&](uint32_t s) { return bars + 8 * s; };
  auto empty = [&](uint32_t s) { return bars + 8 * (kSplitStages + s); };
  auto done = [&](uint32_t a) { return got + 8 + 8 * a; };    // an accumulator is whole
  auto taken = [&](uint32_t a) { return got + 24 + 8 * a; };  // ... and has been read

  if (threadIdx.x == 0) {
    sh.abort = 0;
    for (uint32_t s = 0; s < stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(done(a), 1);
      mbar_init(taken(a), 4);
    }
    mbar_init(got, 1);
    mbar_expect_tx(got, p.slices * part);
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane < 2) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(lane ? &tx : &tw)) : "memory");
  if (warp == 1) tmem_alloc(smem_u32(&sh.tmem), p.tmem_cols);
  __syncwarp();
  tc_fence_before();
  split_sync();  // all CTAs have started: their shared memory may be written
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = uniform(sh.tmem);
  volatile int* const abort = &sh.abort;

  if (warp == 0) {
    if (elect_one()) {
      Ring at;
      for (int k = k0; k < k1; ++k, at.advance(stages)) {
        if (!op_wait1(empty(at.slot), at.phase ^ 1, abort, p.status, 1)) break;
        const uint32_t st = base + at.slot * stage_bytes;
        mbar_expect_tx(full(at.slot), stage_bytes);
        tma_tile(st, &tw, k * kSplitK, w0, full(at.slot));
        tma_tile(st + kSplitBytesW, &tx, k * kSplitK, r0, full(at.slot));
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      Ring at;
      bool ok = true;
      const uint32_t idesc = umma_idesc_bf16(kSplitW, p.box);
      const uint64_t d0 = umma_sdesc_sw(base, 16, 1024, 128);
      for (int k = k0; ok && k < k1; ++k, at.advance(stages)) {
        const uint32_t n = LONG ? (uint32_t)(k - k0) / kSegment : 0;  // accumulators before this one
        const bool first = k == k0 || (LONG && (k - k0) % kSegment == 0);
        if (LONG && first && k > k0) {
          umma_commit(done((n - 1) & 1));
          if (!(ok = op_wait1(taken(n & 1), (n >> 1 & 1) ^ 1, abort, p.status, 5))) break;
        }
        if (!(ok = op_wait1(full(at.slot), at.phase, abort, p.status, 2))) break;
        tc_fence_after();
        const uint64_t d = d0 + at.slot * (stage_bytes / 16);
#pragma unroll
        for (int kk = 0; kk < kSplitK / 16; ++kk)
          umma_bf16(tmem + (n & 1) * kAccCols, d + 2 * kk, d + kSplitBytesW / 16 + 2 * kk, idesc, !first || kk > 0);
        umma_commit(empty(at.slot));
      }
      if (ok) umma_commit(done(LONG ? (uint32_t)(k1 - 1 - k0) / kSegment & 1 : 0));
    }
    __syncwarp();
  } else {
    // this slice's sums, in order of the rows, then a copy to each CTA of what it owns: a lane has an output, a column of tensor
    // memory is a row of x.  (The ring is free: its products have ended.  Stores of single values into the other CTAs took 6 us for
    // 128 rows by 8 slices.)
    const int q = warp & 3;
    float* const mine = reinterpret_cast<float*>(raw + ((p.slices > 1 ? base : sums) - smem_u32(raw))) + 32 * q + lane;
    if (LONG) {
      constexpr int kParts = kSplitRows / 16;
      float sum[kParts][16];
#pragma unroll
      for (int c = 0; c < kParts; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[c][i] = 0.f;
      const int segments = (k1 - k0 + kSegment - 1) / kSegment;
#pragma unroll 1
      for (int s = 0; s < segments; ++s) {
        op_wait(done(s & 1), s >> 1 & 1, abort, p.status, 3);
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kParts; ++c)
          if (16 * c < rows) {
            uint32_t u[16];
            tmem_ld16(tmem + (s & 1) * kAccCols + 16 * c + ((uint32_t)q << 21), u);
            tmem_wait16(u);
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[c][i] += __uint_as_float(u[i]);
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && s + 2 < segments) mbar_arrive(taken(s & 1));
      }
#pragma unroll
      for (int c = 0; c < kParts; ++c)
        if (16 * c < rows) {
#pragma unroll
          for (int i = 0; i < 16; ++i) mine[(16 * c + i) * kSplitW] = sum[c][i];
        }
    } else {
      op_wait(done(0), 0, abort, p.status, 3);
      tc_fence_after();
      for (int c = 0; c < rows; c += 16) {
        uint32_t u[16];
        tmem_ld16(tmem + c + ((uint32_t)q << 21), u);
        tmem_wait16(u);
#pragma unroll
        for (int i = 0; i < 16; ++i) mine[(c + i) * kSplitW] = __uint_as_float(u[i]);
      }
    }
    fence_proxy_async_smem();
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (warp == 2 && lane < p.slices && p.slices > 1) {
      uint32_t to, bar;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(sums + rank * part), "r"(lane));
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(got), "r"(lane));
      asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
                   "r"(base + lane * part), "r"(part), "r"(bar)
                   : "memory");
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  // a warp takes a row at a time, a lane four outputs; what it adds is on its way before the sums are there
  const int col = 4 * lane, width = min(kSplitW, p.n - w0), last = min(own, rows - (int)rank * own);
  const long long row0 = r0 + (long long)rank * own;
  float b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = p.epi.bias && col + i < width ? bf16_to_f(op_ld2(p.epi.bias + w0 + col + i)) : 0.f;
  uint2 ahead = warp < last ? linear_residual(p.epi, row0 + warp, w0 + col, width - col) : make_uint2(0, 0);
  if (p.slices > 1) op_wait(got, 0, abort, p.status, 4);
  if (*abort) {  // an abandoned run leaves copies and products in flight: give them time to end
    const uint64_t t0 = gtime();
    while ((long long)(gtime() - t0) < 10000000ll) {}
  }
  __syncwarp();
  split_arrive();
  for (int r = warp; r < last; r += kSplitThreads / 32) {
    const int then = r + kSplitThreads / 32;
    const uint2 next = then < last ? linear_residual(p.epi, row0 + then, w0 + col, width - col) : make_uint2(0, 0);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    float4 y = *reinterpret_cast<const float4*>(sums_g + r * kSplitW + col);
    v[0] = y.x, v[1] = y.y, v[2] = y.z, v[3] = y.w;
    for (int s = 1; s < p.slices; ++s) {
      y = *reinterpret_cast<const float4*>(sums_g + (s * own + r) * kSplitW + col);
      v[0] += y.x, v[1] += y.y, v[2] += y.z, v[3] += y.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += b[i];
    linear_acts<WIDE>(v, p.epi.act);
    linear_put<WIDE>(p.epi, p.out, p.out_stride, v, ahead, row0 + r, w0 + col, width - col);
    ahead = next;
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
  split_wait();
}

}  // namespace

// Whether the tiles of 256 outputs by 256 rows, a pair of SMs each, would leave more than half of the pairs without one; if so the
// split of the work.  (us of this / of the pairs, 4096 -> 2048: 1 row 5.8 / 15.0, 128 8.2 / 15.4, 256 11.0 / 15.4, 512 15.1 / 16.2, 768
// 20.3 / 17.3, 1024 20.8 / 17.9; 2048 -> 4096: 128 8.8 / 9.8, 256 10.3 / 10.4, 512 14.3 / 11.7; 1024 -> 1024: 128 4.9 / 6.5, 512
// 7.0 / 6.7, 1024 7.6 / 7.4.  The rule gives up to a fifth away above 256 to 600 rows, where pairs have tiles of 64 to 128 rows.)
cudaError_t split_shape(SplitParams& p, int sms, bool* fits) {
  const long long pairs = (long long)((p.n + 255) / 256) * ((p.m + 255) / 256);
  *fits = p.m <= 1024 && pairs * 4 <= sms;
  if (!*fits) return cudaSuccess;
  // 64 rows a tile while every tile has an SM, else 128: of twice as many rows a CTA hands on twice the sums (128 rows, 4096 -> 2048:
  // 11.2 us with 128, 9.0 with 64; 1024 rows 21 and 32)
  p.w_tiles = (p.n + kSplitW - 1) / kSplitW;
  const int most = (p.m + 63) / 64 * p.w_tiles <= sms ? 64 : kSplitRows, r_tiles = (p.m + most - 1) / most;
  p.rows = ((p.m + r_tiles - 1) / r_tiles + 15) / 16 * 16;
  p.box = p.rows;
  p.r_tiles = (p.m + p.rows - 1) / p.rows;
  p.chunks = (p.k + kSplitK - 1) / kSplitK;
  // as many slices as keep all clusters on the GPU at once (16 tiles in 8 slices: 18 us, 15 clusters of 8 fit; in 6: 10.4, at 128 rows a tile)
  static std::atomic<unsigned long long> done{0}, done_wide{0}, done_long{0};
  cudaError_t e = allow_smem(split_kernel<false, false>, kSplitSmem, done);
  if (e == cudaSuccess) e = allow_smem(split_kernel<true, false>, kSplitSmem, done_wide);
  if (e == cudaSuccess) e = allow_smem(split_kernel<true, true>, kSplitSmem, done_long);
  static std::atomic<int> known[8][64];
  for (p.slices = std::min(8, p.chunks); e == cudaSuccess && p.slices > 1; --p.slices) {
    int n = 0;
    e = active_clusters(split_kernel<false, false>, p.slices, kSplitThreads, kSplitSmem, known[p.slices - 1], &n);
    if (p.w_tiles * p.r_tiles <= n) break;
  }
  const int own = (p.box + p.slices - 1) / p.slices, sums = p.slices * own * kSplitW * 4, stage = kSplitBytesW + p.box * kSplitK * 2;
  const int per = (p.chunks + p.slices - 1) / p.slices;
  p.long_sums = p.epi.out_float && per > kSegment;
  p.tmem_cols = p.long_sums ? 2 * kAccCols : 32;
  while (p.tmem_cols < p.box) p.tmem_cols *= 2;
  p.stages = std::min({kSplitStages, per, (kSplitSmem - 1024 - sums) / stage});
  p.ring = std::max(p.stages * stage, p.slices > 1 ? sums : 0);  // (the sums leave from where the stages were)
  p.smem = 1024 + p.ring + sums;
  return e;
}

cudaError_t launch_linear_split(const SplitParams& p, const CUtensorMap& tx, const CUtensorMap& tw, cudaStream_t st) {
  const dim3 grid((unsigned)(p.w_tiles * p.r_tiles * p.slices));
  const auto launch = [&](auto* kernel) { return launch_clusters(kernel, grid, p.slices, kSplitThreads, (size_t)p.smem, st, p, tx, tw); };
  return p.long_sums ? launch(split_kernel<true, true>) : p.epi.out_float ? launch(split_kernel<true, false>) : launch(split_kernel<false, false>);
}

}  // namespace mk
