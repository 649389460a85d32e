// Matrix products grouped by expert:  out[r] = x[rows[r]] W_e^T  for the rows r of expert e,
// or silu(x W_e^T) * (x U_e^T) with two weight sets.
//
// The weights are the M side of the tcgen05 products and the rows the N side, so that a
// ragged group costs what its rows cost (N in steps of 32) and an expert with few rows is one
// pass over its weights.  Two CTAs of a cluster share a product of M = 256 (cta_group::2): each
// holds 128 rows of weights and half of the rows, and the pair reads both halves.  A tile is
//   256 outputs, or with two weight sets 128 outputs (each CTA: 64 gate and 64 up rows), times
//   up to 256 rows of one expert;
// per 64 columns a CTA copies 16 KB of weights and at most 16 KB of rows for 512 cycles of
// products, which shared memory and L2 can take.  (One CTA with 128 x 128 products moves 112 KB
// through 128 bytes a cycle for the same work.  4096 tokens x top-8 of 128 experts, 2048 -> 768
// with SwiGLU and named rows: 223 us with one, 190 us with two when that was changed; 16384 tokens: 694
// and 560 us.)
// Two accumulators of 256 columns fill tensor memory: a tile's epilogue runs beside the next
// tile's products.
//
// One persistent cluster per two SMs walks the tiles in order of (expert, row tile, weight
// block), so that clusters that run together share rows and, across row tiles, weights in
// L2.  Warp roles of a CTA: producer (weights through a 3-D map whose rows stop at the expert's
// last; rows through a plain map), product issue (the first CTA's), four epilogue warps that
// exchange gate and up and transpose through shared memory to store whole output rows and, when
// `rows` is given, four warps that fetch the named rows with 16-byte asynchronous copies
// straight into the swizzled layout.  (Tensor-map gather copies of four rows at a time were tried
// for that: 566 us against 224 us for rows that lie in order.  So was a prefetch of the weights
// into L2 10 stages ahead of the ring: 154 us against 131 for 8 rows an expert.)
// Accumulation is fp32; the result is rounded once.
//
// Measured in a graph: 4096 tokens as above 177 to 180 us (1.15 PFLOP/s and 4.9 TB/s: both bound it; called back
// to back 190 to 200, the clock falls under the power cap), 128 tokens 123 us (6.6 TB/s), the down products
// (768 -> 2048) of 2 tokens 12.7 us, of which weights stream for 5.5, of 4096 tokens 108 us.
#include "mk_ops.cuh"

namespace mk {
namespace {

constexpr int kExpThreads = 192;     // producer, product issue, four epilogue warps
constexpr int kGatherThreads = 128;  // ... and four gather warps when rows are named
constexpr int kTileW = 128;          // weight rows of a CTA
constexpr int kTileR = 256;          // rows of a tile, half of them in either CTA
constexpr int kTileK = 64;           // columns of a stage: one 128-byte swizzle span
constexpr int kBoxR = 32;            // rows per copy of x (one copy of 128 if more than two would be needed)
constexpr int kBytesW = kTileW * kTileK * 2;
// The ring: a stage has 16 KB of weights and room for 32, 64 or 128 rows, as many as the largest
// expert of the call needs: 9, 8 or 6 stages.  (With 6 throughout, 8 rows an expert: 136 us.)
constexpr int kRingBytes = 6 * (kBytesW + kTileR / 2 * kTileK * 2);
constexpr int kMaxExpStages = 9;
constexpr int kChunk = 32;           // rows of an epilogue step
// per epilogue warp a chunk's results; per pair of warps two buffers of gate / up values in fp32
constexpr int kExpSmem = 1024 + kRingBytes + 4 * kChunk * 32 * 2 + 2 * 2 * kChunk * 32 * 4;
struct ExpTile {
  int e, r0, nr;   // expert, first row, rows (<= 256)
  int w0;          // first output
};

constexpr int kTileNotes = 16;  // more than the ring holds tiles

struct ExpShared {
  uint32_t tmem;
  int abort;
  int most;                     // rows of the largest expert
  int pre[kOpMaxExperts + 1];   // prefix sums of the experts' row tiles
  int2 rows[kOpMaxExperts];     // the experts' rows [x, y)
  int warp_sums[(kExpThreads + kGatherThreads) / 32];
  int rows_of[kTileNotes];      // rows of the tiles under way
  unsigned long long bars[3 * kMaxExpStages + 4];
};

static_assert(kExpSmem + sizeof(ExpShared) <= 232448, "exceeds the 227 KB per-block shared memory limit");

// ---- cluster primitives
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address of the first CTA's copy of a shared variable
__device__ __forceinline__ uint32_t map_leader(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The same for a thread that publishes only shared memory of its CTA (rows that it has seen complete): a
// release of everything costs about 2000 cycles (a whole stage's products take 512), one restricted to
// shared memory does not wait for accesses to global memory.
__device__ __forceinline__ void arrive_cluster_smem(uint32_t bar) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A barrier that the other CTA arrives on is waited for at the scope of the cluster.
// For shared memory: the products' reads of a stage, or the rows and weights of both.
__device__ __forceinline__ bool try_wait_stage(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  if (ok) asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
  return ok != 0;
}
// For the accumulators.
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded waits of one thread and of a whole warp, as op_wait1 and op_wait.
template <bool (*TRY)(uint32_t, uint32_t)>
__device__ __forceinline__ bool wait_pair1(uint32_t bar, uint32_t parity, volatile int* abort, int32_t* status, int tag) {
  if (TRY(bar, parity)) return true;
  const uint64_t t0 = gtime();
  while (!TRY(bar, parity)) {
    if (*abort) return false;
    if ((long long)(gtime() - t0) > kOpWaitNs) {
      *abort = 1;
      op_error(status, MK_ERR_TIMEOUT, (int)blockIdx.x, tag, (int)parity);
      return false;
    }
  }
  return true;
}
template <bool (*TRY)(uint32_t, uint32_t)>
__device__ __forceinline__ bool wait_pair(uint32_t bar, uint32_t parity, volatile int* abort, int32_t* status, int tag) {
  if (__all_sync(0xffffffffu, TRY(bar, parity))) return true;
  const uint64_t t0 = gtime();
  while (!__all_sync(0xffffffffu, TRY(bar, parity))) {
    if (__any_sync(0xffffffffu, *abort != 0)) return false;
    if (__any_sync(0xffffffffu, (long long)(gtime() - t0) > kOpWaitNs)) {
      *abort = 1;
      op_error(status, MK_ERR_TIMEOUT, (int)blockIdx.x, tag, (int)parity);
      return false;
    }
  }
  return true;
}
// copies into this CTA that complete on a barrier of either
__device__ __forceinline__ void tma_pair_2d(uint32_t dst, const CUtensorMap* tm, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_pair_3d(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}
__device__ __forceinline__ void umma_bf16_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc),
               "r"(accumulate ? 1u : 0u)
               : "memory");
}
// arrive on the barrier at this address in both CTAs once the products issued so far have ended
__device__ __forceinline__ void umma_commit_pair(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
               "h"((uint16_t)3)
               : "memory");
}

__device__ __forceinline__ void expert_rows(const ExpertParams& p, int e, int& lo, int& hi) {
  const int a = op_ld(p.a.offsets + e), b = op_ld(p.a.offsets + e + 1);
  lo = min(max(a, 0), p.a.n_rows);
  hi = min(max(b, lo), p.a.n_rows);
  if (blockIdx.x == 0 && (lo != a || hi != b)) op_error(p.a.status, MK_ERR_INVALID, e, a, b);
}

__device__ void scan_experts(const ExpertParams& p, ExpShared& sh) {
  const int E = p.a.n_experts, nt = (int)blockDim.x;
  int carry = 0;
  for (int base = 0; base < E; base += nt) {
    const int e = base + (int)threadIdx.x;
    int x = 0;
    if (e < E) {
      int lo, hi;
      expert_rows(p, e, lo, hi);
      sh.rows[e] = make_int2(lo, hi);
      x = (hi - lo + kTileR - 1) / kTileR;
      if (hi > lo) atomicMax(&sh.most, hi - lo);
    }
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sh.warp_sums[w] = x;
    __syncthreads();
    int add = carry;
    for (int i = 0; i < w; ++i) add += sh.warp_sums[i];
    if (e < E) sh.pre[e + 1] = x + add;
    for (int i = 0; i < nt / 32; ++i) carry += sh.warp_sums[i];
    __syncthreads();
  }
}

// The tile that this cluster takes in turn k (false: none)
__device__ __noinline__ bool find_tile(const ExpertParams& p, const ExpShared& sh, int k, int tiles, int wblocks, int wstep, ExpTile& x) {
  const int t = k * ((int)gridDim.x / 2) + (int)blockIdx.x / 2;
  if (t >= tiles) return false;
  const int rt = t / wblocks;
  int lo = 0;
#pragma unroll
  for (int step = kOpMaxExperts / 2; step > 0; step >>= 1)
    if (lo + step < p.a.n_experts && sh.pre[lo + step] <= rt) lo += step;
  x.e = lo;
  x.w0 = (t - rt * wblocks) * wstep;
  // the expert's rows in equal tiles
  const int2 r = sh.rows[lo];
  const int mine = sh.pre[lo + 1] - sh.pre[lo], per = mine == 1 ? r.y - r.x : (r.y - r.x + mine - 1) / mine;
  x.r0 = r.x + (rt - sh.pre[lo]) * per;
  x.nr = min(per, r.y - x.r0);
  return true;
}

__device__ __forceinline__ float silu(float y) { return __fdividef(y, 1.f + __expf(-y)); }

template <bool GLU>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kExpThreads + kGatherThreads, 1)
    expert_kernel(const __grid_constant__ ExpertParams p, const __grid_constant__ CUtensorMap tx,
                  const __grid_constant__ CUtensorMap tx128, const __grid_constant__ CUtensorMap tw,
                  const __grid_constant__ CUtensorMap tu) {
  extern __shared__ uint8_t raw[];
  __shared__ ExpShared sh;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* const epi_g = raw + (base - smem_u32(raw)) + kRingBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  volatile int* abort = &sh.abort;
  const uint32_t bars = smem_u32(sh.bars);
  auto full = [&](uint32_t s) { return bars + 8 * s; };                            // (used in the first CTA only)
  auto empty = [&](uint32_t s) { return bars + 8 * (kMaxExpStages + s); };
  auto afull = [&](uint32_t a) { return bars + 8 * (2 * kMaxExpStages + a); };        // accumulators written
  auto aempty = [&](uint32_t a) { return bars + 8 * (2 * kMaxExpStages + 2 + a); };   // ... and read by both (first CTA only)
  auto gathered = [&](uint32_t s) { return bars + 8 * (2 * kMaxExpStages + 4 + s); }; // this CTA's named rows

  if (threadIdx.x == 0) {
    sh.abort = sh.pre[0] = sh.most = 0;
    for (int s = 0; s < kMaxExpStages; ++s) {
      mbar_init(full(s), p.a.rows ? 2 : 1);  // the copies; the second CTA's named rows
      mbar_init(empty(s), 1);
      mbar_init(gathered(s), kGatherThreads);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(afull(a), 1);
      mbar_init(aempty(a), 2 * 4);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane < 4) {
    const CUtensorMap* tm = lane == 0 ? &tx : lane == 1 ? &tx128 : lane == 2 ? &tw : &tu;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tm)) : "memory");
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(&sh.tmem), 512);
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // the barriers of both CTAs are there
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  scan_experts(p, sh);
  const uint32_t tmem = uniform(sh.tmem);
  constexpr int kStep = GLU ? kTileW : 2 * kTileW;
  const int wblocks = (p.a.n + kStep - 1) / kStep;
  const int tiles = (int)uniform(sh.pre[p.a.n_experts]) * wblocks;  // (below 2^31: checked by the host)
  const int ksteps = (p.a.k + kTileK - 1) / kTileK;
  const uint32_t most = uniform(min(sh.most, kTileR)), room = most <= 64 ? 32 : most <= 128 ? 64 : 128;  // rows of a stage
  const uint32_t stage_bytes = kBytesW + room * kTileK * 2, stages = room == 32 ? 9 : room == 64 ? 8 : 6;
  auto tile = [&](int k, ExpTile& x) -> bool { return uniform(find_tile(p, sh, k, tiles, wblocks, kStep, x)); };
  auto tile1 = [&](int k, ExpTile& x) -> bool { return find_tile(p, sh, k, tiles, wblocks, kStep, x); };  // (one thread)
  const int clusters = (int)gridDim.x / 2, mine = (tiles - (int)blockIdx.x / 2 + clusters - 1) / clusters;  // tiles of this cluster
  ExpTile x;

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (elect_one()) {
      Ring at;
      bool ok = true;
      const int half = GLU ? kTileW / 2 : kTileW;  // weight rows per copy
      const uint32_t lead = map_leader(bars);
      // (the next tile is looked up while this one's stages are under way)
      bool more = tile1(0, x);
      for (int t = 0; ok && more; ++t) {
        const int e = x.e, n2 = (x.nr + 31) / 32 * 16;  // rows of this CTA
        const int w = x.w0 + (int)rank * half, r = x.r0 + (int)rank * n2;
        const uint32_t xrows = p.a.rows ? 0 : n2 <= kBoxR ? kBoxR : n2 <= 2 * kBoxR ? 2 * kBoxR : kTileR / 2;
        const uint32_t bytes = 2 * (kBytesW + xrows * (kTileK * 2));  // of both CTAs
        sh.rows_of[t % kTileNotes] = x.nr;  // for the products, which wait for these copies
        for (int ks = 0; ks < ksteps; ++ks, at.advance(stages)) {
          const uint32_t s = at.slot;
          if (!(ok = wait_pair1<try_wait_stage>(empty(s), at.phase ^ 1, abort, p.a.status, 1))) break;
          const uint32_t st = base + s * stage_bytes, bar = lead + 8 * s;
          if (rank == 0) mbar_expect_tx(full(s), bytes);
          tma_pair_3d(st, &tw, ks * kTileK, w, e, bar);
          if (GLU) tma_pair_3d(st + kBytesW / 2, &tu, ks * kTileK, w, e, bar);
          if (xrows == kTileR / 2) {
            tma_pair_2d(st + kBytesW, &tx128, ks * kTileK, r, bar);
          } else if (xrows) {
            tma_pair_2d(st + kBytesW, &tx, ks * kTileK, r, bar);
            if (xrows > kBoxR) tma_pair_2d(st + kBytesW + kBoxR * kTileK * 2, &tx, ks * kTileK, r + kBoxR, bar);
          }
          if (ks == 0) more = tile1(t + 1, x);
        }
      }
    }
    __syncwarp();
    // an abandoned run leaves copies in flight: give them time to land
    if (*abort) {
      const uint64_t s0 = gtime();
      while ((long long)(gtime() - s0) < 10000000ll) {}
    }
  } else if (warp >= kExpThreads / 32) {
    // ---------------------------------------------------------------- gather
    // eight threads a row (128 bytes of a stage), 16 rows at a time; the copies report themselves
    const int t128 = (int)threadIdx.x - kExpThreads, chunk = t128 & 7, row0 = t128 >> 3;
    const uint32_t swz = (uint32_t)(chunk ^ (row0 & 7)) * 16;  // (16 j keeps the low three bits of the row)
    constexpr int kRows = kTileR / 2 / 16;
    Ring at;
    bool ok = true;
    // A tile's row numbers are read a tile ahead: the ring covers 2600 cycles, less than the numbers and
    // the first rows take one after the other (4096 tokens: 193 us, 2000 to 7000 cycles of every 21000 lost).
    int first, count, names[kRows];
    auto look_up = [&](int t) -> bool {
      if (!tile(t, x)) return false;
      const int n2 = (x.nr + 31) / 32 * 16;
      first = x.r0 + (int)rank * n2;
      count = min(n2, x.nr - (int)rank * n2);  // (may be < 0)
#pragma unroll
      for (int j = 0; j < kRows; ++j) names[j] = row0 + 16 * j < count ? op_ld(p.a.rows + first + row0 + 16 * j) : 0;
      return true;
    };
    bool more = look_up(0);
    for (int t = 0; ok && more; ++t) {
      const uint16_t* src[kRows];
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const int r = min(max(names[j], 0), p.a.n_x - 1);
        if (r != names[j] && x.w0 == 0) op_error(p.a.status, MK_ERR_INVALID, x.e, first + row0 + 16 * j, names[j]);
        src[j] = static_cast<const uint16_t*>(p.a.x) + r * p.a.x_stride + 8 * chunk;
      }
      const int rows_now = count;
      for (int ks = 0; ks < ksteps; ++ks, at.advance(stages)) {
        if (!(ok = wait_pair<try_wait_stage>(empty(at.slot), at.phase ^ 1, abort, p.a.status, 6))) break;
        const uint32_t dst = base + at.slot * stage_bytes + kBytesW + row0 * (kTileK * 2) + swz;
        const int bytes = ks * kTileK + 8 * chunk < p.a.k ? 16 : 0;  // (0: zeros)
#pragma unroll
        for (int j = 0; j < kRows; ++j)
          if (row0 + 16 * j < rows_now) op_cp16(dst + j * 16 * kTileK * 2, bytes ? src[j] + ks * kTileK : src[j], bytes);
        op_cp_arrive(gathered(at.slot));
        if (ks == 0) more = look_up(t + 1);
      }
    }
    op_cp_wait_all();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- product issue (first CTA)
    if (rank != 0) {
      // This thread reports the second CTA's gathered stages, made visible to the products.
      if (p.a.rows && elect_one()) {
        Ring at;
        bool ok = true;
        for (int t = 0; ok && t < mine; ++t)
          for (int ks = 0; ks < ksteps; ++ks, at.advance(stages)) {
            if (!(ok = op_wait1(gathered(at.slot), at.phase, abort, p.a.status, 7))) break;
            fence_proxy_async_smem();
            arrive_cluster_smem(map_leader(full(at.slot)));
          }
      }
    } else if (elect_one()) {
      uint32_t nt = 0;
      Ring at;
      const uint64_t d0 = umma_sdesc_sw(base, 16, 1024, 128);  // stage 0: weights, rows
      bool ok = true;
      for (; ok && (int)nt < mine; ++nt) {
        uint32_t idesc = 0;
        const uint32_t a = nt & 1, acc = tmem + kTileR * a;
        if (!(ok = wait_pair1<try_wait_cluster>(aempty(a), ((nt >> 1) & 1) ^ 1, abort, p.a.status, 2))) break;
        for (int ks = 0; ks < ksteps; ++ks, at.advance(stages)) {
          if (!(ok = wait_pair1<try_wait_stage>(full(at.slot), at.phase, abort, p.a.status, 3))) break;
          if (p.a.rows) {
            if (!(ok = op_wait1(gathered(at.slot), at.phase, abort, p.a.status, 8))) break;
            fence_proxy_async_smem();
          }
          tc_fence_after();
          if (ks == 0) idesc = umma_idesc_bf16(2 * kTileW, (*(volatile int*)&sh.rows_of[nt % kTileNotes] + 31) / 32 * 32);
          const uint64_t d = d0 + at.slot * (stage_bytes / 16);
#pragma unroll
          for (int kk = 0; kk < kTileK / 16; ++kk)
            umma_bf16_pair(acc, d + 2 * kk, d + kBytesW / 16 + 2 * kk, idesc, ks > 0 || kk > 0);
          umma_commit_pair(empty(at.slot));
        }
        if (ok) umma_commit_pair(afull(a));
      }
    }
    __syncwarp();
    if (*abort) {  // let the products in flight end before the memory goes
      const uint64_t s0 = gtime();
      while ((long long)(gtime() - s0) < 10000000ll) {}
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    // A warp has 32 weight rows (lanes) and takes 32 rows of x at a time; it turns its piece of the
    // result in shared memory of its own and stores 64 bytes of every row.  With two weight sets
    // warps 0 and 1 have gate rows and warps 2 and 3 the up rows of the same outputs: each side of
    // a pair gets the other's values for half of the rows.  (A wait that gives up is not followed
    // by an exit: the pair keeps meeting, and every later wait returns at once.)
    const int q = warp & 3;               // lanes 32 q .. of tensor memory
    uint32_t nt = 0, nc = 0;
    constexpr int kTake = GLU ? kChunk / 2 : kChunk;  // rows that this warp stores of a chunk
    const bool up = GLU && q >= 2;
    const int o = GLU ? 32 * (q & 1) : 32 * q;        // first output of this warp in the CTA's
    // whole 16-byte pieces of an output row where its address allows them
    const bool wide = p.a.n % 8 == 0 && p.a.out_stride % 8 == 0 && (reinterpret_cast<uintptr_t>(p.a.out) & 15) == 0;
    uint16_t* const stage = reinterpret_cast<uint16_t*>(epi_g) + q * kChunk * 32;
    float* const exch_g = reinterpret_cast<float*>(epi_g + 4 * kChunk * 32 * 2) + (q & 1) * kChunk * 32;
    for (int t = 0; tile(t, x); ++t, ++nt) {
      const uint32_t a = nt & 1;
      const uint32_t acc = tmem + kTileR * a + ((uint32_t)q << 21);
      const int w0 = x.w0 + (int)rank * (GLU ? kTileW / 2 : kTileW) + o, width = min(32, p.a.n - w0);  // (<= 0: nothing to store)
      wait_pair<try_wait_cluster>(afull(a), (nt >> 1) & 1, abort, p.a.status, 4);
      tc_fence_after();
      uint32_t u[kChunk];
      tmem_ld32(acc, u);
#pragma unroll 1
      for (int c = 0; c < x.nr; c += kChunk, ++nc) {
        float v[kTake];
        tmem_wait32(u);
        if (GLU) {
          float* const exch = exch_g + (nc & 1) * 2 * kChunk * 32;
          // [row][lane]: the first 16 rows from the up warp to the gate warp, the others the other way
#pragma unroll
          for (int i = 0; i < 16; ++i) exch[((up ? 0 : 16) + i) * 32 + lane] = __uint_as_float(up ? u[i] : u[16 + i]);
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(up ? u[16 + i] : u[i]);
        } else {
#pragma unroll
          for (int i = 0; i < kTake; ++i) v[i] = __uint_as_float(u[i]);
        }
        const bool last = c + kChunk >= x.nr;
        if (last) {  // read: the next products may overwrite it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(map_leader(aempty(a)));
        } else {
          tmem_ld32(acc + c + kChunk, u);
        }
        if (GLU) {
          asm volatile("bar.sync %0, 64;" ::"r"(1 + (q & 1)) : "memory");
          const float* const exch = exch_g + (nc & 1) * 2 * kChunk * 32;
#pragma unroll
          for (int i = 0; i < kTake; ++i) {
            const float y = exch[((up ? 16 : 0) + i) * 32 + lane];
            v[i] = up ? silu(y) * v[i] : silu(v[i]) * y;
          }
        }
#pragma unroll
        for (int i = 0; i < kTake; ++i) stage[i * 32 + lane] = to_bf16(v[i]);
        __syncwarp();
        const int r0 = c + (up ? kTake : 0), rows = min(kTake, x.nr - r0);
        uint16_t* const out = static_cast<uint16_t*>(p.a.out) + (x.r0 + r0) * p.a.out_stride + w0;
        if (wide) {
          if (8 * (lane & 3) < width)
            for (int r = lane >> 2; r < rows; r += 8)
              *reinterpret_cast<uint4*>(out + r * p.a.out_stride + 8 * (lane & 3)) =
                  *reinterpret_cast<const uint4*>(stage + r * 32 + 8 * (lane & 3));
        } else if (lane < width) {
          for (int r = 0; r < rows; ++r) out[r * p.a.out_stride + lane] = stage[r * 32 + lane];
        }
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the other may signal it or read its half
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <bool GLU>
cudaError_t launch_glu(const ExpertParams& p, const CUtensorMap& tx, const CUtensorMap& tx128, const CUtensorMap& tw,
                       const CUtensorMap& tu, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(expert_kernel<GLU>, kExpSmem, done);
  if (e != cudaSuccess) return e;
  return launch_early(expert_kernel<GLU>, dim3((unsigned)(p.grid / 2 * 2)), kExpThreads + (p.a.rows ? kGatherThreads : 0), kExpSmem, st,
                      p, tx, tx128, tw, tu);
}

}  // namespace

cudaError_t launch_experts(const ExpertParams& p, const CUtensorMap& tx, const CUtensorMap& tx128, const CUtensorMap& tw,
                           const CUtensorMap& tu, cudaStream_t st) {
  return p.a.w_up ? launch_glu<true>(p, tx, tx128, tw, tu, st) : launch_glu<false>(p, tx, tx128, tw, tu, st);
}

}  // namespace mk
