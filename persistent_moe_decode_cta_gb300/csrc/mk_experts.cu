// Matrix products grouped by expert:  out[r] = x[rows[r]] W_e^T  for the rows r of expert e,
// or silu(x W_e^T) * (x U_e^T) with two weight sets.
//
// The weights are the M side of the tcgen05 products and the rows the N side: a tile is two
// blocks of 128 weight rows (the gate and the up rows of the same 128 outputs, or 256
// outputs of a single product) times up to 128 rows of one expert.  So a ragged group costs
// what its rows cost (N in steps of 16), an expert with few rows is one pass over its
// weights, and gate and up of an output meet in the same thread of the epilogue.  Two
// accumulators of 128 columns, double buffered, fill tensor memory: a tile's epilogue
// runs beside the next tile's products.
//
// One persistent CTA per SM walks the tiles in order of (expert, row tile, weight block), so
// that CTAs that run together share rows and, across row tiles, weights in L2.  Warp roles:
// producer (weights through a 3-D map whose rows stop at the expert's last; rows through a
// plain map), MMA issue, four epilogue warps that transpose through shared memory to store
// whole output rows and, when `rows` is given, four warps that fetch the named rows with
// 16-byte asynchronous copies straight into the swizzled layout.  (Tensor-map gather copies
// of four rows at a time were tried for that: 566 us against 224 us for rows that lie in
// order, 4096 tokens x top-8 of 128 experts, 2048 -> 768 with SwiGLU.)
// Accumulation is fp32; the result is rounded once.
#include "mk_ops.cuh"

namespace mk {
namespace {

constexpr int kExpThreads = 192;   // producer, MMA, four epilogue warps
constexpr int kGatherThreads = 128;  // ... and four gather warps when rows are named
constexpr int kGatherLag = 2;      // stages whose copies a gather thread has in flight beside the newest
constexpr int kTileW = 128;        // weight rows of a block
constexpr int kTileR = 128;        // rows of a tile
constexpr int kTileK = 64;         // columns of a stage: one 128-byte swizzle span
constexpr int kBoxR = 32;          // rows per copy of x (one copy of 128 if more than two would be needed)
constexpr int kExpStages = 4;
constexpr int kBytesW = kTileW * kTileK * 2, kBytesR = kTileR * kTileK * 2;
constexpr int kExpStage = 2 * kBytesW + kBytesR;
constexpr int kExpOut = kTileR * kTileW * 2;  // a block's results, row by row
constexpr int kExpSmem = 1024 + kExpStages * kExpStage + kExpOut;

struct ExpTile {
  int e, r0, nr;   // expert, first row, rows (<= 128)
  int w0;          // first weight row
};

struct ExpShared {
  uint32_t tmem;
  int abort;
  int pre[kOpMaxExperts + 1];   // prefix sums of the experts' row tiles
  int warp_sums[(kExpThreads + kGatherThreads) / 32];
  unsigned long long bars[2 * kExpStages + 5];
};

__device__ __forceinline__ void expert_rows(const ExpertParams& p, int e, bool record, int& lo, int& hi) {
  const int a = __ldg(p.a.offsets + e), b = __ldg(p.a.offsets + e + 1);
  lo = min(max(a, 0), p.a.n_rows);
  hi = min(max(b, lo), p.a.n_rows);
  if (record && (lo != a || hi != b)) op_error(p.a.status, MK_ERR_INVALID, e, a, b);
}

__device__ void scan_experts(const ExpertParams& p, ExpShared& sh) {
  const int E = p.a.n_experts, nt = (int)blockDim.x;
  if (threadIdx.x == 0) sh.pre[0] = 0;
  int carry = 0;
  for (int base = 0; base < E; base += nt) {
    const int e = base + (int)threadIdx.x;
    int x = 0;
    if (e < E) {
      int lo, hi;
      expert_rows(p, e, blockIdx.x == 0, lo, hi);
      x = (hi - lo + kTileR - 1) / kTileR;
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

__device__ __forceinline__ ExpTile find_tile(const ExpertParams& p, const int* pre, int t, int wblocks, int wstep) {
  ExpTile x;
  const int rt = t / wblocks;
  int lo = 0, hi = p.a.n_experts - 1;
  while (lo < hi) {
    const int m = (lo + hi + 1) >> 1;
    if (pre[m] <= rt) lo = m; else hi = m - 1;
  }
  x.e = lo;
  x.w0 = (t - rt * wblocks) * wstep;
  int a, b;
  expert_rows(p, lo, false, a, b);
  x.r0 = a + (rt - pre[lo]) * kTileR;
  x.nr = min(kTileR, b - x.r0);
  return x;
}

__device__ __forceinline__ float silu(float y) { return y / (1.f + __expf(-y)); }

template <bool GLU>
__global__ void __launch_bounds__(kExpThreads + kGatherThreads, 1)
    expert_kernel(const __grid_constant__ ExpertParams p, const __grid_constant__ CUtensorMap tx,
                  const __grid_constant__ CUtensorMap tx128, const __grid_constant__ CUtensorMap tw,
                  const __grid_constant__ CUtensorMap tu) {
  extern __shared__ uint8_t raw[];
  __shared__ ExpShared sh;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t* const out_g = raw + (base - smem_u32(raw)) + kExpStages * kExpStage;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &sh.abort;
  const uint32_t bars = smem_u32(sh.bars);
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (kExpStages + s); };
  auto afull = [&](int a) { return bars + 8 * (2 * kExpStages + a); };      // accumulators written
  auto aempty = [&](int a) { return bars + 8 * (2 * kExpStages + 2 + a); };  // ... and read
  const uint32_t emeet = bars + 8 * (2 * kExpStages + 4);                    // the epilogue warps meet

  if (threadIdx.x == 0) {
    sh.abort = 0;
    for (int s = 0; s < kExpStages; ++s) {
      mbar_init(full(s), p.a.rows ? 1 + kGatherThreads : 1);
      mbar_init(empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(afull(a), 1);
      mbar_init(aempty(a), 128);
    }
    mbar_init(emeet, 128);
    fence_proxy_async_smem();
  }
  scan_experts(p, sh);
  constexpr int kStep = GLU ? kTileW : 2 * kTileW;
  const int wblocks = (p.a.n + kStep - 1) / kStep;
  const int tiles = (int)uniform(sh.pre[p.a.n_experts]) * wblocks;  // (below 2^31: checked by the host)
  if ((int)blockIdx.x >= tiles) return;  // (the whole CTA)
  if (warp == 1) tmem_alloc(smem_u32(&sh.tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int ksteps = (p.a.k + kTileK - 1) / kTileK;

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    uint32_t fill = 0;
    bool ok = true;
    for (int t = (int)blockIdx.x; ok && t < tiles; t += (int)gridDim.x) {
      const ExpTile x = find_tile(p, sh.pre, t, wblocks, kStep);
      const bool second = GLU || uniform(x.w0 + kTileW < p.a.n);
      const int e = (int)uniform(x.e), w0 = (int)uniform(x.w0), r0 = (int)uniform(x.r0), nr = (int)uniform(x.nr);
      const uint32_t xrows = p.a.rows ? 0 : nr <= kBoxR ? kBoxR : nr <= 2 * kBoxR ? 2 * kBoxR : kTileR;
      const uint32_t bytes = (second ? 2 : 1) * kBytesW + xrows * (kTileK * 2);
      for (int ks = 0; ks < ksteps; ++ks, ++fill) {
        const int s = fill % kExpStages;
        if (!(ok = op_wait(empty(s), ((fill / kExpStages) & 1) ^ 1, abort, p.a.status, 1))) break;
        if (elect_one()) {
          const uint32_t st = base + s * kExpStage;
          mbar_expect_tx(full(s), bytes);
          op_tma_3d(st, &tw, ks * kTileK, w0, e, full(s));
          if (second) op_tma_3d(st + kBytesW, GLU ? &tu : &tw, ks * kTileK, GLU ? w0 : w0 + kTileW, e, full(s));
          if (xrows == kTileR) {
            op_tma_2d(st + 2 * kBytesW, &tx128, ks * kTileK, r0, full(s));
          } else if (xrows) {
            op_tma_2d(st + 2 * kBytesW, &tx, ks * kTileK, r0, full(s));
            if (xrows > kBoxR) op_tma_2d(st + 2 * kBytesW + kBoxR * kTileK * 2, &tx, ks * kTileK, r0 + kBoxR, full(s));
          }
        }
        __syncwarp();
      }
    }
    if (*abort) {  // an abandoned run leaves copies in flight: wait for them (bounded)
      const uint32_t n = min(fill, (uint32_t)kExpStages);
      for (uint32_t f = fill - n; f < fill; ++f) mbar_wait(full(f % kExpStages), (f / kExpStages) & 1, 10000000ll);
    }
  } else if (warp >= kExpThreads / 32) {
    // ---------------------------------------------------------------- gather
    // eight threads a row (128 bytes of a stage), 16 rows at a time; a stage is handed over
    // two stages later, when its copies have landed
    const int t128 = (int)threadIdx.x - kExpThreads, chunk = t128 & 7, row0 = t128 >> 3;
    const uint32_t swz = (uint32_t)(chunk ^ (row0 & 7)) * 16;  // (16 j keeps the low three bits of the row)
    uint32_t fill = 0;
    bool ok = true;
    for (int t = (int)blockIdx.x; ok && t < tiles; t += (int)gridDim.x) {
      const ExpTile x = find_tile(p, sh.pre, t, wblocks, kStep);
      const uint16_t* src[kTileR / 16];
#pragma unroll
      for (int j = 0; j < kTileR / 16; ++j) {
        const int i = row0 + 16 * j;
        int r = 0;
        if (i < x.nr) {
          const int s = __ldg(p.a.rows + x.r0 + i);
          r = min(max(s, 0), p.a.n_x - 1);
          if (r != s && x.w0 == 0) op_error(p.a.status, MK_ERR_INVALID, x.e, x.r0 + i, s);
        }
        src[j] = static_cast<const uint16_t*>(p.a.x) + r * p.a.x_stride + 8 * chunk;
      }
      for (int ks = 0; ks < ksteps; ++ks, ++fill) {
        const int s = fill % kExpStages;
        if (!(ok = op_wait(empty(s), ((fill / kExpStages) & 1) ^ 1, abort, p.a.status, 6))) break;
        const uint32_t dst = base + s * kExpStage + 2 * kBytesW + row0 * (kTileK * 2) + swz;
        const int bytes = ks * kTileK + 8 * chunk < p.a.k ? 16 : 0;  // (0: zeros)
#pragma unroll
        for (int j = 0; j < kTileR / 16; ++j)
          if (row0 + 16 * j < x.nr) op_cp16(dst + j * 16 * kTileK * 2, bytes ? src[j] + ks * kTileK : src[j], bytes);
        op_cp_commit();
        if (fill >= kGatherLag) {
          op_cp_wait<kGatherLag>();
          fence_proxy_async_smem();
          mbar_arrive(full((fill - kGatherLag) % kExpStages));
        }
      }
    }
    op_cp_wait<0>();
    fence_proxy_async_smem();
    if (ok)
      for (uint32_t f = fill > kGatherLag ? fill - kGatherLag : 0; f < fill; ++f) mbar_arrive(full(f % kExpStages));
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issue
    uint32_t used = 0, nt = 0;
    const uint32_t tm = uniform(tmem);
    const uint64_t d0 = umma_sdesc_sw(base, 16, 1024, 128);  // stage 0: weights, second weights, rows
    bool ok = true;
    for (int t = (int)blockIdx.x; ok && t < tiles; t += (int)gridDim.x, ++nt) {
      const ExpTile x = find_tile(p, sh.pre, t, wblocks, kStep);
      const bool second = GLU || uniform(x.w0 + kTileW < p.a.n);
      const uint32_t idesc = umma_idesc_bf16(kTileW, (uniform(x.nr) + 15) / 16 * 16);
      const uint32_t a = nt & 1, acc = tm + 256 * a;
      if (!(ok = op_wait(aempty(a), ((nt >> 1) & 1) ^ 1, abort, p.a.status, 2))) break;
      tc_fence_after();
      for (int ks = 0; ks < ksteps; ++ks, ++used) {
        const int s = used % kExpStages;
        if (!(ok = op_wait(full(s), (used / kExpStages) & 1, abort, p.a.status, 3))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t d = d0 + s * (kExpStage / 16);
#pragma unroll
          for (int kk = 0; kk < kTileK / 16; ++kk) {
            umma_bf16(acc, d + 2 * kk, d + 2 * kBytesW / 16 + 2 * kk, idesc, ks > 0 || kk > 0);
            if (second) umma_bf16(acc + 128, d + kBytesW / 16 + 2 * kk, d + 2 * kBytesW / 16 + 2 * kk, idesc, ks > 0 || kk > 0);
          }
          umma_commit(empty(s));
          if (ks == ksteps - 1) umma_commit(afull(a));
        }
        __syncwarp();
      }
    }
    if (*abort) {  // let the products in flight end before the memory goes
      const uint64_t t0 = gtime();
      while ((long long)(gtime() - t0) < 10000000ll) {}
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;               // lanes 32 q .. of tensor memory
    const int col = 32 * q + lane;        // weight row of the block
    uint32_t nt = 0, nm = 0;
    auto meet = [&]() -> bool {           // all four warps, bounded like every wait
      mbar_arrive(emeet);
      return op_wait(emeet, nm++ & 1, abort, p.a.status, 5);
    };
    uint16_t* const stage = reinterpret_cast<uint16_t*>(out_g);
    // whole 16-byte pieces of an output row where its address allows them
    const bool wide = p.a.n % 8 == 0 && p.a.out_stride % 8 == 0 && (reinterpret_cast<uintptr_t>(p.a.out) & 15) == 0;
    bool ok = true;
    for (int t = (int)blockIdx.x; ok && t < tiles; t += (int)gridDim.x, ++nt) {
      const ExpTile x = find_tile(p, sh.pre, t, wblocks, kStep);
      const uint32_t a = nt & 1;
      const uint32_t acc = tmem + 256 * a + ((uint32_t)q << 21);
      if (!(ok = op_wait(afull(a), (nt >> 1) & 1, abort, p.a.status, 4))) break;
      tc_fence_after();
#pragma unroll 1
      for (int blk = 0; ok && blk < (GLU ? 1 : 2); ++blk) {
        const int w0 = x.w0 + blk * kTileW;
        if (w0 >= p.a.n) break;
        for (int c = 0; c < x.nr; c += 16) {
          uint32_t u[16];
          tmem_ld16(acc + 128 * blk + c, u);
          tmem_wait16(u);
          if (GLU) {
            uint32_t v[16];
            tmem_ld16(acc + 128 + c, v);
            tmem_wait16(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(silu(__uint_as_float(u[i])) * __uint_as_float(v[i]));
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) stage[(c + i) * kTileW + col] = to_bf16(__uint_as_float(u[i]));
        }
        if (GLU || blk == 1 || w0 + kTileW >= p.a.n) {
          tc_fence_before();
          mbar_arrive(aempty(a));
        }
        if (!(ok = meet())) break;
        const int tid = (int)threadIdx.x - 64, width = min(kTileW, p.a.n - w0);
        uint16_t* out = static_cast<uint16_t*>(p.a.out) + w0;
        if (wide) {
          const int c8 = tid & 15;
          if (8 * c8 < width)
            for (int r = tid >> 4; r < x.nr; r += 8)
              *reinterpret_cast<uint4*>(out + (x.r0 + r) * p.a.out_stride + 8 * c8) =
                  *reinterpret_cast<const uint4*>(stage + r * kTileW + 8 * c8);
        } else if (tid < width) {
          for (int r = 0; r < x.nr; ++r) out[(x.r0 + r) * p.a.out_stride + tid] = stage[r * kTileW + tid];
        }
        ok = meet();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

template <bool GLU>
static cudaError_t launch_glu(const ExpertParams& p, const CUtensorMap& tx, const CUtensorMap& tx128, const CUtensorMap& tw, const CUtensorMap& tu,
                              cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(expert_kernel<GLU>, kExpSmem, done);
  if (e != cudaSuccess) return e;
  expert_kernel<GLU><<<p.grid, kExpThreads + (p.a.rows ? kGatherThreads : 0), kExpSmem, st>>>(p, tx, tx128, tw, tu);
  return cudaGetLastError();
}

cudaError_t launch_experts(const ExpertParams& p, const CUtensorMap& tx, const CUtensorMap& tx128, const CUtensorMap& tw, const CUtensorMap& tu,
                           cudaStream_t st) {
  return p.a.w_up ? launch_glu<true>(p, tx, tx128, tw, tu, st) : launch_glu<false>(p, tx, tx128, tw, tu, st);
}

}  // namespace mk
