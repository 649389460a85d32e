// The routed layer of a few tokens:  out = residual + sum_j c_j Wd[id_j] (silu(Wg[id_j] x) * (Wu[id_j] x)).
//
// Two kernels.  router_kernel: scores, selection, weights.  layer_kernel: both products, one CTA per SM, with the first product's
// results handed over inside the kernel so that the second one's weights are under way while the last results of the first are
// added up.
//
// With few tokens every selected expert's weights are read for a handful of rows: HBM bounds it, and the products only have to
// keep up.  Every warp has a ring of its own that it fills itself, with tensor-map copies of 8 rows by 64 columns (no barrier
// between warps; 128 columns of 16 rows a step), and multiplies with m16n8k16: with 8 rows an expert a tcgen05 tile would be empty but for a sixteenth.  The
// warps split k; their parts of a result meet in shared memory and are added in the order of the warps.
//
// First product: a unit is 8 outputs of an expert (8 gate and 8 up rows of weights: one 16-row tile) for up to 8 NT of its
// rows, which stay in shared memory for all units of the expert.  The list of units is cut into as many equal runs as there are
// CTAs, and a CTA claims a run when it starts, so that a wait for the first product never waits for a CTA that has yet to
// start.  Second product: a CTA has up to 16 output columns and goes through all experts with them, so that the sum over a
// token's experts stays in the CTA, in the order of the experts: no partial results leave it.
#include <algorithm>

#include "mk_ops.cuh"

namespace mk {
namespace {

// ------------------------------------------------------------------------------------------ router
// A cluster of 8 CTAs has TT tokens and an eighth of the experts a CTA.  A selection can hang on the last bits of two scores, so
// these are sums of exact products (two bf16 factors fit fp32) with the rounding errors of the additions carried along.
constexpr int kRouterCtas = 8, kRouterThreads = 512, kRouterWarps = kRouterThreads / 32;

// (hi, lo) += v, the error of hi + v to lo; two sums at once
__device__ __forceinline__ void add_exact2(uint64_t& hi, uint64_t& lo, uint64_t v) {
  const uint64_t minus = pack2(-1.f, -1.f);
  const uint64_t s = add2(hi, v), z = fma2(hi, minus, s);
  const uint64_t a = fma2(fma2(z, minus, s), minus, hi), b = fma2(z, minus, v);
  lo = add2(lo, add2(a, b));
  hi = s;
}
__device__ __forceinline__ void add_exact(float& hi, float& lo, float v) {
  const float s = hi + v, z = s - hi;
  lo += (hi - (s - z)) + (v - z);
  hi = s;
}
__device__ __forceinline__ uint64_t pair_of(uint32_t bf16x2) {
  const float2 f = bf16x2_to_f2(bf16x2);
  return pack2(f.x, f.y);
}

// order of scores as unsigned integers; NaN above everything, the two zeros equal
__device__ __forceinline__ unsigned long long score_key(double d) {
  if (d != d) return ~0ull;
  const long long v = __double_as_longlong(d == 0.0 ? 0.0 : d);
  return v < 0 ? ~(unsigned long long)v : (unsigned long long)v | (1ull << 63);
}

template <int TT>
__global__ void __cluster_dims__(kRouterCtas, 1, 1) __launch_bounds__(kRouterThreads) router_kernel(const __grid_constant__ MoeParams p) {
  __shared__ double s_score[kOpMaxExperts];  // of the token that this CTA selects for
  extern __shared__ __align__(16) uint8_t raw_x[];  // the tokens' rows
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int t0 = (int)(blockIdx.x / kRouterCtas) * TT, E = p.a.n_experts, d = p.a.d_model;
  const int per = (E + kRouterCtas - 1) / kRouterCtas, e0 = (int)rank * per, e1 = min(E, e0 + per);
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // (all CTAs have started: waited for below)
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && tid < 4) p.sync[tid] = 0;
  uint4* const x = reinterpret_cast<uint4*>(raw_x);
  const int vecs = d / 8;
  // (the first weights are on their way while the tokens' rows come in)
  constexpr int U = TT <= 2 ? 8 : 4;
  uint4 u[U];
  const uint16_t* w = static_cast<const uint16_t*>(p.a.router) + (long long)min(e0 + warp, E - 1) * d;
  auto fetch = [&](int v) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (v + 32 * i < vecs) u[i] = op_ld16(w + 8 * (v + 32 * i));
  };
  fetch(lane);
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const uint16_t* const row = static_cast<const uint16_t*>(p.a.x) + min(t0 + j, p.a.n_tokens - 1) * p.a.x_stride;
    for (int v = tid; v < vecs; v += kRouterThreads) op_cp16(smem_u32(x + j * vecs + v), row + 8 * v, 16);
  }
  op_cp_wait_all();
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  for (int e = e0 + warp; e < e1; e += kRouterWarps) {
    uint64_t hi[TT], lo[TT];
#pragma unroll
    for (int j = 0; j < TT; ++j) hi[j] = lo[j] = 0;
    for (int v = lane; v < vecs; v += 32 * U) {
      if (e != e0 + warp || v != lane) {
        if (v == lane) w = static_cast<const uint16_t*>(p.a.router) + (long long)e * d;
        fetch(v);
      }
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (v + 32 * i < vecs) {
          const uint64_t w4[4] = {pair_of(u[i].x), pair_of(u[i].y), pair_of(u[i].z), pair_of(u[i].w)};
#pragma unroll
          for (int j = 0; j < TT; ++j) {
            const uint4 y = x[j * vecs + v + 32 * i];
            add_exact2(hi[j], lo[j], mul2(w4[0], pair_of(y.x)));
            add_exact2(hi[j], lo[j], mul2(w4[1], pair_of(y.y)));
            add_exact2(hi[j], lo[j], mul2(w4[2], pair_of(y.z)));
            add_exact2(hi[j], lo[j], mul2(w4[3], pair_of(y.w)));
          }
        }
    }
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      const float2 h = unpack2(hi[j]), l = unpack2(lo[j]);
      float a = h.x, b = l.x + l.y;
      add_exact(a, b, h.y);
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const float a2 = __shfl_xor_sync(0xffffffffu, a, o), b2 = __shfl_xor_sync(0xffffffffu, b, o);
        // (the same on both sides of an exchange: addition and its error are symmetric)
        add_exact(a, b, a2);
        b += b2;
      }
      // infinities and NaN: the carried errors are NaN, the sum itself tells
      const double s = fabsf(a) < INFINITY ? (double)a + (double)b : (double)a;
      if (lane == 0) {
        uint32_t to;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(s_score + e)), "r"(j));
        asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(to), "l"(__double_as_longlong(s)) : "memory");
      }
    }
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  const int t = t0 + (int)rank;
  if (warp != 0 || (int)rank >= TT || t >= p.a.n_tokens) return;
  constexpr int kMine = kOpMaxExperts / 32;
  unsigned long long key[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int e = lane + 32 * i;
    key[i] = e < E ? score_key(s_score[e]) : 0;  // (no score's key is 0)
  }
  int id = 0;
  double first = 0;
  float mine = 0.f, total = 0.f;
  for (int j = 0; j < p.a.top_k; ++j) {
    unsigned long long best = key[0];
#pragma unroll
    for (int i = 1; i < kMine; ++i) best = max(best, key[i]);
    const uint32_t top = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32));
    const uint32_t low = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32) == top ? (uint32_t)best : 0u);
    best = (unsigned long long)top << 32 | low;
    int where = kOpMaxExperts;
#pragma unroll
    for (int i = kMine - 1; i >= 0; --i)
      if (key[i] == best) where = lane + 32 * i;
    where = __reduce_min_sync(0xffffffffu, where);
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      if (lane + 32 * i == where) key[i] = 0;
    const double s = s_score[where];
    if (j == 0) first = s;
    const float c = expf((float)(s - first));
    total += c;
    if (lane == j) id = where, mine = c;
  }
  if (lane < p.a.top_k) {
    p.ids[t * p.a.top_k + lane] = id;
    p.weights[t * p.a.top_k + lane] = mine / total;
  }
}

// ------------------------------------------------------------------------------------------- layer
constexpr int kLayerThreads = 256, kLayerWarps = kLayerThreads / 32;
constexpr int kSpan = 64;        // columns of a copy: one 128-byte swizzle span
constexpr int kStepK = 2 * kSpan;
constexpr int kTileBytes = 4096; // weights of a step: 16 rows, two copies of 2 KB
constexpr int kMaxSlots = 10;    // of a warp's ring
constexpr int kAccPitch = 20;

struct LayerShared {
  int off[kOpMaxExperts + 1];       // first row of every expert in the list
  int act[kOpMaxExperts];           // experts that have rows
  int tile_pre[kOpMaxExperts + 1];  // row tiles before each of them
  int2 rows[kOpMaxExperts];         // first row of an active expert's outputs in w_down, first row of its tiles in h
  int n_act, run, next, abort;
  int warp_rows[8], warp_tiles[8], warp_act[8];
  unsigned long long bars[kLayerWarps][kMaxSlots];
};

// offsets in dynamic shared memory, behind the warps' rings; the same on host and device
struct LayerSmem {
  int warp_bytes, red, list, weight, acc, total;
  __host__ __device__ LayerSmem(int nt, bool direct, int slots, int d, int tokens, int top_k) {
    const int entries = tokens * top_k, mine = ((d + kStepK - 1) / kStepK + kLayerWarps - 1) / kLayerWarps;
    warp_bytes = slots * kTileBytes + (slots > mine ? slots : mine) * nt * 2048;  // weights, rows
    red = kLayerWarps * warp_bytes;
    list = red + 2 * kLayerWarps * nt * 32 * 16;  // (the token masks lie here before the first results)
    weight = list + (entries * 2 + 15) / 16 * 16;
    acc = weight + (direct ? entries * 8 : entries) * 4;  // (direct: of every active expert and token)
    acc = (acc + 15) / 16 * 16;
    total = acc + tokens * kAccPitch * 4 + 1024;
  }
};

// acquire-free copies of a box of a matrix
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* tm, int x, int y, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void fence_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

__device__ __forceinline__ float moe_silu(float y) { return __fdividef(y, 1.f + __expf(-y)); }

// NT: row tiles of 8 that share a pass over the weights.  DIRECT (up to 8 tokens): a tile's rows are the tokens, with zeros for
// those that have not selected the expert, so that the second product adds its experts up in registers.
template <int NT, bool DIRECT>
__global__ void __launch_bounds__(kLayerThreads, 1)
    layer_kernel(const __grid_constant__ MoeParams p, const __grid_constant__ CUtensorMap tgate, const __grid_constant__ CUtensorMap tup,
                 const __grid_constant__ CUtensorMap tdown, const __grid_constant__ CUtensorMap th) {
  extern __shared__ uint8_t raw_[];
  __shared__ LayerShared sh;
  const int tid = threadIdx.x, warp = (int)uniform(threadIdx.x >> 5), lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int T = p.a.n_tokens, K = p.a.top_k, E = p.a.n_experts, d = p.a.d_model, f = p.a.d_ff, entries = T * K, S = p.slots;
  const LayerSmem at(NT, DIRECT, S, d, T, K);
  const uint32_t base = (smem_u32(raw_) + 1023u) & ~1023u;
  uint8_t* const raw = raw_ + (base - smem_u32(raw_));
  float4* const red = reinterpret_cast<float4*>(raw + at.red);
  uint32_t* const mask = reinterpret_cast<uint32_t*>(raw + at.red);
  uint16_t* const list = reinterpret_cast<uint16_t*>(raw + at.list);  // token of every row, by expert, then token
  float* const weight = reinterpret_cast<float*>(raw + at.weight);    // ... and its weight (DIRECT: [active expert][8])
  float* const acc = reinterpret_cast<float*>(raw + at.acc);
  const int words = (T + 31) / 32;
  const uint32_t bars = smem_u32(sh.bars[warp]);

  if (tid == 0) {
    for (int w = 0; w < kLayerWarps; ++w)
      for (int s = 0; s < S; ++s) mbar_init(smem_u32(&sh.bars[w][s]), 1);
    fence_proxy_async_smem();
    sh.abort = 0;
    sh.next = -1;
  }
  if (tid >= 32 && tid < 36) {
    const CUtensorMap* tm = tid == 32 ? &tgate : tid == 33 ? &tup : tid == 34 ? &tdown : &th;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tm)) : "memory");
  }
  for (int i = tid; i < E * words; i += kLayerThreads) mask[i] = 0;
  if (DIRECT)
    for (int i = tid; i < entries * 8; i += kLayerThreads) weight[i] = -1.f;
  for (int i = tid; i < T * kAccPitch; i += kLayerThreads) acc[i] = 0.f;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  // ---------------------------------------------------------------- who has which rows
  if (tid == 0) sh.run = (int)atomicAdd(p.sync, 1u);
  int my_id = 0;
  float my_weight = 0.f;
  if (tid < entries) my_id = op_ld(p.ids + tid), my_weight = op_ldf(p.weights + tid);
  for (int i = tid; i < entries; i += kLayerThreads) {
    const int t = i / K;
    atomicOr(mask + (i == tid ? my_id : op_ld(p.ids + i)) * words + (t >> 5), 1u << (t & 31));
  }
  __syncthreads();
  {  // (one expert a thread)
    const int e = tid;
    int n = 0;
    if (e < E)
      for (int w = 0; w < words; ++w) n += __popc(mask[e * words + w]);
    const int k = DIRECT ? (n > 0) : (n + 8 * NT - 1) / (8 * NT);
    int r = n, c = k;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, r, o), b = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) r += a, c += b;
    }
    const unsigned some = __ballot_sync(0xffffffffu, n > 0);
    if (lane == 31) sh.warp_rows[warp] = r, sh.warp_tiles[warp] = c, sh.warp_act[warp] = __popc(some);
    __syncthreads();
    int rows = 0, tiles = 0, active = 0;
    for (int w = 0; w < warp; ++w) rows += sh.warp_rows[w], tiles += sh.warp_tiles[w], active += sh.warp_act[w];
    const int idx = active + __popc(some & ((1u << lane) - 1));
    if (e < E) sh.off[e] = rows + r - n;
    if (n > 0) sh.act[idx] = e, sh.tile_pre[idx] = tiles + c - k;
    if (tid == kLayerThreads - 1) {
      sh.off[E] = rows + r;
      sh.n_act = active + __popc(some);
      sh.tile_pre[sh.n_act] = tiles + c;
    }
  }
  __syncthreads();
  const int A = (int)uniform(sh.n_act), groups = f / 8;
  if (tid < A) sh.rows[tid] = make_int2(sh.act[tid] * d, DIRECT ? tid * 8 : sh.off[sh.act[tid]]);
  for (int i = tid; i < entries; i += kLayerThreads) {
    const int t = i / K, e = i == tid ? my_id : op_ld(p.ids + i);
    const float c = i == tid ? my_weight : op_ldf(p.weights + i);
    if (DIRECT) {
      int lo = 0;  // the expert's place among the active ones
#pragma unroll
      for (int step = kOpMaxExperts / 2; step; step >>= 1)
        if (lo + step < A && sh.act[lo + step] <= e) lo += step;
      weight[lo * 8 + t] = c;
    } else {
      int r = sh.off[e];
      for (int w = 0; w < (t >> 5); ++w) r += __popc(mask[e * words + w]);
      r += __popc(mask[e * words + (t >> 5)] & ((1u << (t & 31)) - 1));
      list[r] = (uint16_t)t;
      weight[r] = c;
    }
  }
  __syncthreads();
  const long long units = (long long)uniform(sh.tile_pre[A]) * groups;
  const int runs = (int)gridDim.x, steps_up = (d + kStepK - 1) / kStepK, steps_down = (f + kStepK - 1) / kStepK;

  // ---------------------------------------------------------------- the warp's ring
  const uint32_t tiles_at = base + warp * at.warp_bytes, rows_at = tiles_at + S * kTileBytes;
  Ring get;
  uint32_t put = 0;
  // where a lane reads its part of a step: 16 rows of weights, 8 rows of x or h (swizzled 128-byte rows)
  const uint32_t r8 = lane & 7, m4 = lane >> 3;
  const uint32_t a_at = (m4 & 1) * 1024 + r8 * 128, a_x = ((m4 >> 1) ^ r8) << 4, b_at = r8 * 128 + ((m4 ^ r8) << 4);

  // ---------------------------------------------------------------- first product
  // A unit: 8 outputs of an expert for one of its row tiles; the units of a tile follow one another.
  struct Up {
    int left;          // units of the run from here on, this one included
    int a, tile, grp;  // active expert, row tile among all, group of outputs
    int end;           // the expert's last row tile + 1
  };
  auto up_begin = [&](int r) {
    const long long u0 = r * units / runs, u1 = (r + 1) * units / runs;
    Up c{(int)(u1 - u0), 0, 0, 0, 0};
    if (c.left <= 0) return c;
    c.tile = (int)(u0 / groups);
    c.grp = (int)(u0 - (long long)c.tile * groups);
    int lo = 0;
#pragma unroll
    for (int step = kOpMaxExperts / 2; step; step >>= 1)
      if (lo + step < A && sh.tile_pre[lo + step] <= c.tile) lo += step;
    c.a = lo;
    c.end = sh.tile_pre[lo + 1];
    return c;
  };
  auto up_next = [&](Up& c) {
    --c.left;
    if (++c.grp < groups) return;
    c.grp = 0;
    if (++c.tile < c.end || c.left <= 0) return;
    c.end = sh.tile_pre[++c.a + 1];
  };
  Up is{}, cs{};   // issuing and consuming sides
  int istep = warp, irow = 0;

  // ---------------------------------------------------------------- second product
  // Blocks of output columns, this CTA's one after another; per block the row tiles of the active experts, of each the steps.
  // DIRECT: the warps deal out the steps of all experts as one list, else those of every tile.
  struct Down {
    int block, a, tile, end, s;
  };
  const int blocks = (d + p.width - 1) / p.width;
  auto down_fit = [&](Down& c) {  // to the next step of this warp, if this is none
    while (c.s >= steps_down) {
      if (DIRECT) {
        c.s -= steps_down;
        ++c.a;
      } else {
        c.s = warp;
        if (++c.tile == c.end) {
          ++c.a;
          if (c.a < A) c.end = sh.tile_pre[c.a + 1];
        }
      }
      if (c.a >= A) {
        c.block += (int)gridDim.x;
        if (c.block >= blocks) return;
        c.a = c.tile = 0;
        c.end = sh.tile_pre[1];
        c.s = warp;
      }
    }
  };
  auto down_begin = [&]() {
    Down c{(int)blockIdx.x, 0, 0, (int)uniform(sh.tile_pre[1]), warp};
    if (!DIRECT && warp >= steps_down) c.block = blocks;  // (a warp without steps)
    if (c.block < blocks) down_fit(c);
    return c;
  };
  Down id = down_begin(), ib = id;  // weights, rows
  int ahead = 0;                    // steps of the second product whose weights are under way and whose rows are not
  const uint32_t down_bytes = 2 * (p.width * 128 + NT * 1024);

  auto issue_weights = [&]() {
    if (elect_one()) {
      const uint32_t bar = bars + 8 * put, dst = tiles_at + put * kTileBytes;
      const int row = sh.rows[id.a].x + id.block * p.width;
      mbar_expect_tx(bar, down_bytes);
      tma_box(dst, &tdown, id.s * kStepK, row, bar);
      tma_box(dst + kTileBytes / 2, &tdown, id.s * kStepK + kSpan, row, bar);
    }
    __syncwarp();
    put = put + 1 == (uint32_t)S ? 0 : put + 1;
    id.s += kLayerWarps;
    down_fit(id);
  };
  auto issue_rows = [&](uint32_t slot) {
    if (elect_one()) {
      const int row = sh.rows[ib.a].y + (DIRECT ? 0 : (ib.tile - sh.tile_pre[ib.a]) * NT * 8);
      const uint32_t dst = rows_at + slot * NT * 2048, bar = bars + 8 * slot;
      tma_box(dst, &th, ib.s * kStepK, row, bar);
      tma_box(dst + NT * 1024, &th, ib.s * kStepK + kSpan, row, bar);
    }
    __syncwarp();
    ib.s += kLayerWarps;
    down_fit(ib);
  };
  int next_run = -1;  // -1: not known yet
  // (at most S steps are under way: a slot is filled again once its step has been multiplied)
  auto issue_next = [&]() {
    if (is.left > 0) {
      if (istep >= steps_up) return;  // (a warp without steps)
      if (elect_one()) {
        const uint32_t bar = bars + 8 * put, dst = tiles_at + put * kTileBytes;
        mbar_expect_tx(bar, kTileBytes);
        tma_box(dst, &tgate, istep * kStepK, irow, bar);
        tma_box(dst + 1024, &tup, istep * kStepK, irow, bar);
        tma_box(dst + kTileBytes / 2, &tgate, istep * kStepK + kSpan, irow, bar);
        tma_box(dst + kTileBytes / 2 + 1024, &tup, istep * kStepK + kSpan, irow, bar);
      }
      __syncwarp();
      put = put + 1 == (uint32_t)S ? 0 : put + 1;
      istep += kLayerWarps;
      if (istep >= steps_up) {
        istep = warp;
        up_next(is);
        if (is.left > 0) irow = sh.act[is.a] * f + 8 * is.grp;
      }
    } else if (next_run >= runs && id.block < blocks && ahead < S) {
      issue_weights();
      ++ahead;
    }
  };

  // (several sums a tile, so that the products need not wait for one another)
  constexpr int kSets = NT == 1 ? 4 : 2;
  float sum[kSets][NT][4];
  auto multiply = [&](uint32_t rows, int nt) {
    op_wait(bars + 8 * get.slot, get.phase, &sh.abort, p.a.status, 2);
    const uint32_t tile = tiles_at + get.slot * kTileBytes + a_at;
#pragma unroll
    for (int half = 0; half < 4; ++half) {
      uint32_t a[8];
      const uint32_t t = tile + (half >> 1) * (kTileBytes / 2), x = a_x ^ ((half & 1) << 6);
      ldsm_x4(t + x, a[0], a[1], a[2], a[3]);
      ldsm_x4(t + (x ^ 32), a[4], a[5], a[6], a[7]);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (j > 0 && j >= nt) break;
        uint32_t b[4];
        ldsm_x4(rows + (half >> 1) * (NT * 1024) + j * 1024 + (b_at ^ ((half & 1) << 6)), b[0], b[1], b[2], b[3]);
        mma_bf16(sum[(2 * half) % kSets][j], a[0], a[1], a[2], a[3], b[0], b[1]);
        mma_bf16(sum[(2 * half + 1) % kSets][j], a[4], a[5], a[6], a[7], b[2], b[3]);
      }
    }
    __syncwarp();
    get.advance(S);
  };
  auto clear = [&]() {
#pragma unroll
    for (int k = 0; k < kSets; ++k)
#pragma unroll
      for (int j = 0; j < NT; ++j) sum[k][j][0] = sum[k][j][1] = sum[k][j][2] = sum[k][j][3] = 0.f;
  };
  // the warps' parts of tile j, added up (by one warp)
  auto add_up = [&](int buf, int j) {
    float4 y = red[((buf * kLayerWarps) * NT + j) * 32 + lane];
#pragma unroll
    for (int w = 1; w < kLayerWarps; ++w) {
      const float4 z = red[((buf * kLayerWarps + w) * NT + j) * 32 + lane];
      y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
    }
    return y;
  };
  auto hand_in = [&](int buf, int nt) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
      if (j < nt) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = sum[0][j][i] + sum[1][j][i];
          if (kSets == 4) v[i] += sum[kSets - 2][j][i] + sum[kSets - 1][j][i];
        }
        red[((buf * kLayerWarps + warp) * NT + j) * 32 + lane] = make_float4(v[0], v[1], v[2], v[3]);
      }
    __syncthreads();
  };
  // this warp's steps of the rows of a tile (n of them from the list's first on; DIRECT: of all tokens)
  auto load_rows = [&](int first, int n) {
    uint32_t dst = rows_at;
    for (int s = warp; s < steps_up; s += kLayerWarps)
      for (int span = 0; span < 2; ++span, dst += NT * 1024) {
        const int k = s * kStepK + span * kSpan + 8 * (int)r8;
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) {
          const int r = (int)m4 + 4 * i;
          if (r < n) {
            const int t = DIRECT ? r : list[first + r];
            const uint16_t* const row = static_cast<const uint16_t*>(p.a.x) + t * p.a.x_stride;
            op_cp16(dst + r * 128 + ((r8 ^ (r & 7)) << 4), k < d ? row + k : row, k < d ? 16 : 0);
          }
        }
      }
    op_cp_wait_all();
    __syncwarp();
  };

  int buf = 0, have = -1;  // the tile whose rows are there
  long long made = 0;
  for (int run = (int)uniform(sh.run); run < runs;) {
    cs = is = up_begin(run);
    istep = warp;
    if (is.left > 0) irow = sh.act[is.a] * f + 8 * is.grp;
    next_run = -1;
    const int all = cs.left, middle = all / 2;
    for (int i = 0; i < S; ++i) issue_next();
    while (cs.left > 0) {
      if (tid == 0 && all - cs.left == middle) *(volatile int*)&sh.next = (int)atomicAdd(p.sync, 1u);
      const int e = sh.act[cs.a], first = sh.off[e] + (DIRECT ? 0 : (cs.tile - sh.tile_pre[cs.a]) * NT * 8);
      const int n = DIRECT ? T : min(sh.off[e + 1] - first, NT * 8), nt = (n + 7) / 8;
      if (DIRECT ? have < 0 : have != cs.tile) load_rows(first, n);
      have = cs.tile;
      clear();
      uint32_t rows = rows_at;
      for (int s = warp; s < steps_up; s += kLayerWarps, rows += NT * 2048) {
        multiply(rows, nt);
        issue_next();
      }
      hand_in(buf, nt);
      next_run = (int)uniform((uint32_t)*(volatile int*)&sh.next);
      const int j = (warp - cs.left) & (kLayerWarps - 1);
      if (j < nt) {
        const float4 y = add_up(buf, j);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = j * 8 + 2 * q + i;
          if (r < n) {
            const float gate = i ? y.y : y.x, up = i ? y.w : y.z, c = weight[DIRECT ? cs.a * 8 + r : first + r];
            // (c < 0: the token has not selected the expert, and its product does not count, whatever it is)
            p.h[(long long)(DIRECT ? cs.a * 8 + r : first + r) * f + 8 * cs.grp + g] = c < 0.f ? (uint16_t)0 : to_bf16(c * (moe_silu(gate) * up));
          }
        }
      }
      buf ^= 1;
      up_next(cs);
      ++made;
    }
    // (a run without units has claimed nothing more)
    if (all == 0 && tid == 0) sh.next = (int)atomicAdd(p.sync, 1u);
    __syncthreads();
    run = next_run = (int)uniform(sh.next);
    __syncthreads();
    if (tid == 0) sh.next = -1;
  }
  // ---------------------------------------------------------------- hand over
  for (; ahead < S && id.block < blocks; ++ahead) issue_weights();
  fence_async_global();  // (the results are read by tensor-map copies)
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    if (made) red_release(p.sync + 1, (unsigned)made);
    const uint64_t t0 = gtime();
    while (ld_acquire(p.sync + 1) != (unsigned)units)
      if ((long long)(gtime() - t0) > kOpWaitNs) {
        op_error(p.a.status, MK_ERR_TIMEOUT, (int)blockIdx.x, 1, (int)ld_acquire(p.sync + 1));
        break;
      }
  }
  __syncthreads();
  fence_async_global();
  {
    uint32_t slot = get.slot;
    for (int i = 0; i < ahead; ++i) {
      issue_rows(slot);
      slot = slot + 1 == (uint32_t)S ? 0 : slot + 1;
    }
  }
  auto take = [&](int nt) {
    multiply(rows_at + get.slot * NT * 2048, nt);
    if (id.block < blocks) {
      const uint32_t slot = put;
      issue_weights();
      issue_rows(slot);
    }
  };

  for (int block = blockIdx.x; block < blocks; block += (int)gridDim.x) {
    const int c0 = block * p.width, wide = min(p.width, d - c0);
    clear();
    if (DIRECT) {
      const int n = A * steps_down;
      for (int s = warp; s < n; s += kLayerWarps) take(1);
      hand_in(buf, 1);
      if (warp == 0) {
        const float4 y = add_up(buf, 0);
        const float v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 2 * q + (i & 1);
          if (t < T) acc[t * kAccPitch + g + 8 * (i >> 1)] = v[i];
        }
      }
      buf ^= 1;
    } else {
      for (int a = 0; a < A; ++a) {
        const int e = sh.act[a], last = sh.off[e + 1];
        for (int first = sh.off[e], turn = a; first < last; first += NT * 8, ++turn) {
          const int n = min(last - first, NT * 8), nt = (n + 7) / 8;
          clear();
          for (int s = warp; s < steps_down; s += kLayerWarps) take(nt);
          hand_in(buf, nt);
          const int j = (warp - turn) & (kLayerWarps - 1);
          if (j < nt) {
            const float4 y = add_up(buf, j);
            const float v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = j * 8 + 2 * q + (i & 1);
              if (r < n) acc[list[first + r] * kAccPitch + g + 8 * (i >> 1)] += v[i];
            }
          }
          buf ^= 1;
        }
      }
    }
    __syncthreads();
    for (int i = tid; i < T * 16; i += kLayerThreads) {
      const int t = i >> 4, c = i & 15;
      float y = acc[t * kAccPitch + c];
      acc[t * kAccPitch + c] = 0.f;
      if (c < wide) {
        if (p.a.residual) y += bf16_to_f(op_ld2(static_cast<const uint16_t*>(p.a.residual) + t * p.a.residual_stride + c0 + c));
        static_cast<uint16_t*>(p.a.out)[t * p.a.out_stride + c0 + c] = to_bf16(y);
      }
    }
    __syncthreads();
  }
  if (sh.abort) {  // an abandoned run leaves copies in flight: give them time to land
    const uint64_t s0 = gtime();
    while ((long long)(gtime() - s0) < 10000000ll) {}
  }
}

template <int TT>
cudaError_t launch_router(const MoeParams& p, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(router_kernel<TT>, TT * kMoeWidest * 2, done);
  if (e != cudaSuccess) return e;
  return launch_early(router_kernel<TT>, dim3((unsigned)((p.a.n_tokens + TT - 1) / TT * kRouterCtas)), kRouterThreads, (size_t)TT * p.a.d_model * 2, st, p);
}

size_t align16(size_t n) { return (n + 15) / 16 * 16; }

constexpr int kMostSmem = 232448 - ((int)sizeof(LayerShared) + 127) / 128 * 128;

// slots of a warp's ring that fit: as many as there is room for
int layer_slots(const mk_moe_args& a, int nt, bool direct) {
  for (int s = kMaxSlots; s >= 2; --s)
    if (LayerSmem(nt, direct, s, a.d_model, a.n_tokens, a.top_k).total <= kMostSmem) return s;
  return 0;
}

template <int NT, bool DIRECT>
cudaError_t launch_layer(const MoeParams& p, const MoeMaps& m, cudaStream_t st) {
  const int smem = LayerSmem(NT, DIRECT, p.slots, p.a.d_model, p.a.n_tokens, p.a.top_k).total;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(layer_kernel<NT, DIRECT>, kMostSmem, done);
  if (e != cudaSuccess) return e;
  return launch_early(layer_kernel<NT, DIRECT>, dim3((unsigned)p.grid), kLayerThreads, (size_t)smem, st, p, m.gate, m.up, m.down, m.h);
}

}  // namespace

long long moe_h_rows(const mk_moe_args& a) {
  const long long entries = (long long)a.n_tokens * a.top_k;
  return a.n_tokens <= kMoeDirect ? 8 * std::min<long long>(a.n_experts, entries) : entries;
}

size_t moe_workspace_bytes(const mk_moe_args& a) {
  const size_t entries = (size_t)a.n_tokens * a.top_k;
  return 16 + 2 * align16(entries * 4) + (size_t)moe_h_rows(a) * a.d_ff * 2;
}

int moe_shape(MoeParams& p) {
  const mk_moe_args& a = p.a;
  const size_t entries = (size_t)a.n_tokens * a.top_k;
  uint8_t* at = static_cast<uint8_t*>(a.workspace);
  p.sync = reinterpret_cast<uint32_t*>(at);
  at += 16;
  p.ids = a.ids ? a.ids : reinterpret_cast<int32_t*>(at);
  at += align16(entries * 4);
  p.weights = a.weights ? a.weights : reinterpret_cast<float*>(at);
  at += align16(entries * 4);
  p.h = reinterpret_cast<uint16_t*>(at);
  // output columns: 16 at most, in blocks of equal width over all CTAs
  const int rounds = (a.d_model + 16 * p.grid - 1) / (16 * p.grid);
  p.width = (a.d_model + rounds * p.grid - 1) / (rounds * p.grid);
  // rows of a tile: what most experts have
  const double mean = (double)entries / a.n_experts;
  p.direct = a.n_tokens <= kMoeDirect;
  p.nt = p.direct || mean <= 3 ? 1 : mean <= 10 ? 2 : 4;
  while ((p.slots = layer_slots(a, p.nt, p.direct)) < 3 && p.nt > 1) p.nt /= 2;
  return p.slots;
}

cudaError_t launch_moe(const MoeParams& p, const MoeMaps& m, cudaStream_t st) {
  const int t = p.a.n_tokens, clusters = 2 * p.grid / kRouterCtas;
  cudaError_t e = t <= clusters       ? launch_router<1>(p, st)
                  : t <= 2 * clusters ? launch_router<2>(p, st)
                  : t <= 4 * clusters ? launch_router<4>(p, st)
                                      : launch_router<8>(p, st);
  if (e != cudaSuccess) return e;
  return p.direct    ? launch_layer<1, true>(p, m, st)
         : p.nt == 1 ? launch_layer<1, false>(p, m, st)
         : p.nt == 2 ? launch_layer<2, false>(p, m, st)
                     : launch_layer<4, false>(p, m, st);
}

}  // namespace mk
