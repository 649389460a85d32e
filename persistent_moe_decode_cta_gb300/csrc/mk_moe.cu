// The routed layer of a few tokens:  out = residual + sum_j c_j Wd[id_j] (silu(Wg[id_j] x) * (Wu[id_j] x)).
//
// router_kernel: scores, selection, weights.  Then, for up to 8 tokens, layer_kernel: both products in one kernel, one CTA per
// SM, with the first product's results handed over inside it so that the second one's weights are under way while the last
// results of the first are added up.  For more tokens the products of mk_experts.cu, between sort_kernel and sum_kernel.
//
// With few tokens every selected expert's weights are read for a handful of rows: HBM bounds it, and the products only have to
// keep up.  In layer_kernel every warp has a ring of its own that it fills itself, with tensor-map copies of 8 rows by 64
// columns (no barrier between warps; 128 columns of 16 rows a step), and multiplies with m16n8k16: with 8 rows an expert a tcgen05
// tile would be empty but for a sixteenth.
//
// Its first product: a unit is 8 outputs of an expert (8 gate and 8 up rows of weights: one 16-row tile), a warp's alone from the
// first column to the last, so that gate and up of an output meet in a lane.  The list of units is cut into as many equal runs
// as there are CTAs, and a CTA claims a run when it starts, so that a wait for the first product never waits for a CTA that has
// yet to start.  Second product: a CTA has up to 16 output columns and goes through all experts with them, the warps taking steps
// in turn; their sums meet at the end, in the order of the warps, and no partial results leave the CTA.
//
// Measured in a graph (2048 wide, 128 experts of 768, 8 a token): 1 token 23.9 us (76 MB; a chain: router 4, start and list 2.5, the
// first product 8, handover 2, the second 4, the rest launches), 4 55.8, 8 90 (5.4 TB/s), 16 142, 128 217 us (router 9, sort 3,
// products 124 and 70, sum 5; 5.6 TB/s); 32 experts of 1024 x 512, 4 a token: 1 token 12.5 us, 8 26, 9 35, 64 40.
#include <algorithm>
#include <type_traits>

#include "mk_linear.cuh"

namespace mk {
namespace {

// ------------------------------------------------------------------------------------------ router
// A cluster of CTAS has TT tokens and its share of the experts a CTA (MANY: more than 64 experts).  A selection can hang on the last
// bits of two scores.  So the fp32 scores come with a bound of their error, and those that lie within it of one another around the selection (one token in
// twenty has such) are computed once more from exact products (two bf16 factors fit fp32), the errors of all additions carried
// along.  (All scores that way: 128 tokens 19 us; every sum of four terms that way, 25.)
constexpr int kRouterThreads = 512, kRouterWarps = kRouterThreads / 32;

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
// (a, b) = the two sums of all lanes together (the same in every lane: addition and its error are symmetric)
__device__ __forceinline__ void add_lanes(uint64_t hi, uint64_t lo, float& a, float& b) {
  const float2 h = unpack2(hi), l = unpack2(lo);
  a = h.x, b = l.x + l.y;
  add_exact(a, b, h.y);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float a2 = __shfl_xor_sync(0xffffffffu, a, o), b2 = __shfl_xor_sync(0xffffffffu, b, o);
    add_exact(a, b, a2);
    b += b2;
  }
}
// w . x by a warp, to 2^-46 of the sum of the terms' sizes (the same in every lane)
__device__ __noinline__ double exact_score(const uint16_t* w, const uint4* x, int vecs) {
  uint64_t hi = 0, lo = 0;
  for (int v0 = threadIdx.x & 31; v0 < vecs; v0 += 256) {
    uint4 u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (v0 + 32 * i < vecs) u[i] = op_ld16(w + 8 * (v0 + 32 * i));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (v0 + 32 * i < vecs) {
        const uint4 y = x[v0 + 32 * i];
        add_exact2(hi, lo, mul2(pair_of(u[i].x), pair_of(y.x)));
        add_exact2(hi, lo, mul2(pair_of(u[i].y), pair_of(y.y)));
        add_exact2(hi, lo, mul2(pair_of(u[i].z), pair_of(y.z)));
        add_exact2(hi, lo, mul2(pair_of(u[i].w), pair_of(y.w)));
      }
  }
  float a, b;
  add_lanes(hi, lo, a, b);
  // (infinities and NaN: the carried errors are NaN, the sum itself tells)
  return fabsf(a) < INFINITY ? (double)a + (double)b : (double)a;
}

// order of scores as unsigned integers; NaN above everything, the two zeros equal
__device__ __forceinline__ unsigned long long score_key(double d) {
  if (d != d) return ~0ull;
  const long long v = __double_as_longlong(d == 0.0 ? 0.0 : d);
  return v < 0 ? ~(unsigned long long)v : (unsigned long long)v | (1ull << 63);
}

struct RouterShared {
  float2 score[kOpMaxExperts];           // of the token that this CTA selects for, and what it may be off by
  float4 flat[kOpMaxExperts / 4];        // the scores alone; -infinity beyond the last
  float best[kMoeTopK + 1];              // ... of the first ranks, in their order
  unsigned long long key[kOpMaxExperts];
  int rank[kOpMaxExperts];
  uint32_t close[kOpMaxExperts / 32];    // experts whose scores are not told apart
  float xn[kRouterWarps];                // parts of the token's square
  float bound;                           // the score of rank K
  int most, odd;                         // bits of the largest error; whether something is infinite or NaN
  int chosen[kMoeTopK];
  float value[kMoeTopK];
};

template <int TT, int CTAS, bool MANY>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kRouterThreads) router_kernel(const __grid_constant__ MoeParams p) {
  extern __shared__ __align__(16) uint8_t raw_x[];  // the tokens' rows
  __shared__ RouterShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int t0 = (int)(blockIdx.x / CTAS) * TT, E = p.a.n_experts, d = p.a.d_model;
  const int per = (E + CTAS - 1) / CTAS, e0 = (int)rank * per, e1 = min(E, e0 + per);
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // (all CTAs have started: waited for below)
  if (tid < kOpMaxExperts / 32) sh.close[tid] = 0;
  if (tid == 0) sh.most = sh.odd = 0;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && tid < 4) p.sync[tid] = 0;
  uint4* const x = reinterpret_cast<uint4*>(raw_x);
  const int vecs = d / 8;
  // (the first weights are on their way while the tokens' rows come in)
  constexpr int U = TT <= 2 ? 8 : 4;
  uint4 u[U];
  const uint16_t* const router = static_cast<const uint16_t*>(p.a.router);
  const uint16_t* w = router + (long long)min(e0 + warp, E - 1) * d;
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
    uint64_t sum[TT], ww = 0;  // products; the row's square
#pragma unroll
    for (int j = 0; j < TT; ++j) sum[j] = 0;
    for (int v = lane; v < vecs; v += 32 * U) {
      if (e != e0 + warp || v != lane) {
        if (v == lane) w = router + (long long)e * d;
        fetch(v);
      }
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (v + 32 * i < vecs) {
          const uint64_t w4[4] = {pair_of(u[i].x), pair_of(u[i].y), pair_of(u[i].z), pair_of(u[i].w)};
#pragma unroll
          for (int k = 0; k < 4; ++k) ww = fma2(w4[k], w4[k], ww);
#pragma unroll
          for (int j = 0; j < TT; ++j) {
            const uint4 y = x[j * vecs + v + 32 * i];
            sum[j] = fma2(w4[3], pair_of(y.w), fma2(w4[2], pair_of(y.z), fma2(w4[1], pair_of(y.y), fma2(w4[0], pair_of(y.x), sum[j]))));
          }
        }
    }
    const float2 w2 = unpack2(ww);
    float wn = w2.x + w2.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) wn += __shfl_xor_sync(0xffffffffu, wn, o);
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      const float2 s2 = unpack2(sum[j]);
      float s = s2.x + s2.y;
#pragma unroll
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0) {
        uint32_t to;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(sh.score + e)), "r"(j));
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(s), "f"(wn) : "memory");
      }
    }
  }
  const int t = t0 + (int)rank, K = p.a.top_k;
  const bool mine_to_select = (int)rank < TT && t < p.a.n_tokens;
  if (mine_to_select) {
    float n = 0.f;
    for (int v = tid; v < vecs; v += kRouterThreads) {
      const uint4 y = x[rank * vecs + v];
      const uint32_t y4[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = bf16x2_to_f2(y4[k]);
        n = fmaf(f.x, f.x, fmaf(f.y, f.y, n));
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0) sh.xn[warp] = n;
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (!mine_to_select) return;
  // A lane adds d / 64 terms (up to 4 more of a step that is not whole) to each of two sums, and 6 additions join them: each is off
  // by 2^-24 of what it adds to at most, |w| |x| in all at most.  Squares below the least float are lost from the norms, each of up to
  // 8192 by 2^-149 at most: kLost; 1.001 covers the norms' roundings, 2^-120 what the products lose in the same way.
  constexpr float kLost = 0x1p-136f;
  float xn = 0.f;
#pragma unroll
  for (int i = 0; i < kRouterWarps; ++i) xn += sh.xn[i];
  const float unit = (d / 64 + 12) * 0x1p-24f * 1.001f * sqrtf(xn + kLost);
  if (tid < kOpMaxExperts) {
    const float off = tid < E ? unit * sqrtf(sh.score[tid].y + kLost) + 0x1p-120f : 0.f;
    if (tid < E) sh.score[tid].y = off;
    const int most = __reduce_max_sync(0xffffffffu, __float_as_int(off));  // (not negative: in the order of the bits)
    if (MANY) {
      reinterpret_cast<float*>(sh.flat)[tid] = tid < E ? sh.score[tid].x : -INFINITY;
      if (tid <= K) sh.best[tid] = NAN;
    }
    const bool odd = tid < E && !(fabsf(sh.score[tid].x) < INFINITY && off < INFINITY);
    if (lane == 0) atomicMax(&sh.most, most);
    if (odd) sh.odd = 1;
  }
  __syncthreads();
  // An expert's rank: how many come before it.  (Two threads an expert, or four where there are few.)
  const int share = kRouterThreads / kOpMaxExperts * (E <= kOpMaxExperts / 2 ? 2 : 1);
  const int e = tid / share, part = tid % share;
  const float2 mine = sh.score[min(e, E - 1)];
  int n = 0;
  bool unsure = true;
  if (MANY) {
    // The larger scores are counted first.  That is it where neighbours among the first ranks lie further apart than two
    // scores can be off together.  (Equal ones leave a rank without a score, a NaN here.  128 experts, 4 tokens: 57.1 us without
    // this, 56.1; 32 experts, 1 token: 12.4 without, 12.8.)
#pragma unroll 4
    for (int f = part; 4 * f < E; f += share) {
      const float4 other = sh.flat[f];
      n += (other.x > mine.x) + (other.y > mine.x) + (other.z > mine.x) + (other.w > mine.x);
    }
    for (int o = share / 2; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (part == 0 && e < E) {
      sh.rank[e] = n;
      if (n <= K) sh.best[n] = mine.x;
    }
    __syncthreads();
    unsure = __syncthreads_or(sh.odd || (tid < K && tid + 1 < E && !(sh.best[tid] - sh.best[tid + 1] > 2.f * __int_as_float(sh.most))));
  }
  if (unsure) {  // every pair with its own errors
    int near = 0;
    n = 0;
#pragma unroll 4
    for (int f = part; f < E; f += share) {
      const float2 other = sh.score[f];
      n += other.x > mine.x || (other.x == mine.x && f < e);
      near |= f != e && !(fabsf(mine.x - other.x) > mine.y + other.y);
    }
    for (int o = share / 2; o; o >>= 1) {
      n += __shfl_xor_sync(0xffffffffu, n, o);
      near |= __shfl_xor_sync(0xffffffffu, near, o);
    }
    if (part == 0 && e < E) {
      sh.rank[e] = n;
      if (n == K) sh.bound = mine.x;
    }
    __syncthreads();
    // Only those that may be among the first K count: not below the score of rank K by more than twice the largest error.  (Where
    // there is no such rank, or NaN among the scores, all of them.)
    near = near && e < E && (sh.odd || K >= E || mine.x >= sh.bound - 2.f * __int_as_float(sh.most));
    if (near && part == 0) atomicOr(sh.close + (e >> 5), 1u << (e & 31));
    if (__syncthreads_or(near)) {
      for (int i = tid; i < E; i += kRouterThreads) sh.key[i] = score_key((double)sh.score[i].x);
      __syncthreads();
      int turn = 0;
      for (int i0 = 0; i0 < E; i0 += 32)
        for (uint32_t left = sh.close[i0 >> 5]; left; left &= left - 1, turn = (turn + 1) % kRouterWarps)
          if (turn == warp) {
            const int i = i0 + __ffs(left) - 1;
            const double s = exact_score(router + (long long)i * d, x + rank * vecs, vecs);
            if (lane == 0) sh.key[i] = score_key(s), sh.score[i].x = (float)s;
          }
      __syncthreads();
      n = 0;
      const unsigned long long key = sh.key[min(e, E - 1)];
      for (int f = part; f < E; f += share) {
        const unsigned long long other = sh.key[f];
        n += other > key || (other == key && f < e);
      }
      for (int o = share / 2; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      if (part == 0 && e < E) sh.rank[e] = n;
      __syncthreads();
    }
  }
  if (tid < E && sh.rank[tid] < K) {
    sh.chosen[sh.rank[tid]] = tid;
    sh.value[sh.rank[tid]] = sh.score[tid].x;
  }
  __syncthreads();
  if (warp == 0) {
    const float mine = lane < K ? __expf(sh.value[lane] - sh.value[0]) : 0.f;
    float total = mine;
#pragma unroll
    for (int o = kMoeTopK / 2; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane < K) {
      p.ids[t * K + lane] = sh.chosen[lane];
      p.weights[t * K + lane] = mine / total;
    }
  }
}

// ------------------------------------------------------------------------------------- few tokens
constexpr int kLayerThreads = 256, kLayerWarps = kLayerThreads / 32;
constexpr int kSpan = 64;         // columns of a copy: one 128-byte swizzle span
constexpr int kStepK = 2 * kSpan;
constexpr int kTileBytes = 4096;  // weights of a step: 16 rows, two copies of 2 KB
constexpr int kGroupBytes = 2048;  // ... and of eight rows of x or h
constexpr int kMaxSlots = 8;      // of a warp's ring

struct LayerShared {
  uint32_t mask[kOpMaxExperts / 32];  // experts that a token has selected
  int act[kOpMaxExperts];             // ... one after another
  int n_act, run, next, abort;
  unsigned long long bars[kLayerWarps][kMaxSlots];
};

// offsets in dynamic shared memory; the same on host and device
struct LayerSmem {
  int rows, red, weight, total;
  __host__ __device__ LayerSmem(int groups, int slots, int d, int entries) {
    rows = kLayerWarps * slots * kTileBytes;  // behind the weights' rings: x, and later the rings for rows of h
    const int x = (d + kStepK - 1) / kStepK * kGroupBytes, h = kLayerWarps * slots * groups * kGroupBytes;
    red = rows + (x > h ? x : h);
    weight = red + kLayerWarps * 32 * 16;
    total = weight + entries * 8 * 4 + 1024;
  }
};

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* tm, int x, int y, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void fence_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }
template <int N>
using Number = std::integral_constant<int, N>;
__device__ __forceinline__ float moe_silu(float y) { return __fdividef(y, 1.f + __expf(-y)); }

// w . h by a warp (the same in every lane), h in its two parts.  For results that are not finite, one at a time: the tiles multiply rows
// of tokens that have not selected an expert, which are zeros, with its weights, and both parts of h, of which one may be zero, and zero
// times infinity is a NaN that the formula does not have.  (What is a NaN stays one: no need to go on.)
__device__ __noinline__ float plain_product(const uint16_t* w, const uint16_t* h, const uint16_t* rest, int f) {
  float y = 0.f;
  for (int i0 = 0; i0 < f; i0 += 256) {
    const int i = i0 + 8 * (threadIdx.x & 31);
    if (i < f) {
      const uint4 a = op_ld16(w + i), b = op_ld16(h + i), c = op_ld16(rest + i);
      const uint32_t a4[4] = {a.x, a.y, a.z, a.w}, b4[4] = {b.x, b.y, b.z, b.w}, c4[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = bf16x2_to_f2(a4[k]), u = bf16x2_to_f2(b4[k]), v = bf16x2_to_f2(c4[k]);
        y = fmaf(x.y, u.y + v.y, fmaf(x.x, u.x + v.x, y));
      }
    }
    if (__any_sync(0xffffffffu, y != y)) return NAN;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
  return y;
}

// Up to 8 tokens.  A tile's rows are the tokens, all of them for every expert, with zeros in h for those that have not selected it: x
// is laid out once, and the second product adds its experts up in registers.  h is kept as a sum of two bf16 values: rounded to one, it
// would be off by as much as the result's own rounding (outputs 1.41 times as far off in the 2-norm).  Up to 4 tokens the second
// values take the other four of eight rows (GROUPS 1), else eight more (2).
template <int GROUPS>
__global__ void __launch_bounds__(kLayerThreads, 1)
    layer_kernel(const __grid_constant__ MoeParams p, const __grid_constant__ CUtensorMap tgate, const __grid_constant__ CUtensorMap tup,
                 const __grid_constant__ CUtensorMap tdown, const __grid_constant__ CUtensorMap th) {
  extern __shared__ uint8_t raw_[];
  __shared__ LayerShared sh;
  const int tid = threadIdx.x, warp = (int)uniform(threadIdx.x >> 5), lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int T = p.a.n_tokens, K = p.a.top_k, d = p.a.d_model, f = p.a.d_ff, entries = T * K, S = p.slots;
  constexpr int kRest = GROUPS == 1 ? 4 : 8;  // rows from a token's first part of h to its second
  const LayerSmem at(GROUPS, S, d, entries);
  const uint32_t base = (smem_u32(raw_) + 1023u) & ~1023u;
  uint8_t* const raw = raw_ + (base - smem_u32(raw_));
  float4* const red = reinterpret_cast<float4*>(raw + at.red);
  float* const weight = reinterpret_cast<float*>(raw + at.weight);  // [active expert][token], -1: not selected
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
  if (tid < kOpMaxExperts / 32) sh.mask[tid] = 0;
  for (int i = tid; i < entries * 8; i += kLayerThreads) weight[i] = -1.f;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  // ---------------------------------------------------------------- who has selected what; x
  if (tid == 0) sh.run = (int)atomicAdd(p.sync, 1u);
  int my_id = 0;
  float my_weight = 0.f;
  if (tid < entries) {
    my_id = op_ld(p.ids + tid);
    my_weight = op_ldf(p.weights + tid);
  }
  const int steps_up = (d + kStepK - 1) / kStepK, steps_down = (f + kStepK - 1) / kStepK;
  const uint32_t tiles_at = base + warp * (S * kTileBytes), rows_at = base + at.rows;
  for (int i = tid; i < steps_up * 128; i += kLayerThreads) {  // 16 bytes each: [step][span][row][8], swizzled
    const int c = i & 7, r = (i >> 3) & 7, span = i / 64, k = span * kSpan + 8 * c;
    if (r < T) {
      const uint16_t* const row = static_cast<const uint16_t*>(p.a.x) + r * p.a.x_stride;
      op_cp16(rows_at + (span * 8 + r) * 128 + ((c ^ r) << 4), k < d ? row + k : row, k < d ? 16 : 0);
    }
  }
  if (tid < entries) atomicOr(sh.mask + (my_id >> 5), 1u << (my_id & 31));
  __syncthreads();
  auto place = [&](int e) {  // of an expert among the active ones
    int n = __popc(sh.mask[e >> 5] & ((1u << (e & 31)) - 1));
    for (int w = 0; w < (e >> 5); ++w) n += __popc(sh.mask[w]);
    return n;
  };
  if (tid < p.a.n_experts) {
    const int a = place(tid);
    if ((sh.mask[tid >> 5] >> (tid & 31)) & 1) sh.act[a] = tid;
    if (tid == p.a.n_experts - 1) sh.n_act = a + ((sh.mask[tid >> 5] >> (tid & 31)) & 1);
  }
  if (tid < entries) weight[place(my_id) * 8 + tid / K] = my_weight;
  __syncthreads();
  const int A = (int)uniform(sh.n_act), groups = f / 8, units = A * groups, runs = (int)gridDim.x;

  // ---------------------------------------------------------------- the warp's ring
  Ring get;
  uint32_t put = 0;
  // where a lane reads its part of a step: 16 rows of weights, 8 rows of x or h (swizzled 128-byte rows)
  const uint32_t r8 = lane & 7, m4 = lane >> 3;
  const uint32_t a_at = tiles_at + (m4 & 1) * 1024 + r8 * 128, a_x = ((m4 >> 1) ^ r8) << 4, b_at = r8 * 128 + ((m4 ^ r8) << 4);

  // First product.  A unit: 8 outputs of an expert; the warps take the units of the CTA's run in turn, all of k each.
  int iu = 0, is = 0, irow = 0, end = 0;  // the issuing side: unit, step, first row; end of the run
  auto unit_row = [&](int u) {
    const int a = u / groups;
    return (int)uniform(sh.act[a] * f + 8 * (u - a * groups));
  };
  // Second product.  Blocks of output columns, this CTA's one after another; the warps deal out the steps of all experts.
  struct Down {
    int block, a, s;
  };
  const int blocks = (d + p.width - 1) / p.width;
  auto down_fit = [&](Down& c) {  // to a step of this warp, if this is none
    while (c.s >= steps_down) {
      c.s -= steps_down;
      if (++c.a >= A) {
        c.block += runs;
        c.a = 0;
        c.s = warp;
        if (c.block >= blocks) return;
      }
    }
  };
  Down id{(int)blockIdx.x, 0, warp}, ib;  // weights; rows
  if (id.block < blocks) down_fit(id);
  ib = id;
  int ahead = 0;  // steps of the second product whose weights are under way and whose rows are not
  const uint32_t down_bytes = 2 * p.width * 128 + GROUPS * kGroupBytes;
  const uint32_t h_at = rows_at + warp * (S * GROUPS * kGroupBytes);

  auto issue_weights = [&]() {
    const int row = (int)uniform(sh.act[id.a] * d + id.block * p.width);
    if (elect_one()) {
      const uint32_t bar = bars + 8 * put, dst = tiles_at + put * kTileBytes;
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
      const uint32_t dst = h_at + slot * (GROUPS * kGroupBytes), bar = bars + 8 * slot;
      tma_box(dst, &th, ib.s * kStepK, ib.a * (8 * GROUPS), bar);
      tma_box(dst + GROUPS * kGroupBytes / 2, &th, ib.s * kStepK + kSpan, ib.a * (8 * GROUPS), bar);
    }
    __syncwarp();
    ib.s += kLayerWarps;
    down_fit(ib);
  };
  int next_run = -1;  // -1: not known yet
  // (at most S steps are under way: a slot is filled again once its step has been multiplied)
  auto issue_next = [&]() {
    if (iu < end) {
      if (elect_one()) {
        const uint32_t bar = bars + 8 * put, dst = tiles_at + put * kTileBytes;
        mbar_expect_tx(bar, kTileBytes);
        tma_box(dst, &tgate, is * kStepK, irow, bar);
        tma_box(dst + 1024, &tup, is * kStepK, irow, bar);
        tma_box(dst + kTileBytes / 2, &tgate, is * kStepK + kSpan, irow, bar);
        tma_box(dst + kTileBytes / 2 + 1024, &tup, is * kStepK + kSpan, irow, bar);
      }
      __syncwarp();
      put = put + 1 == (uint32_t)S ? 0 : put + 1;
      if (++is == steps_up) {
        is = 0;
        iu += kLayerWarps;
        if (iu < end) {
          irow = unit_row(iu);
        } else if (warp == 0 && lane == 0) {
          // (the run is under way: what is left to claim, if anything, is a CTA's that has not started)
          *(volatile int*)&sh.next = (int)atomicAdd(p.sync, 1u);
        }
      }
    } else {
      if (next_run < 0) next_run = (int)uniform((uint32_t)*(volatile int*)&sh.next);
      if (next_run >= runs && id.block < blocks && ahead < S) {
        issue_weights();
        ++ahead;
      }
    }
  };

  // (several sums a tile, so that the products need not wait for one another)
  constexpr int kSets = 4;
  float sum[kSets][4];
  auto clear = [&]() {
#pragma unroll
    for (int k = 0; k < kSets; ++k) sum[k][0] = sum[k][1] = sum[k][2] = sum[k][3] = 0.f;
  };
  // one step with eight rows of x, or GROUPS times eight rows of h
  auto multiply = [&](uint32_t rows, auto groups) {
    constexpr int kGroups = decltype(groups)::value;
    op_wait(bars + 8 * get.slot, get.phase, &sh.abort, p.a.status, 2);
    const uint32_t tile = a_at + get.slot * kTileBytes;
#pragma unroll
    for (int half = 0; half < 4; ++half) {
      uint32_t a[8];
      const uint32_t t = tile + (half >> 1) * (kTileBytes / 2), x = a_x ^ ((half & 1) << 6);
      ldsm_x4(t + x, a[0], a[1], a[2], a[3]);
      ldsm_x4(t + (x ^ 32), a[4], a[5], a[6], a[7]);
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        uint32_t b[4];
        ldsm_x4(rows + (half >> 1) * (kGroups * kGroupBytes / 2) + j * 1024 + (b_at ^ ((half & 1) << 6)), b[0], b[1], b[2], b[3]);
        mma_bf16(sum[(2 * half) % kSets], a[0], a[1], a[2], a[3], b[0], b[1]);
        mma_bf16(sum[(2 * half + 1) % kSets], a[4], a[5], a[6], a[7], b[2], b[3]);
      }
    }
    __syncwarp();
    get.advance(S);
  };
  auto total = [&](int i) { return (sum[0][i] + sum[1][i]) + (sum[2][i] + sum[3][i]); };

  unsigned made = 0;
  bool first = true;
  for (int run = (int)uniform(sh.run); run < runs;) {
    const int u0 = (int)((long long)run * units / runs), u1 = (int)((long long)(run + 1) * units / runs);
    iu = u0 + warp, is = 0, end = u1;
    next_run = -1;
    if (iu < end) irow = unit_row(iu);
    else if (warp == 0 && lane == 0) *(volatile int*)&sh.next = (int)atomicAdd(p.sync, 1u);  // (an empty run)
    for (int i = 0; i < S; ++i) issue_next();
    if (first) {  // x is there
      op_cp_wait_all();
      __syncthreads();
      first = false;
    }
    for (int u = u0 + warp; u < u1; u += kLayerWarps) {
      clear();
      for (int s = 0; s < steps_up; ++s) {
        multiply(rows_at + s * kGroupBytes, Number<1>());
        issue_next();
      }
      const int a = u / groups, col = 8 * (u - a * groups) + g;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * q + i;
        if (t < T) {
          // (c < 0: the token has not selected the expert, and its product does not count, whatever it is)
          const float c = weight[a * 8 + t], y = c * (moe_silu(total(i)) * total(i + 2));
          uint16_t* const h = p.h + (long long)(a * (8 * GROUPS) + t) * f + col;
          h[0] = c < 0.f ? (uint16_t)0 : to_bf16(y);
          h[(long long)kRest * f] = c < 0.f ? (uint16_t)0 : bf16_rest(y);
        }
      }
    }
    made += (unsigned)(u1 - u0);
    // (until the claim is known there may be weights to fetch, but nothing says which)
    __syncthreads();
    run = next_run = (int)uniform((uint32_t)*(volatile int*)&sh.next);
    __syncthreads();
    if (tid == 0) sh.next = -1;
  }
  // ---------------------------------------------------------------- hand over
  op_cp_wait_all();
  for (; ahead < S && id.block < blocks; ++ahead) issue_weights();
  fence_async_global();      // (the results are read by tensor-map copies,
  fence_proxy_async_smem();  // which also write to where x was)
  __syncthreads();
  if (tid == 0) {
    if (made) red_release(p.sync + 1, made);
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
  for (int block = blockIdx.x; block < blocks; block += runs) {
    const int c0 = block * p.width, wide = min(p.width, d - c0), n = A * steps_down;
    clear();
    // (a value a thread: the residual is on its way before its sum is there)
    const int c = tid & 15, t = tid >> 4;
    const bool mine = tid < 128 && t < T && c < wide;
    const uint16_t* const residual = static_cast<const uint16_t*>(p.a.residual);
    const float ahead_y = mine && residual ? bf16_to_f(op_ld2(residual + t * p.a.residual_stride + c0 + c)) : 0.f;
    for (int s = warp; s < n; s += kLayerWarps) {
      multiply(h_at + get.slot * (GROUPS * kGroupBytes), Number<GROUPS>());
      if (id.block < blocks) {
        const uint32_t slot = put;
        issue_weights();
        issue_rows(slot);
      }
    }
    red[warp * 32 + lane] = make_float4(total(0), total(1), total(2), total(3));
    __syncthreads();
    // the warps' parts, in their order
    float y = 0.f;
    if (mine) {
      const int from = (c & 7) * 4 + (t >> 1), part = (t & 1) + 2 * (c >> 3);
#pragma unroll
      for (int w = 0; w < kLayerWarps; ++w) {
        y += reinterpret_cast<const float*>(red + w * 32 + from)[part];
        if (GROUPS == 1) y += reinterpret_cast<const float*>(red + w * 32 + from + kRest / 2)[part];
      }
    }
    for (unsigned odd = __ballot_sync(0xffffffffu, !(fabsf(y) < INFINITY)); odd; odd &= odd - 1) {  // the token's own experts alone
      const int i = 32 * warp + __ffs(odd) - 1, ti = i >> 4, ci = c0 + (i & 15);
      float z = 0.f;
      for (int a = 0; a < A && z == z; ++a)
        if (!(weight[a * 8 + ti] < 0.f)) {
          const uint16_t* const h = p.h + (long long)(a * (8 * GROUPS) + ti) * f;
          z += plain_product(static_cast<const uint16_t*>(p.a.w_down) + ((long long)sh.act[a] * d + ci) * f, h, h + (long long)kRest * f, f);
        }
      if (tid == i) y = z;
    }
    if (mine) {
      if (residual) y += ahead_y;
      static_cast<uint16_t*>(p.a.out)[t * p.a.out_stride + c0 + c] = to_bf16(y);
    }
    __syncthreads();
  }
  if (sh.abort) {  // an abandoned run leaves copies in flight: give them time to land
    const uint64_t s0 = gtime();
    while ((long long)(gtime() - s0) < 10000000ll) {}
  }
}

// ------------------------------------------------------------------------------------ more tokens
// The products of mk_experts.cu between two small kernels: the rows of every expert in order (by expert, then token), and the sum
// of a token's rows.
constexpr int kSortThreads = 1024, kSumThreads = 256;

__global__ void __launch_bounds__(kSortThreads) sort_kernel(const __grid_constant__ MoeParams p) {
  __shared__ uint32_t mask[kOpMaxExperts][kMoeTokens / 32];  // tokens of an expert
  __shared__ int off[kOpMaxExperts], sums[kOpMaxExperts / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, K = p.a.top_k, entries = p.a.n_tokens * K;
  for (int i = tid; i < kOpMaxExperts * (kMoeTokens / 32); i += kSortThreads) mask[0][i] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  constexpr int kMine = kMoeTokens * kMoeTopK / kSortThreads;
  int ids[kMine];
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int i = tid + j * kSortThreads;
    if (i < entries) ids[j] = op_ld(p.ids + i);
  }
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int i = tid + j * kSortThreads, t = i / K;
    if (i < entries) atomicOr(&mask[ids[j]][t >> 5], 1u << (t & 31));
  }
  __syncthreads();
  int n = 0, before = 0;
  if (tid < kOpMaxExperts) {
#pragma unroll
    for (int w = 0; w < kMoeTokens / 32; ++w) n += __popc(mask[tid][w]);
    before = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += a;
    }
    if (lane == 31) sums[warp] = before;
  }
  __syncthreads();
  if (tid < kOpMaxExperts) {
    for (int w = 0; w < warp; ++w) before += sums[w];
    off[tid] = before - n;
    if (tid < p.a.n_experts) p.offsets[tid + 1] = before, p.offsets_h[tid + 1] = 2 * before;
    if (tid == 0) p.offsets[0] = p.offsets_h[0] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int i = tid + j * kSortThreads, t = i / K;
    if (i < entries) {
      int r = off[ids[j]] + __popc(mask[ids[j]][t >> 5] & ((1u << (t & 31)) - 1));
      for (int w = 0; w < (t >> 5); ++w) r += __popc(mask[ids[j]][w]);
      p.rows[r] = t;
      p.places[i] = r;
    }
  }
}

// The four sums of every lane in `odd` once more, from the rows of h (a cold path, so that it takes no registers of the other).
__device__ __noinline__ float4 plain_sums(const MoeParams& p, int t, int c, unsigned odd, float4 y) {
  const int K = p.a.top_k, d = p.a.d_model, f = p.a.d_ff;
  for (; odd; odd &= odd - 1) {
    const int from = __ffs(odd) - 1, c0 = __shfl_sync(0xffffffffu, c, from);
    float v[4];
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      float z = 0.f;
      for (int j = 0; j < K && z == z; ++j) {
        const uint16_t* const h = p.h + (long long)op_ld(p.places + t * K + j) * (2 * f);
        const uint16_t* const w = static_cast<const uint16_t*>(p.a.w_down) + ((long long)op_ld(p.ids + t * K + j) * d + c0 + i) * f;
        z = fmaf(op_ldf(p.weights + t * K + j), plain_product(w, h, h + f, f), z);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i == k) v[k] = z;
    }
    if ((threadIdx.x & 31) == from) y = make_float4(v[0], v[1], v[2], v[3]);
  }
  return y;
}

// out[t] = residual[t] + sum_j c_j y[place of (t, j)], four columns a thread
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const __grid_constant__ MoeParams p) {
  const int t = blockIdx.x, c = 4 * (blockIdx.y * kSumThreads + threadIdx.x), K = p.a.top_k, d = p.a.d_model;
  pdl_wait();
  pdl_trigger();
  LinearEpi epi{};
  epi.residual = static_cast<const uint16_t*>(p.a.residual);
  epi.residual_stride = p.a.residual_stride;
  epi.vec = p.vec;
  const uint2 ahead = linear_residual(epi, t, c, d - c);
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < d) {
#pragma unroll 4
    for (int j = 0; j < K; ++j) {
      const float w = op_ldf(p.weights + t * K + j);
      const uint4 u = op_ld16(p.y + (long long)op_ld(p.places + t * K + j) * d + c);
      v[0] = fmaf(w, __uint_as_float(u.x), v[0]), v[1] = fmaf(w, __uint_as_float(u.y), v[1]);
      v[2] = fmaf(w, __uint_as_float(u.z), v[2]), v[3] = fmaf(w, __uint_as_float(u.w), v[3]);
    }
  }
  const bool fine = fabsf(v[0]) < INFINITY && fabsf(v[1]) < INFINITY && fabsf(v[2]) < INFINITY && fabsf(v[3]) < INFINITY;
  const unsigned odd = __ballot_sync(0xffffffffu, !fine);
  if (odd) {
    const float4 y = plain_sums(p, t, c, odd, make_float4(v[0], v[1], v[2], v[3]));
    v[0] = y.x, v[1] = y.y, v[2] = y.z, v[3] = y.w;
  }
  linear_put<false>(epi, p.a.out, p.a.out_stride, v, ahead, t, c, d - c);
}

// ----------------------------------------------------------------------------------------- launches
template <int TT, int CTAS, bool MANY>
cudaError_t launch_router(const MoeParams& p, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0}, done_wide{0};
  cudaError_t e = allow_smem(router_kernel<TT, CTAS, MANY>, TT * kMoeWidest * 2, done);
  if (e == cudaSuccess && CTAS > 8) e = allow_wide_clusters(router_kernel<TT, CTAS, MANY>, done_wide);
  if (e != cudaSuccess) return e;
  return launch_early(router_kernel<TT, CTAS, MANY>, dim3((unsigned)((p.a.n_tokens + TT - 1) / TT * CTAS)), kRouterThreads, (size_t)TT * p.a.d_model * 2, st, p);
}

template <bool MANY>
cudaError_t launch_router(const MoeParams& p, int tt, cudaStream_t st) {
  return tt == 1   ? launch_router<1, 8, MANY>(p, st)
         : tt == 2 ? launch_router<2, 8, MANY>(p, st)
         : tt == 4 ? launch_router<4, 8, MANY>(p, st)
                   : launch_router<8, 8, MANY>(p, st);
}

size_t align16(size_t n) { return (n + 15) / 16 * 16; }

constexpr int kMostSmem = 232448 - ((int)sizeof(LayerShared) + 127) / 128 * 128;

// slots of a warp's ring that fit: as many as there is room for
int layer_slots(const mk_moe_args& a, int groups) {
  for (int s = kMaxSlots; s >= 2; --s)
    if (LayerSmem(groups, s, a.d_model, a.n_tokens * a.top_k).total <= kMostSmem) return s;
  return 0;
}

template <int GROUPS>
cudaError_t launch_layer(const MoeParams& p, const MoeMaps& m, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(layer_kernel<GROUPS>, kMostSmem, done);
  if (e != cudaSuccess) return e;
  const int smem = LayerSmem(GROUPS, p.slots, p.a.d_model, p.a.n_tokens * p.a.top_k).total;
  return launch_early(layer_kernel<GROUPS>, dim3((unsigned)p.grid), kLayerThreads, (size_t)smem, st, p, m.gate, m.up, m.down, m.h);
}

}  // namespace

// Groups of eight rows of h for a kernel of few tokens, 0: the products of mk_experts.cu.  Up to 8 tokens the one kernel, whose tiles
// waste the fewest products (2048 wide, 128 experts of 768, 8 a token; us of the one kernel / sort, products and sum: 1 token 23.9 / 34.8,
// 4 55.8 / 71.5, 5 73.2 / 75.2, 8 93.5 / 100.1, 16, with 32 rows of h, 167 / 146; of 32 experts of 1024 x 512 1 12.5 / 22.3, 5
// 23.0 / 28.2, 8 25.4 / 33.5; 9 to 16 of those in one kernel have not been measured, in several 9 take 34.9, 16 37.2).
int moe_groups(const mk_moe_args& a) {
  const int groups = a.n_tokens <= 4 ? 1 : a.n_tokens <= kMoeFew ? 2 : 0;
  return groups && a.n_tokens * a.top_k <= kLayerThreads && layer_slots(a, groups) >= 3 ? groups : 0;
}

long long moe_h_rows(const mk_moe_args& a) {
  const long long entries = (long long)a.n_tokens * a.top_k, groups = moe_groups(a);
  return groups ? 8 * groups * std::min<long long>(a.n_experts, entries) : 2 * entries;
}

size_t moe_workspace_bytes(const mk_moe_args& a) {
  const size_t entries = (size_t)a.n_tokens * a.top_k;
  size_t n = 16 + 2 * align16(entries * 4) + align16((size_t)moe_h_rows(a) * a.d_ff * 2);
  if (!moe_groups(a)) n += 2 * align16(entries * 4) + 2 * align16((size_t)(a.n_experts + 1) * 4) + entries * a.d_model * 4;
  return n;
}

void moe_shape(MoeParams& p) {
  const mk_moe_args& a = p.a;
  const size_t entries = (size_t)a.n_tokens * a.top_k;
  uint8_t* at = static_cast<uint8_t*>(a.workspace);
  const auto take = [&](size_t bytes) {
    uint8_t* const here = at;
    at += align16(bytes);
    return here;
  };
  p.groups = moe_groups(a);
  p.sync = reinterpret_cast<uint32_t*>(take(16));
  int32_t* const ids = reinterpret_cast<int32_t*>(take(entries * 4));
  float* const weights = reinterpret_cast<float*>(take(entries * 4));
  p.ids = a.ids ? a.ids : ids;
  p.weights = a.weights ? a.weights : weights;
  p.h = reinterpret_cast<uint16_t*>(take((size_t)moe_h_rows(a) * a.d_ff * 2));
  if (p.groups) {
    p.slots = layer_slots(a, p.groups);
    // output columns: 16 at most, in blocks of equal width over all CTAs
    const int rounds = (a.d_model + 16 * p.grid - 1) / (16 * p.grid);
    p.width = (a.d_model + rounds * p.grid - 1) / (rounds * p.grid);
  } else {
    p.rows = reinterpret_cast<int32_t*>(take(entries * 4));
    p.places = reinterpret_cast<int32_t*>(take(entries * 4));
    p.offsets = reinterpret_cast<int32_t*>(take((size_t)(a.n_experts + 1) * 4));
    p.offsets_h = reinterpret_cast<int32_t*>(take((size_t)(a.n_experts + 1) * 4));
    p.y = reinterpret_cast<float*>(at);
  }
  p.vec = a.out_stride % 4 == 0 && reinterpret_cast<uintptr_t>(a.out) % 8 == 0 &&
          (!a.residual || (a.residual_stride % 4 == 0 && reinterpret_cast<uintptr_t>(a.residual) % 8 == 0));
}

cudaError_t launch_moe_router(const MoeParams& p, cudaStream_t st) {
  // As few tokens a cluster as keep it at one CTA an SM.  For hardly any tokens a cluster of 16 where its CTAs still have 32 KB of
  // weights each (1 token, 128 x 2048: 23.8 us in place of 24.2; 32 x 1024: 13.2 and 12.8).
  const int t = p.a.n_tokens, clusters = std::max(1, p.grid / 8);
  const bool wide = t <= 4 && (long long)p.a.n_experts * p.a.d_model * 2 >= 16 * 32768;
  const int tt = t <= clusters ? 1 : t <= 2 * clusters ? 2 : t <= 4 * clusters ? 4 : 8;
  const cudaError_t e = p.a.n_experts > 64 ? wide ? launch_router<1, 16, true>(p, st) : launch_router<true>(p, tt, st)
                                           : wide ? launch_router<1, 16, false>(p, st) : launch_router<false>(p, tt, st);
  if (e != cudaSuccess || p.groups) return e;
  return launch_early(sort_kernel, dim3(1), kSortThreads, 0, st, p);
}

cudaError_t launch_moe_few(const MoeParams& p, const MoeMaps& m, cudaStream_t st) {
  return p.groups == 1 ? launch_layer<1>(p, m, st) : launch_layer<2>(p, m, st);
}

cudaError_t launch_moe_sum(const MoeParams& p, cudaStream_t st) {
  return launch_early(sum_kernel, dim3((unsigned)p.a.n_tokens, (unsigned)((p.a.d_model + 4 * kSumThreads - 1) / (4 * kSumThreads))), kSumThreads, 0, st, p);
}

}  // namespace mk
