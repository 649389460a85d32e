// The routed layer of a few tokens:  out = residual + sum_j c_j Wd[id_j] (silu(Wg[id_j] x) * (Wu[id_j] x)).
//
// Two kernels.  router_kernel: scores, selection, weights.  layer_kernel: both products, one CTA per SM, with the first product's
// results handed over inside the kernel so that the second one's weights are under way while the last results of the first are
// added up.
//
// With few tokens every selected expert's weights are read for a handful of rows: HBM bounds it, and the products only have to
// keep up.  So the weights go straight from HBM to the lane that multiplies them, without barriers or a shared ring: each
// warp has a ring of its own, filled by 16-byte asynchronous copies, and every lane reads back what it copied itself.
// (m16n8k16 wants pairs of k apart from one another in a lane; since the order of k does not matter to a sum, a lane's 16 bytes
// in a row count as four such pairs, for weights and rows alike.)  The warps split k; their parts of a result meet in
// shared memory and are added in the order of the warps.
//
// First product: a unit is 8 outputs of an expert (8 gate and 8 up rows of weights: one 16-row tile) for up to 8 NT of its
// rows.  The list of units is cut into as many equal runs as there are CTAs, and a CTA claims a run when it starts, so that a
// wait for the first product never waits for a CTA that has yet to start.  Second product: a CTA has up to 16 output
// columns and goes through all experts with them, so that the sum over a token's experts stays in the CTA, in the order
// of the experts: no partial results leave it.
#include "mk_ops.cuh"

namespace mk {
namespace {

// ------------------------------------------------------------------------------------------ router
// A cluster of 8 CTAs has TT tokens and an eighth of the experts a CTA.  A selection can hang on the last bits of two scores, so
// these are sums of exact products (two bf16 factors fit fp32) with the rounding errors of the additions carried along.
constexpr int kRouterCtas = 8, kRouterThreads = 256, kRouterWarps = kRouterThreads / 32;

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
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int t0 = (int)(blockIdx.x / kRouterCtas) * TT, E = p.a.n_experts, d = p.a.d_model;
  const int per = (E + kRouterCtas - 1) / kRouterCtas, e0 = (int)rank * per, e1 = min(E, e0 + per);
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // (all CTAs have started: waited for below)
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && tid < 4) p.sync[tid] = 0;
  const uint16_t* x[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) x[j] = static_cast<const uint16_t*>(p.a.x) + min(t0 + j, p.a.n_tokens - 1) * p.a.x_stride;
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  for (int e = e0 + warp; e < e1; e += kRouterWarps) {
    const uint16_t* const w = static_cast<const uint16_t*>(p.a.router) + (long long)e * d;
    uint64_t hi[TT], lo[TT];
#pragma unroll
    for (int j = 0; j < TT; ++j) hi[j] = lo[j] = 0;
#pragma unroll(TT <= 2 ? 4 : 2)
    for (int k = 8 * lane; k < d; k += 256) {
      const uint4 u = op_ld16(w + k);
      uint4 v[TT];
#pragma unroll
      for (int j = 0; j < TT; ++j) v[j] = op_ld16(x[j] + k);
      const uint64_t w4[4] = {pair_of(u.x), pair_of(u.y), pair_of(u.z), pair_of(u.w)};
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        add_exact2(hi[j], lo[j], mul2(w4[0], pair_of(v[j].x)));
        add_exact2(hi[j], lo[j], mul2(w4[1], pair_of(v[j].y)));
        add_exact2(hi[j], lo[j], mul2(w4[2], pair_of(v[j].z)));
        add_exact2(hi[j], lo[j], mul2(w4[3], pair_of(v[j].w)));
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
constexpr int kStepK = 64;  // columns of a step: two 16-byte pieces a lane and row

template <int NT>
constexpr int kSlots = NT == 1 ? 8 : NT == 2 ? 5 : 3;  // of a warp's ring
template <int NT>
constexpr int kSlotBytes = (4 + 2 * NT) * 32 * 16;
constexpr int kAccPitch = 20;

template <int NT>
struct LayerSmem {  // offsets in dynamic shared memory
  int red, list, weight, acc, ent, total;
  __host__ __device__ LayerSmem(int tokens, int entries) {
    red = kLayerWarps * kSlots<NT> * kSlotBytes<NT>;
    list = red + 2 * kLayerWarps * NT * 32 * 16;            // (the token masks lie here before the first results)
    weight = list + (entries * 2 + 15) / 16 * 16;
    acc = weight + (entries * 4 + 15) / 16 * 16;
    ent = acc + tokens * kAccPitch * 4;
    total = ent + (NT == 1 ? kOpMaxExperts * 8 * 2 : 0);
  }
};

struct LayerShared {
  int off[kOpMaxExperts + 1];    // first row of every expert in the list
  int act[kOpMaxExperts];        // experts that have rows
  int pre[kOpMaxExperts + 1];    // units before each of them
  int tile_pre[kOpMaxExperts + 1];
  int n_act, run, next;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ float moe_silu(float y) { return __fdividef(y, 1.f + __expf(-y)); }

template <int NT>
__global__ void __launch_bounds__(kLayerThreads, 1) layer_kernel(const __grid_constant__ MoeParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ LayerShared sh;
  constexpr int S = kSlots<NT>;
  constexpr bool kDirect = NT == 1;  // second product: a tile's rows are the tokens, and its sums stay in registers
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int T = p.a.n_tokens, K = p.a.top_k, E = p.a.n_experts, d = p.a.d_model, f = p.a.d_ff, entries = T * K;
  const LayerSmem<NT> at(T, entries);
  float4* const red = reinterpret_cast<float4*>(raw + at.red);
  uint32_t* const mask = reinterpret_cast<uint32_t*>(raw + at.red);
  uint16_t* const list = reinterpret_cast<uint16_t*>(raw + at.list);  // token << 4 | slot, by expert, then token
  float* const weight = reinterpret_cast<float*>(raw + at.weight);    // ... and its weight
  float* const acc = reinterpret_cast<float*>(raw + at.acc);
  int16_t* const ent = reinterpret_cast<int16_t*>(raw + at.ent);      // [active expert][token]: its row of h, or -1
  const int words = (T + 31) / 32;

  for (int i = tid; i < E * words; i += kLayerThreads) mask[i] = 0;
  if (kDirect)
    for (int i = tid; i < kOpMaxExperts * 8; i += kLayerThreads) ent[i] = -1;
  for (int i = tid; i < T * kAccPitch; i += kLayerThreads) acc[i] = 0.f;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  // ---------------------------------------------------------------- who has which rows
  if (tid == 0) {
    sh.run = (int)atomicAdd(p.sync, 1u);
    sh.next = -1;
  }
  for (int i = tid; i < entries; i += kLayerThreads) {
    const int t = i / K;
    atomicOr(mask + op_ld(p.ids + i) * words + (t >> 5), 1u << (t & 31));
  }
  __syncthreads();
  if (warp == 0) {
    // (one warp: the experts in order, 32 at a time)
    int rows = 0, tiles = 0, active = 0;
    for (int base = 0; base < E; base += 32) {
      const int e = base + lane;
      int n = 0;
      if (e < E)
        for (int w = 0; w < words; ++w) n += __popc(mask[e * words + w]);
      const int k = (n + 8 * NT - 1) / (8 * NT);
      int r = n, c = k;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, r, o), b = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) r += a, c += b;
      }
      const unsigned some = __ballot_sync(0xffffffffu, n > 0);
      const int idx = active + __popc(some & ((1u << lane) - 1));
      if (e < E) sh.off[e] = rows + r - n;
      if (n > 0) {
        sh.act[idx] = e;
        sh.tile_pre[idx] = tiles + c - k;
      }
      rows += __shfl_sync(0xffffffffu, r, 31);
      tiles += __shfl_sync(0xffffffffu, c, 31);
      active += __popc(some);
    }
    if (lane == 0) {
      sh.off[E] = rows;
      sh.tile_pre[active] = tiles;
      sh.n_act = active;
    }
  }
  __syncthreads();
  const int A = sh.n_act, groups = f / 8;
  for (int i = tid; i < entries; i += kLayerThreads) {
    const int t = i / K, e = op_ld(p.ids + i);
    int r = sh.off[e];
    for (int w = 0; w < (t >> 5); ++w) r += __popc(mask[e * words + w]);
    r += __popc(mask[e * words + (t >> 5)] & ((1u << (t & 31)) - 1));
    list[r] = (uint16_t)(t << 4 | (i - t * K));
    weight[r] = op_ldf(p.weights + i);
    if (kDirect) {
      int lo = 0;  // the expert's place among the active ones
#pragma unroll
      for (int step = kOpMaxExperts / 2; step; step >>= 1)
        if (lo + step < A && sh.act[lo + step] <= e) lo += step;
      ent[lo * 8 + t] = (int16_t)i;
    }
  }
  __syncthreads();
  const long long units = (long long)sh.tile_pre[A] * groups;
  const int runs = (int)gridDim.x;

  // ---------------------------------------------------------------- the warp's ring
  const uint32_t ring = smem_u32(raw) + warp * (S * kSlotBytes<NT>) + lane * 16;
  const uint8_t* const ring_g = raw + warp * (S * kSlotBytes<NT>) + lane * 16;
  uint32_t put = 0, get = 0;  // slots, modulo S
  auto bump = [](uint32_t& s) { s = s + 1 == (uint32_t)S ? 0u : s + 1; };

  // ---------------------------------------------------------------- first product
  struct Up {             // a place in the list of units
    int left;             // units of the run from here on, this one included
    int a, g, tile, tiles, e, n;   // active expert, group of outputs, row tile (of tiles), the expert, its rows
  };
  auto up_at = [&](long long u, int left) {
    Up c;
    c.left = left;
    if (left <= 0) return c;
    int lo = 0;
#pragma unroll
    for (int step = kOpMaxExperts / 2; step; step >>= 1)
      if (lo + step < A && (long long)sh.tile_pre[lo + step] * groups <= u) lo += step;
    c.a = lo;
    c.e = sh.act[lo];
    c.n = sh.off[c.e + 1] - sh.off[c.e];
    c.tiles = sh.tile_pre[lo + 1] - sh.tile_pre[lo];
    const int rem = (int)(u - (long long)sh.tile_pre[lo] * groups);
    c.g = rem / c.tiles;
    c.tile = rem - c.g * c.tiles;
    return c;
  };
  auto up_next = [&](Up& c) {
    if (--c.left <= 0) return;
    if (++c.tile < c.tiles) return;
    c.tile = 0;
    if (++c.g < groups) return;
    c.g = 0;
    ++c.a;
    c.e = sh.act[c.a];
    c.n = sh.off[c.e + 1] - sh.off[c.e];
    c.tiles = sh.tile_pre[c.a + 1] - sh.tile_pre[c.a];
  };
  const int steps_up = (d + kStepK - 1) / kStepK, steps_down = (f + kStepK - 1) / kStepK;
  const uint16_t *a0 = nullptr, *a1 = nullptr, *rows[NT];  // where the lane's pieces come from (the issuing side's)
  auto up_rows = [&](const Up& c) {
    const long long r = ((long long)c.e * f + 8 * c.g + g) * d;
    a0 = static_cast<const uint16_t*>(p.a.w_gate) + r;
    a1 = static_cast<const uint16_t*>(p.a.w_up) + r;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int n = (c.tile * NT + j) * 8 + g;
      rows[j] = n < c.n ? static_cast<const uint16_t*>(p.a.x) + (list[sh.off[c.e] + n] >> 4) * p.a.x_stride : nullptr;
    }
  };
  auto copy = [&](uint32_t dst, const uint16_t* row, int k, int width) {
    cp16(dst, k < width ? row + k : row, k < width ? 16 : 0);
    cp16(dst + 512, k + 32 < width ? row + k + 32 : row, k + 32 < width ? 16 : 0);
  };
  Up is{}, cs{};   // issuing and consuming sides
  int istep = warp;
  auto run_begin = [&](int r) {
    const long long u0 = r * units / runs, u1 = (r + 1) * units / runs;
    cs = is = up_at(u0, (int)(u1 - u0));
    istep = warp;
    if (is.left > 0) up_rows(is);
  };

  // ---------------------------------------------------------------- second product
  // Blocks of output columns, this CTA's one after another; per block the active experts' tiles, of each the steps.  With
  // kDirect the steps of all experts form one list that the warps deal out, else the warps deal out those of a tile.
  struct Down {
    int block, a, tile, s;
    bool more;
  };
  const int blocks = (d + p.width - 1) / p.width;
  auto down_fit = [&](Down& c) {  // the next place at or behind this one that has a step for this warp
    while (c.block < blocks) {
      if (c.s < steps_down) return;
      if (kDirect) {
        c.s -= steps_down;
        ++c.a;
      } else {
        c.s = warp;
        if (++c.tile >= sh.tile_pre[c.a + 1] - sh.tile_pre[c.a]) c.tile = 0, ++c.a;
        if (c.s >= steps_down && c.a < A) continue;
      }
      if (c.a >= A) {
        c.block += (int)gridDim.x;
        c.a = c.tile = 0;
        c.s = warp;
        if (c.s >= steps_down && !kDirect) c.block = blocks;  // (a warp without steps)
      }
    }
  };
  auto down_begin = [&]() {
    Down c{(int)blockIdx.x, 0, 0, warp, true};
    if (!kDirect && warp >= steps_down) c.block = blocks;
    down_fit(c);
    return c;
  };
  auto down_next = [&](Down& c) {
    c.s += kLayerWarps;
    down_fit(c);
  };
  auto down_weights = [&](const Down& c, uint32_t slot) {
    const int c0 = c.block * p.width, wide = min(p.width, d - c0), k = c.s * kStepK + 8 * q;
    const uint16_t* const w = static_cast<const uint16_t*>(p.a.w_down) + ((long long)sh.act[c.a] * d + c0 + g) * f;
    const uint32_t dst = ring + slot * kSlotBytes<NT>;
    if (g < wide) copy(dst, w, k, f);
    if (g + 8 < wide) copy(dst + 1024, w + 8ll * f, k, f);
  };
  auto down_rows = [&](const Down& c, uint32_t slot) {
    const int k = c.s * kStepK + 8 * q;
    const uint32_t dst = ring + slot * kSlotBytes<NT> + 2048;
    if (kDirect) {
      const int i = ent[c.a * 8 + g];
      const uint16_t* const row = p.h + (long long)max(i, 0) * f;
      cp16(dst, i >= 0 && k < f ? row + k : row, i >= 0 && k < f ? 16 : 0);
      cp16(dst + 512, i >= 0 && k + 32 < f ? row + k + 32 : row, i >= 0 && k + 32 < f ? 16 : 0);
    } else {
      const int e = sh.act[c.a], o = sh.off[e], n = sh.off[e + 1] - o;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int r = (c.tile * NT + j) * 8 + g;
        if (r < n) {
          const int x = list[o + r];
          copy(dst + j * 1024, p.h + (long long)((x >> 4) * K + (x & 15)) * f, k, f);
        }
      }
    }
  };
  Down id = down_begin(), first_down = id;
  int ahead = 0;  // steps of the second product whose weights are under way

  // ---------------------------------------------------------------- issue one step of what comes next
  int next_run = -1;  // -1: not known yet
  auto issue_first = [&]() {
    if (is.left > 0 && istep < steps_up) {
      const int k = istep * kStepK + 8 * q;
      const uint32_t dst = ring + put * kSlotBytes<NT>;
      copy(dst, a0, k, d);
      copy(dst + 1024, a1, k, d);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        if (rows[j]) copy(dst + 2048 + j * 1024, rows[j], k, d);
      bump(put);
      istep += kLayerWarps;
      if (istep >= steps_up) {
        istep = warp;
        up_next(is);
        if (is.left > 0) up_rows(is);
      }
    } else if (next_run >= runs && id.block < blocks && ahead < S) {
      down_weights(id, put);
      bump(put);
      down_next(id);
      ++ahead;
    }
    op_cp_commit();
  };

  float sum[NT][4];
  auto multiply = [&](int nt) {
    const uint8_t* const s = ring_g + get * kSlotBytes<NT>;
    const uint4 g0 = *reinterpret_cast<const uint4*>(s), g1 = *reinterpret_cast<const uint4*>(s + 512);
    const uint4 u0 = *reinterpret_cast<const uint4*>(s + 1024), u1 = *reinterpret_cast<const uint4*>(s + 1536);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (j >= nt) break;
      const uint4 b0 = *reinterpret_cast<const uint4*>(s + 2048 + j * 1024), b1 = *reinterpret_cast<const uint4*>(s + 2560 + j * 1024);
      mma_bf16(sum[j], g0.x, u0.x, g0.y, u0.y, b0.x, b0.y);
      mma_bf16(sum[j], g0.z, u0.z, g0.w, u0.w, b0.z, b0.w);
      mma_bf16(sum[j], g1.x, u1.x, g1.y, u1.y, b1.x, b1.y);
      mma_bf16(sum[j], g1.z, u1.z, g1.w, u1.w, b1.z, b1.w);
    }
    bump(get);
  };
  auto clear = [&]() {
#pragma unroll
    for (int j = 0; j < NT; ++j) sum[j][0] = sum[j][1] = sum[j][2] = sum[j][3] = 0.f;
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
      if (j < nt) red[((buf * kLayerWarps + warp) * NT + j) * 32 + lane] = make_float4(sum[j][0], sum[j][1], sum[j][2], sum[j][3]);
    __syncthreads();
  };

  // (the ring is at most S steps ahead: a slot is filled again after its step has been multiplied, by the lane that read it)
  int buf = 0;
  long long made = 0;
  for (int run = sh.run; run < runs;) {
    run_begin(run);
    next_run = -1;
    const int all = cs.left, middle = all / 2;
    for (int i = 0; i < S - 1; ++i) issue_first();
    while (cs.left > 0) {
      if (tid == 0 && all - cs.left == middle) sh.next = (int)atomicAdd(p.sync, 1u);
      const int nt = min(NT, (cs.n - cs.tile * NT * 8 + 7) / 8);
      clear();
      for (int s = warp; s < steps_up; s += kLayerWarps) {
        issue_first();
        op_cp_wait<S - 1>();
        multiply(nt);
      }
      hand_in(buf, nt);
      next_run = (int)uniform((uint32_t)*(volatile int*)&sh.next);
      const int j = (warp - cs.left) & (kLayerWarps - 1);
      if (j < nt) {
        const float4 y = add_up(buf, j);
        const int r0 = (cs.tile * NT + j) * 8 + 2 * q, o = sh.off[cs.e];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (r0 + i < cs.n) {
            const int x = list[o + r0 + i];
            const float gate = i ? y.y : y.x, up = i ? y.w : y.z;
            p.h[(long long)((x >> 4) * K + (x & 15)) * f + 8 * cs.g + g] = to_bf16(weight[o + r0 + i] * (moe_silu(gate) * up));
          }
      }
      buf ^= 1;
      up_next(cs);
      ++made;
    }
    // (a run without units has claimed nothing more)
    if (all == 0 && tid == 0) sh.next = (int)atomicAdd(p.sync, 1u);
    op_cp_wait_all();
    __syncthreads();
    run = next_run = sh.next;
    __syncthreads();
    if (tid == 0) sh.next = -1;
  }
  // ---------------------------------------------------------------- hand over
  for (; ahead < S && id.block < blocks; ++ahead) {
    down_weights(id, put);
    bump(put);
    down_next(id);
  }
  op_cp_commit();
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
  {
    Down c = first_down;
    uint32_t slot = get;
    for (int i = 0; i < ahead; ++i) {
      down_rows(c, slot);
      bump(slot);
      down_next(c);
    }
    op_cp_commit();
    op_cp_wait_all();
  }
  auto issue_second = [&]() {
    if (id.block < blocks) {
      down_weights(id, put);
      down_rows(id, put);
      bump(put);
      down_next(id);
    }
    op_cp_commit();
  };
  int ready = ahead;  // steps that are known to be there
  auto take = [&](int nt) {
    if (ready > 0) {
      --ready;
    } else {
      op_cp_wait<S - 1>();
    }
    multiply(nt);
    issue_second();
  };

  for (int block = blockIdx.x; block < blocks; block += (int)gridDim.x) {
    const int c0 = block * p.width, wide = min(p.width, d - c0);
    clear();
    if (kDirect) {
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
        const int e = sh.act[a], o = sh.off[e], n = sh.off[e + 1] - o, tiles = sh.tile_pre[a + 1] - sh.tile_pre[a];
        for (int tile = 0; tile < tiles; ++tile) {
          const int nt = min(NT, (n - tile * NT * 8 + 7) / 8);
          clear();
          for (int s = warp; s < steps_down; s += kLayerWarps) take(nt);
          hand_in(buf, nt);
          const int j = (warp - a) & (kLayerWarps - 1);
          if (j < nt) {
            const float4 y = add_up(buf, j);
            const float v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = (tile * NT + j) * 8 + 2 * q + (i & 1);
              if (r < n) acc[(list[o + r] >> 4) * kAccPitch + g + 8 * (i >> 1)] += v[i];
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
  op_cp_wait_all();
}

template <int NT>
cudaError_t launch_layer(const MoeParams& p, cudaStream_t st) {
  const int smem = LayerSmem<NT>(p.a.n_tokens, p.a.n_tokens * p.a.top_k).total;
  constexpr int kMost = NT == 1 ? 8 : NT == 2 ? 64 : kMoeTokens;  // tokens of this form
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(layer_kernel<NT>, LayerSmem<NT>(kMost, kMost * kMoeTopK).total, done);
  if (e != cudaSuccess) return e;
  return launch_early(layer_kernel<NT>, dim3((unsigned)p.grid), kLayerThreads, (size_t)smem, st, p);
}

template <int TT>
cudaError_t launch_router(const MoeParams& p, cudaStream_t st) {
  return launch_early(router_kernel<TT>, dim3((unsigned)((p.a.n_tokens + TT - 1) / TT * kRouterCtas)), kRouterThreads, 0, st, p);
}

size_t align16(size_t n) { return (n + 15) / 16 * 16; }

}  // namespace

size_t moe_workspace_bytes(const mk_moe_args& a) {
  const size_t entries = (size_t)a.n_tokens * a.top_k;
  return 16 + 2 * align16(entries * 4) + align16(entries * a.d_ff * 2);
}

cudaError_t launch_moe(const MoeParams& args, cudaStream_t st) {
  MoeParams p = args;
  const size_t entries = (size_t)p.a.n_tokens * p.a.top_k;
  uint8_t* at = static_cast<uint8_t*>(p.a.workspace);
  p.sync = reinterpret_cast<uint32_t*>(at);
  at += 16;
  p.ids = p.a.ids ? p.a.ids : reinterpret_cast<int32_t*>(at);
  at += align16(entries * 4);
  p.weights = p.a.weights ? p.a.weights : reinterpret_cast<float*>(at);
  at += align16(entries * 4);
  p.h = reinterpret_cast<uint16_t*>(at);
  // output columns: 16 at most, in blocks of equal width over all CTAs
  p.rounds = (p.a.d_model + 16 * p.grid - 1) / (16 * p.grid);
  p.width = (p.a.d_model + p.rounds * p.grid - 1) / (p.rounds * p.grid);
  const int t = p.a.n_tokens, clusters = 2 * p.grid / kRouterCtas;
  cudaError_t e = t <= clusters       ? launch_router<1>(p, st)
                  : t <= 2 * clusters ? launch_router<2>(p, st)
                  : t <= 4 * clusters ? launch_router<4>(p, st)
                                      : launch_router<8>(p, st);
  if (e != cudaSuccess) return e;
  return t <= 8 ? launch_layer<1>(p, st) : t <= 64 ? launch_layer<2>(p, st) : launch_layer<4>(p, st);
}

}  // namespace mk
