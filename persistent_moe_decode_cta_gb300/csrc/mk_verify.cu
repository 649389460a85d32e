// Verification of drafted tokens.  A child i with token x of node v is accepted if u_i q(x) < r(x), where r = p at first and
// r <- (r - q)+ / sum (r - q)+ after a rejection; the next token is drawn from what is left where no child is accepted.
//
// Two kernels.  row_kernel reads the logits of every node that has children once, in pieces, for the largest and the sum of the
// exponentials: all that the tests of first children need beside two numbers a child.  walk_kernel has a cluster of CTAs per
// sequence that walks from the root: an accepted child costs no more than a look at shared memory; at the first rejection in a
// row (or at the last node) the cluster reads that row, out of L2 where it has been read, and from then on keeps the row's
// exponentials in shared memory, a piece a CTA.  The drafting model's rows are read only where one of its tokens was rejected.
// Siblings of proposed tokens (no probabilities) need no row, only what the rejected ones had.
//
// Numbers.  The drawn token is where a running sum over up to 2^18 probabilities passes u times the whole: errors of fp32 would
// move borders enough to change one draw of a few hundred.  So the exponentials of the walk are 64-bit integers (2^-44 of the
// largest, right to 2^-32 of themselves), and their sums are exact: neither order nor split matters.  A verdict is one of those
// numbers too: where the fp32 sum of row_kernel, to 2^-15, does not tell, the row is added up first.  With R the integers
// left and W their sum, r = R / W, and a rejection leaves (R - q W)+: in terms of the row's exponentials E
// R = (E - q A)+ where A grows by W with every rejection; E is kept and A is one number, a double: W is up to 2^62 (2^18 tokens as
// likely as the largest), and 511 siblings can be rejected in one row.
//
// Measured in a graph (float32, 151936 tokens): 8 chains of 9 nodes 28 us, of them the rows 9 (39 MB), the rest the longest walk's chain:
// nodes 2.5, steps 1 to 2, the row out of L2 and its exponentials 4 to 5, every meeting of the cluster 0.5, a cut 2, the draw 0.5;
// 16 trees of 32 nodes 73 us (rows 33, 161 MB); bf16, 8 trees of 16 22 us; 5 nodes of 32000 tokens 12 us.
#include "mk_ops.cuh"

namespace mk {
namespace {

constexpr int kRowThreads = 256, kRowValues = 32;  // values a thread
constexpr int kWalkThreads = 512, kWalkWarps = kWalkThreads / 32;
constexpr int kWalkCtas = 16;              // of a cluster at most
constexpr int kFixed = 44;                 // fraction bits of an exponential
constexpr int kBlock = 128;                // elements that a warp takes at a time: four a lane
constexpr int kWalkSmem = 232448 - 8192;   // dynamic shared memory at most

__device__ __forceinline__ float load_logit(const void* p, long long at, bool f32) {
  return f32 ? op_ldf(static_cast<const float*>(p) + at) : bf16_to_f(op_ld2(static_cast<const uint16_t*>(p) + at));
}

// Elements at .. at + 3 of a row of `n` (beyond it: `fill`), in one access where the row's address allows it.
__device__ __forceinline__ float4 load4(const void* row, int at, int n, bool f32, bool wide, float fill) {
  if (wide && at + 4 <= n) {
    if (f32) {
      const uint4 u = op_ld16(static_cast<const float*>(row) + at);
      return make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
    }
    const uint2 u = op_ld8(static_cast<const uint16_t*>(row) + at);
    const float2 a = bf16x2_to_f2(u.x), b = bf16x2_to_f2(u.y);
    return make_float4(a.x, a.y, b.x, b.y);
  }
  float4 v;
  v.x = at < n ? load_logit(row, at, f32) : fill;
  v.y = at + 1 < n ? load_logit(row, at + 1, f32) : fill;
  v.z = at + 2 < n ? load_logit(row, at + 2, f32) : fill;
  v.w = at + 3 < n ? load_logit(row, at + 3, f32) : fill;
  return v;
}
__device__ __forceinline__ bool is_wide(const void* row, bool f32) { return (reinterpret_cast<uintptr_t>(row) & (f32 ? 15 : 7)) == 0; }

__device__ __forceinline__ const void* logit_row(const mk_verify_args& a, int b, int node) {
  const long long at = b * a.logits_stride[0] + node * a.logits_stride[1];
  return a.logits_float ? static_cast<const void*>(static_cast<const float*>(a.logits) + at)
                        : static_cast<const void*>(static_cast<const uint16_t*>(a.logits) + at);
}

// log2(e) / temperature as a sum of two floats, to 2^-46; a temperature of 0 (the largest logit alone counts) reads as 1 here
struct Heat {
  float t, hi, lo;
  __device__ __forceinline__ explicit Heat(float temperature) : t(temperature) {
    const float x = t > 0.f ? fminf(fmaxf(t, 1e-30f), 1e30f) : 1.f;
    const float r = 1.f / x, e = fmaf(-r, x, 1.f) * r;  // 1 / x = r + e
    constexpr float kH = 1.44269502162933349609375f, kL = 1.92596299112661746887e-8f;
    hi = __fmul_rn(kH, r);
    lo = fmaf(kH, r, -hi) + fmaf(kH, e, kL * r);
  }
};
__device__ __forceinline__ float temperature(const mk_verify_args& a, int b) { return a.temperature ? op_ldf(a.temperature + b) : 1.f; }
__device__ __forceinline__ int node_count(const mk_verify_args& a, int b) { return a.counts ? op_ld(a.counts + b) : a.n_nodes; }

// -------------------------------------------------------------------------------------------- rows
// Largest and sum of exponentials of two sets of logits, as those of their union.
struct Peak {
  float top, sum;
  int arg;
  __device__ __forceinline__ void merge(float t, float s, int a, float beta) {
    const float all = fmaxf(top, t);
    const float from = all == -INFINITY ? 0.f : all;  // (two empty sets)
    sum = sum * ex2((top - from) * beta) + s * ex2((t - from) * beta);
    arg = t > top ? a : t == top ? min(a, arg) : arg;
    top = all;
  }
};

// One block per piece of a row: {largest, sum of exp((l - largest) / T), index of the largest (the lowest; at temperature 0, where
// the sum only tells whether there is a NaN)}.  Its loads and instructions bound it: 4.5 TB/s and 60 % of the issue slots (161 MB in
// 35.6 us, the rows with children of 16 trees of 32 nodes).  32 values a thread, all of them on their way at once.  (Half as many:
// 49 us in place of 42 for all rows of those trees; a ring of bulk copies a warp: 52.)
template <bool F32>
__global__ void __launch_bounds__(kRowThreads) row_kernel(const __grid_constant__ VerifyParams p) {
  constexpr int kVec = F32 ? 4 : 8;  // elements of 16 bytes
  constexpr int kRowLoads = kRowValues / kVec;
  __shared__ Peak s_peak[kRowThreads / 32];
  const int piece = blockIdx.x, node = blockIdx.y, b = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const int count = node_count(p.a, b);
  if (node >= count) return;
  // a node without children: its row matters only where the walk ends there, and the walk looks at it by itself
  bool inner = !p.a.parents && node + 1 < count;
  if (p.a.parents)
    for (int j = node + 1 + lane; j < min(count, p.a.n_nodes); j += 32) inner |= op_ld(p.a.parents + (long long)b * p.a.n_nodes + j) == node;
  if (!__any_sync(0xffffffffu, inner)) return;
  const uint8_t* const row = static_cast<const uint8_t*>(logit_row(p.a, b, node));
  const Heat heat(temperature(p.a, b));
  const float beta = heat.hi;
  const bool greedy = heat.t == 0.f, wide = (reinterpret_cast<uintptr_t>(row) & 15) == 0;
  const int n = p.a.vocab, at = piece * kRowThreads * kRowValues + kVec * threadIdx.x;
  uint32_t u[kRowLoads][4];
#pragma unroll
  for (int i = 0; i < kRowLoads; ++i) {
    const int j = at + i * kRowThreads * kVec;
    if (wide && j + kVec <= n) {
      const uint4 w = op_ld16(row + (long long)j * (F32 ? 4 : 2));
      u[i][0] = w.x, u[i][1] = w.y, u[i][2] = w.z, u[i][3] = w.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) u[i][k] = F32 ? 0xff800000u : 0xff80ff80u;  // (-infinity)
    }
  }
  if (!wide || at + (kRowLoads - 1) * kRowThreads * kVec + kVec > n) {  // what is no whole vector, value by value
#pragma unroll
    for (int i = 0; i < kRowLoads; ++i) {
      const int j = at + i * kRowThreads * kVec;
      if (wide && j + kVec <= n) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (F32) {
          if (j + k < n) u[i][k] = __float_as_uint(load_logit(row, j + k, true));
        } else {
          if (j + 2 * k < n) u[i][k] = (u[i][k] & 0xffff0000u) | op_ld2(row + 2ll * (j + 2 * k));
          if (j + 2 * k + 1 < n) u[i][k] = (u[i][k] & 0xffffu) | (uint32_t)op_ld2(row + 2ll * (j + 2 * k + 1)) << 16;
        }
      }
    }
  }
  // the thread's largest first (a running one, rescaled at every vector: 8 x 9 nodes 33.1 us in place of 32.0 with the walk)
  Peak mine{-INFINITY, 0.f, 0x7fffffff};
#pragma unroll
  for (int i = 0; i < kRowLoads; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (F32) {
        mine.top = fmaxf(mine.top, __uint_as_float(u[i][k]));
      } else {
        const float2 f = bf16x2_to_f2(u[i][k]);
        mine.top = fmaxf(mine.top, fmaxf(f.x, f.y));
      }
    }
  const float from = mine.top == -INFINITY ? 0.f : mine.top;
#pragma unroll
  for (int i = 0; i < kRowLoads; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (F32) {
        mine.sum += ex2((__uint_as_float(u[i][k]) - from) * beta);
      } else {
        const float2 f = bf16x2_to_f2(u[i][k]);
        mine.sum += ex2((f.x - from) * beta) + ex2((f.y - from) * beta);
      }
    }
  if (greedy) {
#pragma unroll
    for (int i = kRowLoads - 1; i >= 0; --i)
#pragma unroll
      for (int k = 3; k >= 0; --k) {
        const int j = at + i * kRowThreads * kVec;
        if (F32) {
          if (__uint_as_float(u[i][k]) == mine.top) mine.arg = j + k;
        } else {
          const float2 f = bf16x2_to_f2(u[i][k]);
          if (f.y == mine.top) mine.arg = j + 2 * k + 1;
          if (f.x == mine.top) mine.arg = j + 2 * k;
        }
      }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1)
    mine.merge(__shfl_xor_sync(0xffffffffu, mine.top, o), __shfl_xor_sync(0xffffffffu, mine.sum, o), __shfl_xor_sync(0xffffffffu, mine.arg, o), beta);
  if (lane == 0) s_peak[warp] = mine;
  __syncthreads();
  if (warp == 0) {
    mine = s_peak[lane % (kRowThreads / 32)];
#pragma unroll
    for (int o = kRowThreads / 64; o; o >>= 1)
      mine.merge(__shfl_xor_sync(0xffffffffu, mine.top, o), __shfl_xor_sync(0xffffffffu, mine.sum, o), __shfl_xor_sync(0xffffffffu, mine.arg, o),
                 beta);
    if (lane == 0) p.parts[((long long)b * p.a.n_nodes + node) * p.pieces + piece] = make_float4(mine.top, mine.sum, __int_as_float(mine.arg), 0.f);
  }
}

// ------------------------------------------------------------------------------------- exponentials
// 2^(i/512), i = 0 .. 511, in units of 2^-62
constexpr int kPowers = 512;
struct Powers {
  unsigned long long v[kPowers];
  constexpr Powers() : v() {
    for (int i = 0; i < kPowers; ++i) {
      const double x = i / 512.0 * 0.69314718055994530942;
      double y = 1;
      for (int k = 22; k > 0; --k) y = 1 + x / k * y;  // the exponential series
      v[i] = (unsigned long long)(y * 4503599627370496.0 + 0.5) << 10;
    }
  }
};
__device__ const Powers powers = Powers();

struct U2 {
  unsigned long long x, y;
};
__device__ __forceinline__ uint64_t both(float v) { return pack2(v, v); }
// (adding 1.5 * 2^23 rounds to an integer and leaves it in the low bits)
constexpr float kMagic = 12582912.f;
__device__ __forceinline__ int low_bits(float v) { return __float_as_int(v) - 0x4b400000; }

// exp((l - top) / T) in units of 2^-44 of two logits at once, for finite l <= top to 2^-32 of itself; 0 for anything else.  top: the
// row's largest logit; bh + bl: log2(e) / T.  (With packed operations, which are rounded one by one, whatever follows them.  To 2^-41
// it took 1.5 times the instructions: 8 x 9 nodes 30.4 us with that and a row's copies in one piece, 28.3 with this and two halves.
// What is off is a random 2^-35.5 in the mean: of 10^6 draws from 2^17 tokens it moves about one.)
__device__ __forceinline__ U2 exp_fixed(float l0, float l1, float top, float bh, float bl, const unsigned long long* table) {
  const uint64_t minus = both(-1.f), l = pack2(l0, l1), b = both(bh);
  // l - top as dh + dl, exactly; times log2(e) / T as pl - np, np at most 46: beyond that nothing is left (nor of NaN)
  const uint64_t dh = add2(l, both(-top)), z = fma2(l, minus, dh);
  const uint64_t dl = fma2(add2(both(top), z), minus, fma2(fma2(z, minus, dh), minus, l));
  const float2 n2 = unpack2(mul2(dh, both(-bh)));
  const uint64_t np = pack2(fminf(n2.x, 46.f), fminf(n2.y, 46.f)), pl = fma2(dh, both(bl), fma2(dl, b, fma2(dh, b, np)));
  // -np = k / 512 - nr, exactly; y = 1024 (pl - nr) ln 2, |y| < 0.69; e = 1024 (exp(y / 1024) - 1) by its series
  constexpr float kLn2 = 1024 * 0.693147182464599609375f;
  const uint64_t m = fma2(np, both(-512.f), both(kMagic)), nr = fma2(add2(m, both(-kMagic)), both(1.f / 512.f), np);
  const uint64_t y = fma2(nr, both(-kLn2), mul2(pl, both(kLn2)));
  const uint64_t e = fma2(mul2(y, y), fma2(y, both(0x1p-20f / 6), both(0x1p-11f)), y);
  // the table's entry t plus t e, the latter as an integer of 2^-40
  const float2 mf = unpack2(m);
  const uint32_t k0 = __float_as_uint(mf.x), k1 = __float_as_uint(mf.y);  // k + 0x4b400000
  const unsigned long long t0 = table[k0 & 511], t1 = table[k1 & 511];
  const float2 w = unpack2(mul2(pack2((float)(uint32_t)(t0 >> 32), (float)(uint32_t)(t1 >> 32)), e));
  const unsigned long long v0 = t0 + (unsigned long long)((long long)__float2int_rn(w.x) * (1ll << 22));
  const unsigned long long v1 = t1 + (unsigned long long)((long long)__float2int_rn(w.y) * (1ll << 22));
  // (shifted by 62 - 44 and the whole part of k / 512, rounded)
  constexpr uint32_t kShift = 61 - kFixed + (0x4b400000u >> 9);
  return U2{((v0 >> (kShift - (k0 >> 9) & 63)) + 1) >> 1, ((v1 >> (kShift - (k1 >> 9) & 63)) + 1) >> 1};
}
// (of single logits: one copy of the code, since a cold kernel waits for its instructions longer than it runs them)
__device__ __noinline__ unsigned long long exp_one(float l, float top, float bh, float bl, const unsigned long long* table) {
  return exp_fixed(l, l, top, bh, bl, table).x;
}
struct Exp {
  float top, bh, bl;
  const unsigned long long* table;
  __device__ __forceinline__ U2 operator()(float l0, float l1) const { return exp_fixed(l0, l1, top, bh, bl, table); }
  __device__ __forceinline__ unsigned long long operator()(float l) const { return exp_one(l, top, bh, bl, table); }
};

// (E - q A)+ with A = ah + am (to 2^-48 of itself), all in units of 2^-44, of two probabilities at once
struct Cut {
  float ah, am;
  __device__ __forceinline__ explicit Cut(double a) : ah((float)a), am((float)(a - (double)ah)) {}
  __device__ __forceinline__ U2 operator()(unsigned long long e0, unsigned long long e1, float q0, float q1) const {
    const uint64_t q = pack2(fminf(fmaxf(q0, 0.f), 1.f), fminf(fmaxf(q1, 0.f), 1.f));  // (NaN: 0)
    // q A as th + tl, then as an integer in two steps of 23 bits; E is 2^44 at most
    const uint64_t th = mul2(q, both(ah)), tl = fma2(q, both(am), fma2(q, both(ah), mul2(q, both(-ah))));
    const uint64_t m1 = fma2(th, both(0x1p-23f), both(kMagic));
    const uint64_t m2 = add2(add2(fma2(add2(m1, both(-kMagic)), both(-0x1p23f), th), tl), both(kMagic));
    const float2 t = unpack2(th), hi = unpack2(m1), lo = unpack2(m2);
    const long long y0 = (long long)e0 - ((long long)low_bits(hi.x) * (1ll << 23) + low_bits(lo.x));
    const long long y1 = (long long)e1 - ((long long)low_bits(hi.y) * (1ll << 23) + low_bits(lo.y));
    return U2{t.x < 0x1p44f && y0 > 0 ? (unsigned long long)y0 : 0ull, t.y < 0x1p44f && y1 > 0 ? (unsigned long long)y1 : 0ull};
  }
  __device__ __forceinline__ unsigned long long operator()(unsigned long long e, float q) const { return (*this)(e, e, q, q).x; }
};

// -------------------------------------------------------------------------------------------- walk
struct __align__(16) Node {
  int parent, token;   // parent -1: not a child of anything
  int first, next;     // its first child, its parent's next child; -1: none
  float u;             // its uniform
  float l, q;          // logit and draft probability of the token in the parent's row
  int fits;            // whether it is accepted as long as no sibling was rejected: a verdict
  float top, sum;      // of its own row
  int arg, pad;
};
enum { kCut, kDraw, kWhole, kEnd };

// Whether a child is accepted, u q left < y, where `left`, what there is of the parent's row, is off by `off` at most; kUnsure: that
// does not tell.
enum { kNo, kYes, kUnsure };
// What is off by where `left` comes from row_kernel's sum, relative to that.  The sum: an exponent (l - top) / T log2(e) by 5 2^-24 of
// itself (one that matters among 2^18 tokens is 18 at most: 2^-18), the exponentials by 2^-22 a dozen times (themselves and from maximum to
// maximum: 2^-18), 50 additions by 2^-24 each (2^-18); then half a dozen roundings of the test itself: less than
constexpr float kSumOff = 0x1p-15f;
template <class T>
__device__ __forceinline__ int verdict(T uq, T left, T off, T y) {
  const T border = uq * left;
  return fabs(border - y) < uq * off ? kUnsure : border < y ? kYes : kNo;
}
__device__ __forceinline__ float unit(unsigned long long y) { return (float)y * 0x1p-44f; }

struct WalkShared {
  Node* node;                          // [n_nodes], and behind them
  int* path;                           // [n_nodes]
  int* gone;                           // [n_nodes] tokens of rejected children (drafts without probabilities)
  unsigned long long part[2][kWalkCtas];  // the CTAs' sums, written by each into all
  unsigned long long bars[2];          // ... and where a set says that it is whole
  unsigned long long warp_sum[2][kWalkWarps];
  unsigned long long power[kPowers];
  float t;
  int count, abort;
  int step, at, length, n_gone, next;
};

__host__ __device__ constexpr int node_bytes(int n) { return (n * ((int)sizeof(Node) + 8) + 15) / 16 * 16; }

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cta_count() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void walk_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_cta(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
// a value into another CTA's shared memory, and its 8 bytes off what a barrier there waits for
__device__ __forceinline__ void put_async(uint32_t at, unsigned long long v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(at), "l"(v), "r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait_sums(uint32_t bar, uint32_t parity) {
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
// As op_wait: of a whole warp, given up after a time.  (The CTA then goes on with wrong sums, without further waits and without sending
// its own, so that the others give up too, and its call has an error recorded.)
__device__ __noinline__ void wait_sums(uint32_t bar, uint32_t parity, volatile int* abort, int32_t* status) {
  const uint64_t t0 = gtime();
  while (!__all_sync(0xffffffffu, try_wait_sums(bar, parity))) {
    if (__any_sync(0xffffffffu, *abort != 0)) return;
    if (__any_sync(0xffffffffu, (long long)(gtime() - t0) > kOpWaitNs)) {
      *abort = 1;
      op_error(status, MK_ERR_TIMEOUT, (int)blockIdx.x, 1, (int)parity);
      return;
    }
  }
}

__device__ __forceinline__ unsigned long long warp_total(unsigned long long v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// What every CTA of the cluster looks up for the whole walk.  (By one of them and copied to the others it took 1.2 us longer.)
// `first_cta`: the one that records what is wrong.
__device__ void gather_nodes(const VerifyParams& p, WalkShared& sh, int b, bool first_cta) {
  const mk_verify_args& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool f32 = a.logits_float != 0;
  // (loads that need nothing of one another first)
  int count = node_count(a, b);
  const Heat heat(temperature(a, b));
  const long long mine_at = (long long)b * a.n_nodes + tid;
  Node x{};
  if (tid < a.n_nodes) {
    x.parent = tid == 0 ? -1 : a.parents ? op_ld(a.parents + mine_at) : tid - 1;
    x.token = tid == 0 ? 0 : op_ld(a.tokens + mine_at);
    x.u = op_ldf(a.uniforms + mine_at);
  }
  if (count < 1 || count > a.n_nodes) {
    if (first_cta && tid == 0) op_error(a.status, MK_ERR_INVALID, b, -1, count);
    count = 0;
  } else if (!(heat.t >= 0.f)) {
    if (first_cta && tid == 0) op_error(a.status, MK_ERR_INVALID, b, -1, __float_as_int(heat.t));
    count = 0;
  }
  if (tid == 0) sh.count = count, sh.t = heat.t;
  if (tid < count) {
    const int i = tid;
    bool fine = true;
    if (!(x.u >= 0.f && x.u < 1.f)) {
      if (first_cta) op_error(a.status, MK_ERR_INVALID, b, i, __float_as_int(x.u));
      x.u = 0.f;
      fine = false;
    } else if (i > 0 && (x.parent < 0 || x.parent >= i)) {
      if (first_cta) op_error(a.status, MK_ERR_INVALID, b, i, x.parent);
      fine = false;
    } else if (x.token < 0 || x.token >= a.vocab) {
      if (first_cta) op_error(a.status, MK_ERR_INVALID, b, i, x.token);
      fine = false;
    }
    if (i > 0 && fine) {
      x.l = load_logit(logit_row(a, b, x.parent), x.token, f32);
      x.q = a.draft_probs ? fminf(fmaxf(op_ldf(a.draft_probs + b * a.draft_stride[0] + x.parent * a.draft_stride[1] + x.token), 0.f), 1.f) : 1.f;
    } else {
      x.parent = -1;
    }
    Node& to = sh.node[i];  // (top, sum and arg are another warp's)
    to.parent = x.parent, to.token = x.token, to.first = to.next = -1, to.u = x.u, to.l = x.l, to.q = x.q;
  }
  // the pieces of every row (up to 32 nodes: beside the first warp, which waits for two loads in a row above)
  const bool beside = count <= 32;
  for (int i = beside ? warp - 1 : warp; i >= 0 && i < count; i += beside ? kWalkWarps - 1 : kWalkWarps) {
    const float4* part = p.parts + ((long long)b * a.n_nodes + i) * p.pieces;
    Peak mine{-INFINITY, 0.f, 0x7fffffff};
    for (int j = lane; j < p.pieces; j += 32) {
      const uint4 u = op_ld16(part + j);
      mine.merge(__uint_as_float(u.x), __uint_as_float(u.y), (int)u.z, heat.hi);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
      mine.merge(__shfl_xor_sync(0xffffffffu, mine.top, o), __shfl_xor_sync(0xffffffffu, mine.sum, o), __shfl_xor_sync(0xffffffffu, mine.arg, o),
                 heat.hi);
    if (lane == 0) {
      sh.node[i].top = mine.top;
      sh.node[i].sum = mine.sum;
      sh.node[i].arg = mine.arg;
    }
  }
  __syncthreads();
  if (tid < count) {
    // the children in order, and the test of each against its parent's whole row
    const int up = sh.node[tid].parent;
    int first = -1, next = -1;
#pragma unroll 8
    for (int j = count - 1; j > tid; --j) {
      const int of = sh.node[j].parent;
      if (of == tid) first = j;
      if (of == up) next = j;
    }
    int fits = kNo;
    if (up >= 0) {
      const Node x = sh.node[tid], v = sh.node[up];
      const Exp ex{v.top, heat.hi, heat.lo, sh.power};
      fits = heat.t == 0.f ? (x.token == v.arg && x.u * x.q < 1.f ? kYes : kNo)  // (p is 1 at the largest)
                           : verdict(x.u * x.q, v.sum, v.sum * kSumOff, unit(ex(x.l)));
    }
    sh.node[tid].first = first;
    sh.node[tid].next = up < 0 ? -1 : next;
    sh.node[tid].fits = fits;
  }
}

// The sum, or the largest, of what the warps of all CTAs hand in, in turn `*turn`.  (Two sets in turn: a CTA may send the next pass's
// sums while another still reads this one's, but nobody is two passes ahead, since a pass needs everybody's.)
template <bool LARGEST = false>
__device__ __forceinline__ unsigned long long exchange(WalkShared& sh, unsigned long long warp_sum, uint32_t* turn, int32_t* status) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ctas = cta_count(), set = *turn & 1, bar = smem_u32(&sh.bars[set]);
  if (lane == 0) sh.warp_sum[set][warp] = warp_sum;
  __syncthreads();
  if (threadIdx.x < ctas && !*static_cast<volatile int*>(&sh.abort)) {  // (one that gave up a wait may walk on when the others have left)
    unsigned long long mine = 0;
#pragma unroll
    for (int i = 0; i < kWalkWarps; ++i) mine = LARGEST ? max(mine, sh.warp_sum[set][i]) : mine + sh.warp_sum[set][i];
    if (threadIdx.x == 0) mbar_expect_tx(bar, ctas * 8);
    put_async(map_cta(&sh.part[set][cta_rank()], threadIdx.x), mine, map_cta(&sh.bars[set], threadIdx.x));
  }
  __syncwarp();
  wait_sums(bar, *turn >> 1 & 1, &sh.abort, status);
  unsigned long long total = 0;
#pragma unroll
  for (uint32_t i = 0; i < kWalkCtas; ++i) {
    const unsigned long long v = i < ctas ? sh.part[set][i] : 0;
    total = LARGEST ? max(total, v) : total + v;
  }
  ++*turn;
  return total;
}

// One cluster per sequence.  Every CTA's first thread walks by itself, all of them from the same numbers (their own copies of the
// nodes, and sums that each has of all), so that they ask for the same passes.  The sums of a pass are sent to every CTA, whose barrier
// counts them.  (With barriers of the cluster in their
// place, and one CTA's nodes copied to the others, 8 x 9 nodes took 32.1 us, without 30.4.)
__global__ void __launch_bounds__(kWalkThreads, 1) walk_kernel(const __grid_constant__ VerifyParams p) {
  extern __shared__ __align__(128) uint8_t raw[];
  __shared__ __align__(16) WalkShared sh;
  // nodes, path, tokens gone; behind them the CTA's piece of the row's exponentials
  unsigned long long* const e = reinterpret_cast<unsigned long long*>(raw + node_bytes(p.a.n_nodes));
  const mk_verify_args& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cta_rank(), ctas = cta_count();
  const int b = (int)(blockIdx.x / ctas);
  const bool f32 = a.logits_float != 0;
  // a piece a CTA, a part of it a warp, in whole blocks
  const int blocks = (a.vocab + kBlock - 1) / kBlock, mine = (blocks + (int)ctas - 1) / (int)ctas, per = (mine + kWalkWarps - 1) / kWalkWarps;
  const int base = (int)rank * mine * kBlock;                                       // first element of the CTA
  const int first = min(warp * per, mine), n_blocks = min(per, mine - first);       // blocks of this warp
  const int from = first * kBlock + 4 * lane;                                       // first element of this lane in the piece
  for (int i = tid; i < kPowers; i += kWalkThreads) sh.power[i] = powers.v[i];
  if (tid == 0) {
    sh.node = reinterpret_cast<Node*>(raw);
    sh.path = reinterpret_cast<int*>(raw + a.n_nodes * sizeof(Node));
    sh.gone = sh.path + a.n_nodes;
    sh.abort = 0;
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&sh.bars[i]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // (all CTAs have started, their barriers are there)
  pdl_wait();
  pdl_trigger();
  gather_nodes(p, sh, b, rank == 0);
  __syncthreads();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  const int count = sh.count;
  const Heat heat(sh.t);
  Exp ex{0.f, heat.hi, heat.lo, sh.power};
  int at = 0, row_at = -1;
  uint32_t turn = 0;  // passes so far
  // of the row at `at`: A and W, and what this warp has of W
  double A = 0;
  unsigned long long W = 0, warp_sum = 0;
  bool loaded = false, stuck = false;
  // the first thread's: the child to test (-2: at a new node), the proposed tokens that are gone and what they had
  int child = -2, length = 0, n_gone = 0;
  unsigned long long gone_sum = 0;
  bool whole = true;  // no child rejected yet

  for (;;) {
    if (tid == 0) {
      int step = -1;
      while (step < 0) {
        if (count == 0) {
          step = kEnd;
          sh.next = -1;
        } else if (child == -2) {
          const Node& v = sh.node[at];
          sh.path[length++] = at;
          child = v.first;
          n_gone = 0;
          gone_sum = 0;
          whole = true;
          // (a NaN in the row is a NaN in the sum.  Nothing is known of a row without children.)
          if (child >= 0 && !(fabsf(v.top) < INFINITY && v.sum > 0.f)) {
            if (rank == 0) op_error(a.status, MK_ERR_INVALID, b, at, __float_as_int(v.top));
            step = kEnd;
            sh.next = -1;
          }
        } else if (child < 0) {
          step = kDraw;
          if (heat.t == 0.f && sh.node[at].first >= 0) {
            step = kEnd;
            sh.next = sh.node[at].arg;
          }
        } else {
          const Node& c = sh.node[child];
          const bool proposed = heat.t != 0.f && !a.draft_probs;
          int taken = whole || heat.t == 0.f ? c.fits : kUnsure;
          if (taken == kUnsure || (proposed && taken == kNo)) {
            ex.top = sh.node[at].top;
            unsigned long long y = ex(c.l);
            if (a.draft_probs) {
              if (!whole) y = Cut(A)(y, c.q);
            } else {
              for (int g = 0; g < n_gone; ++g)
                if (sh.gone[g] == c.token) y = 0;
            }
            bool more;  // whether anything but this token is left
            if (loaded && row_at == at) {
              taken = verdict((double)c.u * (double)c.q, (double)(W - gone_sum), 0.0, (double)y);
              more = W - gone_sum > y;
            } else {  // (in doubles: 8 trees of 16 nodes 23.3 us in place of 21.7)
              const float all = sh.node[at].sum, off = all * kSumOff, left = all - unit(gone_sum);
              taken = verdict(c.u * c.q, left, off, unit(y));
              more = left - unit(y) > off;
              if (proposed && taken == kNo && !more) taken = kUnsure;
            }
            if (proposed && taken == kNo && y > 0 && more) {
              gone_sum += y;
              sh.gone[n_gone++] = c.token;
            }
          }
          if (taken == kUnsure) {
            step = kWhole;
          } else if (taken == kYes) {
            at = child;
            child = -2;
          } else {
            child = c.next;
            whole = false;
            if (heat.t != 0.f && a.draft_probs) step = kCut;
          }
        }
      }
      sh.step = step;
      sh.at = at;
      sh.n_gone = n_gone;
    }
    __syncthreads();
    const int step = sh.step, gone = step == kDraw ? sh.n_gone : 0, asked = sh.at;
    __syncthreads();  // (the first thread may go on)
    if (step == kEnd) break;
    loaded = loaded && row_at == asked && gone == 0;  // (once more without the tokens that are gone)
    at = row_at = asked;
    const bool draft = a.draft_probs != nullptr;
    const float* const drow = draft ? a.draft_probs + b * a.draft_stride[0] + at * a.draft_stride[1] : nullptr;
    const bool qwide = is_wide(drow, true);
    // ------------------------------------------------------------ the row's exponentials into shared memory, and their sum
    if (!loaded) {
      const void* const row = logit_row(a, b, at);
      const bool wide = is_wide(row, f32);
      // (all copies first, each into the first half of what the lane turns it into: lanes wait for their own only, for the second
      // half of them behind the first half's exponentials.  Rolled loops: unrolled, the code of a pass that runs once is fetched for
      // longer than it runs.)
      const int half = (n_blocks + 1) / 2;
      if (wide) {
        const int size = f32 ? 16 : 8;
        for (int k = 0; k < n_blocks; ++k) {
          const int j = base + from + k * kBlock;
          const uint32_t to = smem_u32(e + from + k * kBlock);
          const void* const src = static_cast<const uint8_t*>(row) + (long long)j * (size / 4);
          if (j + 4 <= a.vocab) {
            if (f32)
              op_cp16(to, src, 16);
            else
              op_cp8(to, src);
          }
          if (k + 1 == half) asm volatile("cp.async.commit_group;" ::: "memory");
        }
      }
      if (draft && step == kCut && qwide)  // (into L2)
        for (int k = 0; k < n_blocks; ++k) {
          const int j = base + from + k * kBlock;
          if (lane % 8 == 0 && j < a.vocab) asm volatile("prefetch.global.L2 [%0];" ::"l"(drow + j) : "memory");
        }
      auto logits = [&](int k) {
        const int j = base + from + k * kBlock;
        if (!wide || j + 4 > a.vocab) return load4(row, j, a.vocab, f32, false, -INFINITY);
        const float4 v = *reinterpret_cast<const float4*>(e + from + k * kBlock);
        if (f32) return v;
        const float2 lo = bf16x2_to_f2(__float_as_uint(v.x)), hi = bf16x2_to_f2(__float_as_uint(v.y));
        return make_float4(lo.x, lo.y, hi.x, hi.y);
      };
      if (sh.node[at].first < 0) {
        // the largest logit and its index (the lowest), as one number: what is larger, and of equal ones what comes first, is larger
        float top = -INFINITY;
        int arg = 0;
        bool odd = false;
        op_cp_wait_all();
#pragma unroll 1
        for (int k = 0; k < n_blocks; ++k) {
          const float4 v = logits(k);
          const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            odd |= !(x[i] < INFINITY);
            if (x[i] > top) top = x[i], arg = base + from + k * kBlock + i;
          }
        }
        const uint32_t bits = __float_as_uint(top + 0.f);  // (one zero)
        unsigned long long key = (unsigned long long)(bits >> 31 ? ~bits : bits | 0x80000000u) << 32 | (uint32_t)~arg;
        if (odd) key = ~0ull;  // (NaN or infinite)
#pragma unroll
        for (int o = 16; o; o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
        key = exchange<true>(sh, key, &turn, a.status);
        const uint32_t high = (uint32_t)(key >> 32);
        top = key == ~0ull ? INFINITY : __uint_as_float(high >> 31 ? high & 0x7fffffffu : ~high);
        ex.top = top;
        if (!(fabsf(top) < INFINITY) || heat.t == 0.f) {
          if (tid == 0) {
            sh.next = fabsf(top) < INFINITY ? (int)~(uint32_t)key : -1;
            if (rank == 0 && sh.next < 0) op_error(a.status, MK_ERR_INVALID, b, at, __float_as_int(top));
          }
          break;
        }
      } else {
        ex.top = sh.node[at].top;
        // (the last group is open: the copies of the second half)
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      }
      unsigned long long sum = 0;
#pragma unroll 1
      for (int k = 0; k < n_blocks; ++k) {
        if (k == half) op_cp_wait_all();
        const int j = base + from + k * kBlock;
        ulonglong2* const to = reinterpret_cast<ulonglong2*>(e + from + k * kBlock);
        const float4 v = logits(k);
        const U2 lo = ex(v.x, v.y), hi = ex(v.z, v.w);
        unsigned long long y[4] = {lo.x, lo.y, hi.x, hi.y};
        for (int g = 0; g < gone; ++g) {
          const int d = sh.gone[g] - j;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (d == i) y[i] = 0;
        }
        to[0] = make_ulonglong2(y[0], y[1]);
        to[1] = make_ulonglong2(y[2], y[3]);
        sum += y[0] + y[1] + y[2] + y[3];
      }
      warp_sum = warp_total(sum);
      A = 0;
      W = exchange(sh, warp_sum, &turn, a.status);
      loaded = true;
      stuck = false;
    }
    if (step == kWhole) continue;
    if (step == kCut) {
      if (!stuck) {
        const Cut cut(A + (double)W);
        unsigned long long sum = 0;
        for (int k = 0; k < n_blocks; k += 4) {
          float4 qs[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (k + i < n_blocks) qs[i] = load4(drow, base + from + (k + i) * kBlock, a.vocab, true, qwide, 0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (k + i < n_blocks) {
              const ulonglong2* const y = reinterpret_cast<const ulonglong2*>(e + from + (k + i) * kBlock);
              const ulonglong2 lo = y[0], hi = y[1];
              const U2 c = cut(lo.x, lo.y, qs[i].x, qs[i].y), d = cut(hi.x, hi.y, qs[i].z, qs[i].w);
              sum += c.x + c.y + d.x + d.y;
            }
        }
        sum = warp_total(sum);
        const unsigned long long now = exchange(sh, sum, &turn, a.status);
        if (now) {
          A += (double)W;
          W = now;
          warp_sum = sum;
        } else {
          stuck = true;  // nothing would be left: it stays as it was
        }
      }
      continue;
    }
    // ------------------------------------------------------------ the first index whose running sum passes u times the whole
    // (u has 24 bits: u 2^64 is exact from 2^-40 on)
    if (W == 0) {  // (a wait was given up: something is left of every row)
      if (tid == 0) sh.next = -1;
      break;
    }
    const unsigned long long goal = __umul64hi((unsigned long long)((double)sh.node[0].u * 0x1p64), W);
    if (stuck) {  // (the last pass did not count)
      exchange(sh, warp_sum, &turn, a.status);
    }
    unsigned long long sum = 0;
    const uint32_t set = (turn - 1) & 1;  // the last pass's
#pragma unroll
    for (uint32_t i = 0; i < kWalkCtas; ++i) sum += i < rank ? sh.part[set][i] : 0;
#pragma unroll
    for (int i = 0; i < kWalkWarps; ++i) sum += i < warp ? sh.warp_sum[set][i] : 0;
    if (goal >= sum && goal < sum + warp_sum) {  // this warp's
      const Cut cut(A);
      bool found = false;
      for (int k0 = 0; k0 < n_blocks && !found; k0 += 4) {
        float4 qs[4];
        if (A > 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (k0 + i < n_blocks) qs[i] = load4(drow, base + from + (k0 + i) * kBlock, a.vocab, true, qwide, 0.f);
        }
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
          const int k = k0 + k4;
          if (k >= n_blocks || found) break;
          const ulonglong2* const at4 = reinterpret_cast<const ulonglong2*>(e + from + k * kBlock);
          const ulonglong2 lo = at4[0], hi = at4[1];
          unsigned long long y[4] = {lo.x, lo.y, hi.x, hi.y};
          if (A > 0) {
            const U2 c = cut(lo.x, lo.y, qs[k4].x, qs[k4].y), d = cut(hi.x, hi.y, qs[k4].z, qs[k4].w);
            y[0] = c.x, y[1] = c.y, y[2] = d.x, y[3] = d.y;
          }
          const unsigned long long own = y[0] + y[1] + y[2] + y[3];
          unsigned long long upto = own;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long z = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += z;
          }
          const unsigned past = __ballot_sync(0xffffffffu, sum + upto > goal);
          if (past) {
            found = true;
            if (lane == __ffs(past) - 1) {
              unsigned long long s = sum + upto - own;
              int i = 0;
#pragma unroll
              for (int j = 0; j < 3; ++j)
                if (i == j && s + y[j] <= goal) s += y[j], ++i;
              a.next_tokens[b] = base + from + k * kBlock + i;
            }
          } else {
            sum += __shfl_sync(0xffffffffu, upto, 31);
          }
        }
      }
    }
    if (tid == 0) sh.next = -2;  // written
    break;
  }
  if (rank == 0) {
    if (tid == 0) {
      sh.length = length;
      if (sh.next != -2) a.next_tokens[b] = sh.next;
    }
    __syncthreads();
    for (int i = tid; i < a.n_nodes; i += kWalkThreads) a.accepted[(long long)b * a.n_nodes + i] = i < sh.length ? sh.path[i] : -1;
  }
  // No CTA leaves while another may send to it: it has had all that was sent.  One that gave up waiting stays until the others leave.
  if (sh.abort) walk_sync();
}

int row_pieces(const mk_verify_args& a) { return (a.vocab + kRowThreads * kRowValues - 1) / (kRowThreads * kRowValues); }

}  // namespace

size_t verify_workspace_bytes(const mk_verify_args& a) {
  return (size_t)std::max(1, a.batch) * a.n_nodes * row_pieces(a) * sizeof(float4);
}

cudaError_t launch_verify(VerifyParams& p, cudaStream_t st) {
  p.parts = static_cast<float4*>(p.a.workspace);
  p.pieces = row_pieces(p.a);
  const dim3 grid((unsigned)p.pieces, (unsigned)p.a.n_nodes, (unsigned)p.a.batch);
  static std::atomic<unsigned long long> done{0}, done16{0};
  cudaError_t e = p.a.logits_float ? launch_early(row_kernel<true>, grid, kRowThreads, 0, st, p) : launch_early(row_kernel<false>, grid, kRowThreads, 0, st, p);
  constexpr int kSizes = 8;
  static std::atomic<int> known[kSizes][64];
  if (e == cudaSuccess) e = allow_smem(walk_kernel, kWalkSmem, done);
  if (e == cudaSuccess) e = allow_wide_clusters(walk_kernel, done16);
  // CTAs of a cluster: a walk with one pass over a row takes about 10 us and 1 more for every 12.5 blocks of a CTA's piece of it (8 x 9
  // nodes of 151936: 37.5 us in clusters of 6, 32.1 in 8, 29.3 in 10, 28.1 in 12).  Where the clusters do not fit the GPU all at
  // once (7 of 16 CTAs do, 8 of 12, 15 of 8, 23 of 6) the last ones start as the first end, which are not equally long (16 trees of
  // 32 nodes: 73.3 us in clusters of 8, 81.9 in 6)
  static const int sizes[kSizes] = {16, 12, 10, 8, 6, 4, 2, 1};
  const int blocks = (p.a.vocab + kBlock - 1) / kBlock, nodes = node_bytes(p.a.n_nodes);
  int ctas = 0;
  double least = 0;
  for (int i = 0; e == cudaSuccess && i < kSizes; ++i) {
    const int piece = (blocks + sizes[i] - 1) / sizes[i];
    if (nodes + piece * kBlock * 8 > kWalkSmem) continue;
    int fit = 0;
    e = active_clusters(walk_kernel, sizes[i], kWalkThreads, kWalkSmem, known[i], &fit);
    if (e != cudaSuccess || fit < 1) continue;
    const double cost = std::max(1.0, (double)p.a.batch / fit) * (10 + piece / 12.5);
    if (!ctas || cost < least) least = cost, ctas = sizes[i];
  }
  if (e != cudaSuccess) return e;
  if (!ctas) return cudaErrorInvalidConfiguration;
  const size_t smem = nodes + (size_t)((blocks + ctas - 1) / ctas) * kBlock * 8;
  return launch_clusters(walk_kernel, dim3((unsigned)(p.a.batch * ctas)), ctas, kWalkThreads, smem, st, p);
}

}  // namespace mk
