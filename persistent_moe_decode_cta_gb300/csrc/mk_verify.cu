// Verification of drafted tokens.  A child i with token x of node v is accepted if u_i q(x) < r(x), where r = p at first and
// r <- (r - q)+ / sum (r - q)+ after a rejection; the next token is drawn from what is left where no child is accepted.
//
// Two kernels.  row_kernel reads every node's logits once, in pieces, for the largest and the sum of the exponentials: all
// that the tests of first children need beside two numbers a child.  walk_kernel has a cluster of CTAs per sequence that walks
// from the root: an accepted child costs no more than a look at shared memory; at the first rejection in a row (or at the
// last node) the cluster reads that row again, out of L2, and from then on keeps the row's exponentials in shared memory, a
// piece a CTA.  The drafting model's rows are read only where one of its tokens was rejected.
//
// Numbers.  The drawn token is where a running sum over up to 2^18 probabilities passes u times the whole: errors of fp32 would
// move borders enough to change one draw of a few hundred.  So the exponentials of the walk are 64-bit integers (2^-44 of the
// largest), exponentiated in pairs of floats, and their sums are exact: neither order nor split matters.  With R the integers
// left and W their sum, r = R / W, and a rejection leaves (R - q W)+: in terms of the row's exponentials E
// R = (E - q A)+ where A grows by W with every rejection; E is kept and A is one number.
#include "mk_ops.cuh"

namespace mk {
namespace {

constexpr int kRowThreads = 256;
constexpr int kWalkThreads = 512, kWalkWarps = kWalkThreads / 32;
constexpr int kWalkCtas = 16;              // of a cluster at most
constexpr int kFixed = 44;                 // fraction bits of an exponential
constexpr int kBlock = 128;                // elements that a warp takes at a time: four a lane

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

// log2(e) / temperature; a temperature of 0 (the largest logit alone counts) reads as 1 here
__device__ __forceinline__ double heat(const mk_verify_args& a, int b, float* t) {
  *t = a.temperature ? op_ldf(a.temperature + b) : 1.f;
  return 1.4426950408889634074 / (*t > 0.f ? (double)*t : 1.0);
}
__device__ __forceinline__ int node_count(const mk_verify_args& a, int b) { return a.counts ? op_ld(a.counts + b) : a.n_nodes; }

// -------------------------------------------------------------------------------------------- rows
// One block per piece of a row: {largest, sum of exp((l - largest) / T), index of the largest (the lowest)}.  The piece stays in
// registers between the two.  HBM bounds it.
template <int ITER>
__global__ void __launch_bounds__(kRowThreads) row_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ float s_max[kRowThreads / 32];
  __shared__ float s_sum[kRowThreads / 32];
  __shared__ int s_arg[kRowThreads / 32];
  const int piece = blockIdx.x, node = blockIdx.y, b = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  if (node >= node_count(p.a, b)) return;
  const bool f32 = p.a.logits_float != 0;
  const void* row = logit_row(p.a, b, node);
  const bool wide = is_wide(row, f32);
  float t;
  const float beta = (float)fmin(heat(p.a, b, &t), 1e30);
  const int base = piece * (kRowThreads * 4 * ITER) + 4 * threadIdx.x;
  float4 v[ITER];
#pragma unroll
  for (int i = 0; i < ITER; ++i) v[i] = load4(row, base + i * kRowThreads * 4, p.a.vocab, f32, wide, -INFINITY);
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < ITER; ++i) top = fmaxf(fmaxf(fmaxf(top, v[i].x), fmaxf(v[i].y, v[i].z)), v[i].w);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) s_max[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRowThreads / 32; ++i) top = fmaxf(top, s_max[i]);
  const float from = top == -INFINITY ? 0.f : top;  // (a piece of nothing: sums of zeros)
  float sum = 0.f;
  int arg = 0x7fffffff;
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const float x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sum += ex2((x[j] - from) * beta);
      if (x[j] == top) arg = min(arg, base + i * kRowThreads * 4 + j);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    arg = min(arg, __shfl_xor_sync(0xffffffffu, arg, o));
  }
  if (lane == 0) s_sum[warp] = sum, s_arg[warp] = arg;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kRowThreads / 32; ++i) sum += s_sum[i], arg = min(arg, s_arg[i]);
    p.parts[((long long)b * p.a.n_nodes + node) * p.pieces + piece] = make_float4(top, sum, __int_as_float(arg), 0.f);
  }
}

// ------------------------------------------------------------------------------------- exponentials
// 2^(i/256), i = -128 .. 128, in units of 2^-52 and as a sum of two floats (exp2 of a double is good to 2^-52)
constexpr int kTable = 257;
struct __align__(16) Power {
  unsigned long long fix;
  float hi, lo;
};

struct Exp {
  float top;        // the row's largest logit
  float bh, bl;     // log2(e) / T as a sum of two floats
  const Power* table;
  // exp((l - top) / T) in units of 2^-44, for finite l <= top, to 2^-41 of itself; 0 for anything else.
  __device__ __forceinline__ unsigned long long operator()(float l) const {
    // l - top as dh + dl, exactly; times log2(e) / T as ph + pl
    const float dh = l - top, z = dh - l, dl = (l - (dh - z)) - (top + z);
    // (every product that is used twice is rounded once: __fmul_rn is not fused into what follows)
    const float ph = __fmul_rn(dh, bh);
    if (!(ph >= -50.f)) return 0;
    const float pl = fmaf(dh, bh, -ph) + fmaf(dh, bl, dl * bh);
    // ph = n + i / 256 + r, exactly
    const float n = rintf(ph), f = ph - n, i = rintf(f * 256.f), r = fmaf(i, -1.f / 256.f, f);
    // y = (r + pl) ln 2 as yh + yl, |y| < 2^-9; exp(y) - 1 = y + y^2 (1/2 + y/6 + y^2/24)
    constexpr float kLn2h = 0.693147182464599609375f, kLn2l = -1.904654299957767e-9f;
    const float yh = __fmul_rn(r, kLn2h), yl = fmaf(r, kLn2h, -yh) + fmaf(r, kLn2l, pl * kLn2h);
    const float s = fmaf(yh * yh, fmaf(yh, fmaf(yh, 1.f / 24.f, 1.f / 6.f), 0.5f), fmaf(yh, yl, yl));
    const float eh = yh + s, el = s - (eh - yh);
    // times the table's entry T = th + tl: w = T (exp(y) - 1) as wh + wl, then as an integer of 2^-52 in two steps of 22 bits
    const Power t = table[128 + (int)i];
    const float wh = __fmul_rn(t.hi, eh), wl = fmaf(t.hi, eh, -wh) + fmaf(t.hi, el, t.lo * eh);
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer and leaves it in the low bits
    const float m1 = fmaf(wh, 0x1p30f, kMagic), rest = fmaf(m1 - kMagic, -0x1p-30f, wh) + wl;
    const float m2 = fmaf(rest, 0x1p52f, kMagic);
    const int hi = __float_as_int(m1) - __float_as_int(kMagic), lo = __float_as_int(m2) - __float_as_int(kMagic);
    const unsigned long long v = t.fix + (unsigned long long)(((long long)hi << 22) + lo);
    const int shift = 52 - kFixed - (int)n;  // 8 .. 58
    return (v + (1ull << (shift - 1))) >> shift;
  }
};

// (E - q A)+ with A = ah + am (to 2^-48 of itself), all in units of 2^-44
struct Cut {
  float ah, am;
  __device__ __forceinline__ explicit Cut(unsigned long long a) {
    ah = __ull2float_rn(a);
    am = (float)(long long)(a - __float2ull_rn(ah));
  }
  __device__ __forceinline__ unsigned long long operator()(unsigned long long e, float q) const {
    q = fminf(fmaxf(q, 0.f), 1.f);  // (NaN: 0)
    const float th = __fmul_rn(q, ah);
    if (!(th < 0x1p46f)) return 0;  // E is 2^44 at most
    const float tl = fmaf(q, ah, -th) + q * am;
    const long long left = (long long)e - (__float2ll_rn(th) + __float2ll_rn(tl));
    return left > 0 ? (unsigned long long)left : 0ull;
  }
};

// -------------------------------------------------------------------------------------------- walk
struct Node {
  int parent, token;   // parent -1: not a child of anything
  float u;             // its uniform
  float l, q;          // logit and draft probability of the token in the parent's row
  float top, sum;      // of its own row
  int arg;
};
struct Part {
  unsigned long long sum;
  unsigned long long bad;
};
enum { kLoad = 1, kCut = 2, kDraw = 3, kEnd = 4 };

struct WalkShared {
  Node node[kOpMaxAccept];
  int path[kOpMaxAccept];
  int gone[kOpMaxAccept];              // tokens of rejected children (drafts without probabilities)
  Part part[2][kWalkCtas];             // the CTAs' sums, written by each into all
  unsigned long long warp_sum[kWalkWarps];
  Power table[kTable];
  unsigned long long a, w;             // A and W of the row
  float t;
  int count, at, length, n_gone, step, next, stuck, loaded, parity;
};

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
__device__ __forceinline__ void put64(uint32_t at, unsigned long long v) {
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}
__device__ __forceinline__ uint4 get128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ unsigned long long warp_total(unsigned long long v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// What the first CTA of the cluster looks up for the whole walk.
__device__ void gather_nodes(const VerifyParams& p, WalkShared& sh, int b) {
  const mk_verify_args& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool f32 = a.logits_float != 0;
  int count = node_count(a, b);
  float t;
  const float beta = (float)fmin(heat(a, b, &t), 1e30);
  if (count < 1 || count > a.n_nodes) {
    if (tid == 0) op_error(a.status, MK_ERR_INVALID, b, -1, count);
    count = 0;
  } else if (!(t >= 0.f)) {
    if (tid == 0) op_error(a.status, MK_ERR_INVALID, b, -1, __float_as_int(t));
    count = 0;
  }
  if (tid == 0) sh.count = count, sh.t = t;
  for (int i = tid; i < count; i += kWalkThreads) {
    const long long at = (long long)b * a.n_nodes + i;
    Node x{};
    x.parent = i == 0 ? -1 : a.parents ? op_ld(a.parents + at) : i - 1;
    x.u = op_ldf(a.uniforms + at);
    bool fine = true;
    if (!(x.u >= 0.f && x.u < 1.f)) {
      op_error(a.status, MK_ERR_INVALID, b, i, __float_as_int(x.u));
      x.u = 0.f;
      fine = false;
    }
    if (i > 0) {
      x.token = op_ld(a.tokens + at);
      if (x.parent < 0 || x.parent >= i) {
        op_error(a.status, MK_ERR_INVALID, b, i, x.parent);
        fine = false;
      } else if (x.token < 0 || x.token >= a.vocab) {
        op_error(a.status, MK_ERR_INVALID, b, i, x.token);
        fine = false;
      }
      if (fine) {
        x.l = load_logit(logit_row(a, b, x.parent), x.token, f32);
        x.q = a.draft_probs ? fminf(fmaxf(op_ldf(a.draft_probs + b * a.draft_stride[0] + x.parent * a.draft_stride[1] + x.token), 0.f), 1.f) : 1.f;
      } else {
        x.parent = -1;
      }
    }
    sh.node[i] = x;
  }
  __syncthreads();
  // the pieces of every row
  for (int i = warp; i < count; i += kWalkWarps) {
    const float4* part = p.parts + ((long long)b * a.n_nodes + i) * p.pieces;
    float top = -INFINITY, sum = 0.f;
    int arg = 0x7fffffff;
    for (int j = lane; j < p.pieces; j += 32) {
      const uint4 u = op_ld16(part + j);
      const float m = __uint_as_float(u.x), s = __uint_as_float(u.y);
      if (m > top) {
        sum *= ex2((top - m) * beta);
        top = m;
        arg = (int)u.z;
      }
      sum += m == -INFINITY ? s : s * ex2((m - top) * beta);
    }
    float all = top;
#pragma unroll
    for (int o = 16; o; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
    if (top != all) {
      sum = top == -INFINITY ? sum : sum * ex2((top - all) * beta);
      arg = 0x7fffffff;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      arg = min(arg, __shfl_xor_sync(0xffffffffu, arg, o));
    }
    if (lane == 0) {
      sh.node[i].top = all;
      sh.node[i].sum = sum;
      sh.node[i].arg = arg;
    }
  }
}

// The CTAs' sums of a pass, in all of them; their total.  (Two sets in turn: a CTA may write the next pass's sums while another
// still reads this one's, but no CTA is two barriers ahead.)
__device__ __forceinline__ unsigned long long exchange(WalkShared& sh, unsigned long long warp_sum, bool bad, int* parity, bool* any) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ctas = cta_count(), rank = cta_rank();
  if (lane == 0) sh.warp_sum[warp] = warp_sum;
  bad = __syncthreads_or(bad);
  if (threadIdx.x < ctas) {
    unsigned long long mine = 0;
    for (int i = 0; i < kWalkWarps; ++i) mine += sh.warp_sum[i];
    const uint32_t to = map_cta(&sh.part[*parity][rank], threadIdx.x);
    put64(to, mine);
    put64(to + 8, bad);
  }
  walk_sync();
  unsigned long long total = 0, flags = 0;
  for (uint32_t i = 0; i < ctas; ++i) total += sh.part[*parity][i].sum, flags |= sh.part[*parity][i].bad;
  *any = flags != 0;
  *parity ^= 1;
  return total;
}

// One cluster per sequence.  Every CTA takes the same decisions from the same numbers (the first CTA's copy of the nodes, and sums
// that each has of all), so that all of them pass the same barriers.
__global__ void __launch_bounds__(kWalkThreads, 1) walk_kernel(const __grid_constant__ VerifyParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ __align__(16) WalkShared sh;
  unsigned long long* const e = reinterpret_cast<unsigned long long*>(raw);  // the CTA's piece of the row's exponentials
  const mk_verify_args& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cta_rank(), ctas = cta_count();
  const int b = (int)(blockIdx.x / ctas);
  const bool f32 = a.logits_float != 0;
  // a piece a CTA, a part of it a warp, in whole blocks
  const int blocks = (a.vocab + kBlock - 1) / kBlock, mine = (blocks + (int)ctas - 1) / (int)ctas, per = (mine + kWalkWarps - 1) / kWalkWarps;
  const int base = (int)rank * mine * kBlock;                                  // first element of the CTA
  const int first = min(warp * per, mine), last = min(first + per, mine);      // blocks of this warp
  for (int i = tid; i < kTable; i += kWalkThreads) {
    const double y = exp2((i - 128) / 256.0);
    sh.table[i] = Power{(unsigned long long)__double2ll_rn(y * 0x1p52), (float)y, (float)(y - (double)(float)y)};
  }
  pdl_wait();
  pdl_trigger();
  if (rank == 0) gather_nodes(p, sh, b);
  walk_sync();
  if (rank != 0) {
    if (tid == 0) {
      const uint32_t from = map_cta(&sh.t, 0);
      uint32_t x, y;
      asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(x) : "r"(from) : "memory");
      asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(y) : "r"(from + 4) : "memory");
      sh.t = __uint_as_float(x);
      sh.count = (int)y;
    }
    __syncthreads();
    for (int i = tid; i < 2 * sh.count; i += kWalkThreads)
      *(reinterpret_cast<uint4*>(sh.node) + i) = get128(map_cta(reinterpret_cast<const uint4*>(sh.node) + i, 0));
  }
  __syncthreads();
  const int count = sh.count;
  const float t = sh.t;
  const double beta = 1.4426950408889634074 / (t > 0.f ? (double)t : 1.0);
  Exp ex;
  ex.bh = (float)fmin(beta, 1e30);
  ex.bl = beta < 1e30 ? (float)(beta - (double)ex.bh) : 0.f;
  ex.table = sh.table;
  int parity = 0, at = 0, length = 0, next = -1;
  bool bad = count == 0;

  while (!bad) {
    const Node here = sh.node[at];
    if (tid == 0) sh.path[length] = at;
    ++length;
    bad = !(fabsf(here.top) < INFINITY && here.sum > 0.f);  // (a NaN in the row is a NaN in the sum)
    if (bad) {
      if (rank == 0 && tid == 0) op_error(a.status, MK_ERR_INVALID, b, at, __float_as_int(here.top));
      break;
    }
    const void* const row = logit_row(a, b, at);
    const float* const draft = a.draft_probs ? a.draft_probs + b * a.draft_stride[0] + at * a.draft_stride[1] : nullptr;
    const bool wide = is_wide(row, f32), qwide = is_wide(draft, true);
    ex.top = here.top;
    int n_gone = 0, taken = -1;
    bool loaded = false, stuck = false;
    unsigned long long A = 0, W = 0;                       // of the row once it is loaded
    double left = (double)here.sum * 0x1p44;               // ... and before that, without the tokens that are gone

    // the row's exponentials into shared memory, and their sum
    auto load = [&]() {
      unsigned long long sum = 0;
      for (int k = first; k < last; ++k) {
        const int j = base + k * kBlock + 4 * lane;
        const float4 v = load4(row, j, a.vocab, f32, wide, -INFINITY);
        unsigned long long y[4] = {ex(v.x), ex(v.y), ex(v.z), ex(v.w)};
        for (int g = 0; g < n_gone; ++g) {
          const int d = sh.gone[g] - j;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (d == i) y[i] = 0;
        }
        ulonglong2* const to = reinterpret_cast<ulonglong2*>(e + k * kBlock + 4 * lane);
        to[0] = make_ulonglong2(y[0], y[1]);
        to[1] = make_ulonglong2(y[2], y[3]);
        sum += y[0] + y[1] + y[2] + y[3];
      }
      bool any;
      W = exchange(sh, warp_total(sum), false, &parity, &any);
      loaded = true;
    };

    for (int i = at + 1; i < count && taken < 0; ++i) {
      const Node c = sh.node[i];
      if (c.parent != at) continue;
      if (t == 0.f) {  // p is 1 at the largest: a draft of anything else is rejected, and changes nothing
        if (c.token == here.arg && (double)c.u * c.q < 1.0) taken = i;
        continue;
      }
      unsigned long long y = ex(c.l);
      if (draft) {
        if (A) y = Cut(A)(y, c.q);
      } else {
        for (int g = 0; g < n_gone; ++g)
          if (sh.gone[g] == c.token) y = 0;
      }
      const double whole = loaded ? (double)W : left;
      if ((double)c.u * (double)c.q * whole < (double)y) {
        taken = i;
      } else if (draft) {
        if (!loaded) load();
        if (!stuck) {
          const Cut cut(A + W);
          unsigned long long sum = 0;
          for (int k = first; k < last; ++k) {
            const int j = k * kBlock + 4 * lane;
            const float4 q = load4(draft, base + j, a.vocab, true, qwide, 0.f);
            const ulonglong2 lo = *reinterpret_cast<const ulonglong2*>(e + j), hi = *reinterpret_cast<const ulonglong2*>(e + j + 2);
            sum += cut(lo.x, q.x) + cut(lo.y, q.y) + cut(hi.x, q.z) + cut(hi.y, q.w);
          }
          const unsigned long long before = sh.warp_sum[warp];
          sum = warp_total(sum);
          bool any;
          const unsigned long long now = exchange(sh, sum, false, &parity, &any);
          if (now) {
            A += W;
            W = now;
          } else {  // nothing is left: it stays as it was
            stuck = true;
            __syncthreads();
            if (lane == 0) sh.warp_sum[warp] = before;
          }
        }
      } else if (left > (double)y) {
        left -= (double)y;
        __syncthreads();
        if (tid == 0) sh.gone[n_gone] = c.token;
        ++n_gone;
        __syncthreads();
      }
    }
    if (taken >= 0) {
      at = taken;
      continue;
    }
    // the next token: the first index whose running sum passes u times the whole
    if (t == 0.f) {
      next = here.arg;
      break;
    }
    if (!loaded) load();
    __syncthreads();
    bad = W == 0;
    if (bad) break;
    // (u has 24 bits: u 2^64 is exact from 2^-40 on)
    const unsigned long long goal = __umul64hi((unsigned long long)((double)sh.node[0].u * 0x1p64), W);
    // whose piece it lies in: the parts of the last pass that counted
    unsigned long long sum = 0;
    const Cut cut(A);
    // sums of the CTAs before this one, from their warps' sums
    if (tid == 0) {
      unsigned long long own = 0;
      for (int i = 0; i < kWalkWarps; ++i) own += sh.warp_sum[i];
      for (uint32_t i = 0; i < ctas; ++i) put64(map_cta(&sh.part[parity][rank], i), own);
    }
    walk_sync();
    for (uint32_t i = 0; i < rank; ++i) sum += sh.part[parity][i].sum;
    for (int i = 0; i < warp; ++i) sum += sh.warp_sum[i];
    const unsigned long long end = sum + sh.warp_sum[warp];
    if (goal >= sum && goal < end) {  // this warp's
      for (int k = first; k < last; ++k) {
        const int j = k * kBlock + 4 * lane;
        unsigned long long y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = e[j + i];
        if (A) {
          const float4 q = load4(draft, base + j, a.vocab, true, qwide, 0.f);
          y[0] = cut(y[0], q.x), y[1] = cut(y[1], q.y), y[2] = cut(y[2], q.z), y[3] = cut(y[3], q.w);
        }
        const unsigned long long own = y[0] + y[1] + y[2] + y[3];
        unsigned long long upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long z = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += z;
        }
        const unsigned found = __ballot_sync(0xffffffffu, sum + upto > goal);
        if (found) {
          if (lane == __ffs(found) - 1) {
            unsigned long long s = sum + upto - own;
            int i = 0;
            while (i < 3 && s + y[i] <= goal) s += y[i++];
            a.next_tokens[b] = base + j + i;
          }
          break;
        }
        sum += __shfl_sync(0xffffffffu, upto, 31);
      }
    }
    next = -2;  // written
    break;
  }
  __syncthreads();
  if (rank == 0) {
    for (int i = tid; i < a.n_nodes; i += kWalkThreads) a.accepted[(long long)b * a.n_nodes + i] = i < length ? sh.path[i] : -1;
    if (tid == 0 && next != -2) a.next_tokens[b] = next;
  }
  walk_sync();  // no CTA leaves while another may write to it or read its nodes
}

// Pieces of a row: 2048 to 8192 elements, the more the fewer rows there are
int row_iter(const mk_verify_args& a) {
  const long long rows = (long long)a.batch * a.n_nodes;
  for (int iter = 8; iter > 2; iter /= 2)
    if (rows * ((a.vocab + kRowThreads * 4 * iter - 1) / (kRowThreads * 4 * iter)) >= 600) return iter;
  return 2;
}
int row_pieces(const mk_verify_args& a) {
  const int piece = kRowThreads * 4 * row_iter(a);
  return (a.vocab + piece - 1) / piece;
}

}  // namespace

size_t verify_workspace_bytes(const mk_verify_args& a) {
  return (size_t)std::max(1, a.batch) * a.n_nodes * row_pieces(a) * sizeof(float4);
}

cudaError_t launch_verify(VerifyParams& p, cudaStream_t st) {
  p.parts = static_cast<float4*>(p.a.workspace);
  p.pieces = row_pieces(p.a);
  const dim3 grid((unsigned)p.pieces, (unsigned)p.a.n_nodes, (unsigned)p.a.batch);
  const int iter = row_iter(p.a);
  cudaError_t e = iter == 8   ? launch_early(row_kernel<8>, grid, kRowThreads, 0, st, p)
                  : iter == 4 ? launch_early(row_kernel<4>, grid, kRowThreads, 0, st, p)
                              : launch_early(row_kernel<2>, grid, kRowThreads, 0, st, p);
  if (e != cudaSuccess) return e;
  // a piece of the exponentials has to fit shared memory
  const int ctas = p.a.vocab <= 8 * kBlock * 180 ? 8 : kWalkCtas;
  const int blocks = (p.a.vocab + kBlock - 1) / kBlock, mine = (blocks + ctas - 1) / ctas;
  const size_t smem = (size_t)mine * kBlock * 8;
  static std::atomic<unsigned long long> done{0};
  e = allow_smem(walk_kernel, 180 * kBlock * 8, done);
  if (e != cudaSuccess) return e;
  if (ctas > 8) {
    e = cudaFuncSetAttribute(walk_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  return launch_clusters(walk_kernel, dim3((unsigned)(p.a.batch * ctas)), ctas, kWalkThreads, smem, st, p);
}

}  // namespace mk
