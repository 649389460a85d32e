// Norm of every query and key head, position rotation and append to the paged cache.
//
// Per head x of hd values: x' = R(p)(g * x / sqrt(mean(x^2) + eps)); R rotates the pairs
// (i, i + hd/2) by p * theta^(-2i/hd).  A slot of hd/16 lanes holds a head: lane j the
// values 8j..8j+7 of each half (two 16-byte loads), so that a pair never leaves its
// lane and the mean is a shuffle over hd/16 lanes.  V heads are copied by the same slots.
// A token's cosines and sines are computed once, into shared memory, while the loads of the block's
// first heads are in flight.  The angle's fraction of a turn is exact in 64-bit fixed point
// (position * turns, modulo 1), so that positions of any size keep fp32 accuracy.
// Everything is fp32; each result is rounded to bf16 once.  The bytes bound it, and with few tokens
// the launch (128 tokens of 40 heads of 128: 2.8 us on the GPU).
#include "mk_ops.cuh"

#include <algorithm>

namespace mk {
namespace {

constexpr int kRopeMaxThreads = 512;
constexpr int kRopeMost = 12;            // tokens behind one another in a block, at most (8002 tokens 31.0 us; 6: 31.4, 24: 33.6)
constexpr int kRopeSmem = 16 * 1024;     // ... and of their angles

struct Head8 {  // values 8j..8j+7 of the lower and of the upper half of a head
  uint4 lo, hi;
};

// four pairs of floats
__device__ __forceinline__ void widen(uint4 u, uint64_t (&x)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf16x2_to_f2(w[i]);
    x[i] = pack2(f.x, f.y);
  }
}
__device__ __forceinline__ uint32_t narrow2(uint64_t x) {
  const float2 f = unpack2(x);
  return pack_bf16(f.x, f.y);
}
__device__ __forceinline__ uint4 narrow(const uint64_t (&x)[4]) {
  return make_uint4(narrow2(x[0]), narrow2(x[1]), narrow2(x[2]), narrow2(x[3]));
}

// HD / 16 lanes a head, `slots` lanes of a token's heads in this block (blockIdx.y: which),
// `side` tokens side by side and P behind one another.  Every thread copies its own 32 bytes of the next
// AHEAD tokens to shared memory, so that loads are in flight without registers and without a barrier.
template <int HD, int AHEAD>
__global__ void __launch_bounds__(kRopeMaxThreads, 2) rope_kernel(const __grid_constant__ RopeParams p, int slots, int side, int P) {
  constexpr int LPH = HD / 16;
  // per token of the block, piece i of four angles and lane: cosines and sines of angles 8 lane + 2 i and
  // 2 i + 1, so that the lanes of a head read side by side; behind them the tokens under way
  extern __shared__ float4 cs[];
  uint4* const mine_s = reinterpret_cast<uint4*>(cs + side * P * (HD / 4)) + threadIdx.x;
  const int n = p.a.n_nodes;
  const int tokens = p.c.batch * n;  // (below 2^31: checked by the host)
  const int t0 = (int)blockIdx.x * side * P;
  const int tl = (int)threadIdx.x / slots, r = (int)threadIdx.x - tl * slots + (int)blockIdx.y * slots;
  const int head = r / LPH, lane = r % LPH;
  const int hq = p.a.n_q_heads, hkv = p.c.n_kv_heads;
  const bool mine = tl < side && head < hq + 2 * hkv;
  const int kind = head < hq ? 0 : head < hq + hkv ? 1 : 2;
  const int hk = kind == 0 ? head : head - hq - (kind == 2 ? hkv : 0);
  auto stride = [&](int i) -> long long { return kind == 0 ? p.a.q_stride[i] : kind == 1 ? p.a.k_stride[i] : p.a.v_stride[i]; };
  const uint16_t* src = static_cast<const uint16_t*>(kind == 0 ? p.a.q : kind == 1 ? p.a.k : p.a.v) + hk * stride(2) + 8 * lane;
  const long long s0 = stride(0), s1 = stride(1);

  pdl_wait();
  pdl_trigger();
  struct At {
    int b, node;
  };
  // the token `side` further on (n may be smaller than that)
  auto step = [&](At& x) {
    for (x.node += side; x.node >= n; x.node -= n) ++x.b;
  };
  At get, put;
  get.b = (t0 + tl) / n;
  get.node = t0 + tl - get.b * n;
  put = get;
  auto fetch = [&](int k) {
    if (mine && k < P && t0 + k * side + tl < tokens) {
      const uint16_t* x = src + get.b * s0 + get.node * s1;
      const uint32_t at = smem_u32(mine_s + 2 * (k % AHEAD) * (int)blockDim.x);
      op_cp16(at, x, 16);
      op_cp16(at + 16 * blockDim.x, x + HD / 2, 16);
    }
    op_cp_commit();
    step(get);
  };
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) fetch(k);
  uint4 gl = make_uint4(0, 0, 0, 0), gh = gl;
  const void* gain = kind == 0 ? p.a.q_gain : p.a.k_gain;
  const bool norm = kind != 2 && gain != nullptr;
  if (norm) {
    gl = op_ld16(static_cast<const uint4*>(gain) + lane);
    gh = op_ld16(static_cast<const uint4*>(gain) + LPH + lane);
  }

  for (int i = threadIdx.x; i < side * P * (HD / 2); i += (int)blockDim.x) {
    const int t = t0 + i / (HD / 2);
    if (t >= tokens) break;
    const int pos = p.a.positions ? op_ld(p.a.positions + t) : op_ld(p.c.seq_lens + t / n) + t % n;
    const unsigned long long u = (unsigned long long)(long long)pos * p.turns[i % (HD / 2)];
    float s, c;
    sincospif((float)(int)(u >> 32) * 4.656612873077393e-10f, &s, &c);  // half turns = signed fraction * 2^-31
    const int f = i % (HD / 2);
    float2* out = reinterpret_cast<float2*>(cs + (i / (HD / 2)) * (HD / 4) + (f / 2 % 4) * LPH + f / 8);  // (cos, cos), (sin, sin)
    reinterpret_cast<float*>(out)[f % 2] = c;
    reinterpret_cast<float*>(out)[2 + f % 2] = s;
  }
  __syncthreads();

#pragma unroll 1
  for (int k = 0; k < P && t0 + k * side < tokens; ++k, step(put)) {
    const int b = put.b, node = put.node;
    uint16_t* dst = nullptr;
    const bool live = mine && t0 + k * side + tl < tokens;
    const int cnt = live ? p.a.counts ? op_ld(p.a.counts + b) : n : 0;
    if (live && node < cnt) {
      if (kind == 0) {
        dst = static_cast<uint16_t*>(p.a.q_out) + b * p.a.out_stride[0] + node * p.a.out_stride[1] + hk * p.a.out_stride[2] + 8 * lane;
      } else {
        const int len = op_ld(p.c.seq_lens + b);
        const long long at = (long long)len + node;
        if (len < 0 || cnt > n || (long long)len + cnt > 16ll * p.c.max_pages) {
          op_error(p.a.status, MK_ERR_INVALID, b, node, len);
        } else {
          const int page = op_ld(p.c.page_table + (long long)b * p.c.max_pages + at / kOpPage);
          if (page < 0 || page >= p.c.n_pages)
            op_error(p.a.status, MK_ERR_BAD_PAGE, b, (int)(at / kOpPage), page);
          else
            dst = static_cast<uint16_t*>(kind == 1 ? p.c.k : p.c.v) +
                  (((long long)page * hkv + hk) * kOpPage + at % kOpPage) * HD + 8 * lane;
        }
      }
    }
    op_cp_wait<AHEAD - 1>();
    const uint4* from = mine_s + 2 * (k % AHEAD) * (int)blockDim.x;
    Head8 h = {from[0], from[blockDim.x]};
    uint64_t lo[4], hi[4];
    widen(h.lo, lo);
    widen(h.hi, hi);
    uint64_t sq = mul2(lo[0], lo[0]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i) sq = fma2(lo[i], lo[i], sq);
      sq = fma2(hi[i], hi[i], sq);
    }
    const float2 sum = unpack2(sq);
    float ss = sum.x + sum.y;
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (AHEAD > 1) fetch(k + AHEAD);  // (into the place that has just been read)
    if (!dst) continue;
    if (kind != 2) {
      if (norm) {
        const float rs = rsqrtf(ss * (1.f / HD) + p.a.eps);
        const uint64_t r2 = pack2(rs, rs);
        uint64_t g[4];
        widen(gl, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) lo[i] = mul2(lo[i], mul2(r2, g[i]));
        widen(gh, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) hi[i] = mul2(hi[i], mul2(r2, g[i]));
      }
      const float4* c = cs + (k * side + tl) * (HD / 4) + lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 w = c[i * LPH];
        const uint64_t co = pack2(w.x, w.y), si = pack2(w.z, w.w), ms = pack2(-w.z, -w.w);
        const uint64_t a = lo[i], d = hi[i];
        lo[i] = fma2(a, co, mul2(d, ms));
        hi[i] = fma2(d, co, mul2(a, si));
      }
      h.lo = narrow(lo);
      h.hi = narrow(hi);
    }
    *reinterpret_cast<uint4*>(dst) = h.lo;
    *reinterpret_cast<uint4*>(dst + HD / 2) = h.hi;
  }
}

template <int HD>
cudaError_t launch_hd(const RopeParams& p, int sms, cudaStream_t st) {
  const int all = (p.a.n_q_heads + 2 * p.c.n_kv_heads) * (HD / 16);
  const int ny = (all + kRopeMaxThreads - 1) / kRopeMaxThreads;
  // lanes of a token in one block: whole heads
  const int slots = ((all + ny - 1) / ny + HD / 16 - 1) / (HD / 16) * (HD / 16);
  const int side = slots < 256 ? 256 / slots : 1;  // small models: several tokens fill a block
  const int threads = (slots * side + 31) / 32 * 32;
  const long long tokens = (long long)p.c.batch * p.a.n_nodes;
  // Tokens behind one another: as few as fill the SMs (1024 threads each) in whole rounds of blocks
  // (8002 tokens of 32 + 2 * 4 heads of 128, 164 MB: two rounds of 9 tokens 30.8 us, 5.3 TB/s; one of 18 34.6;
  // 16 tokens, 1.1 rounds, 43.2; two tokens a block in registers, without the copies ahead, 35.7)
  const long long round = (long long)sms * (2 * kRopeMaxThreads / threads) * side;
  const int most = (int)std::min<long long>(kRopeMost, kRopeSmem / (side * HD * 4));
  const long long rounds = (tokens * ny + round * most - 1) / (round * most);
  const int P = (int)((tokens * ny + round * rounds - 1) / (round * rounds)), per = side * P;
  const dim3 grid((unsigned)((tokens + per - 1) / per), (unsigned)ny);
  const size_t smem = (size_t)per * (HD / 4) * sizeof(float4) + (size_t)(P > 1 ? 2 : 1) * 2 * threads * sizeof(uint4);
  return launch_early(P > 1 ? rope_kernel<HD, 2> : rope_kernel<HD, 1>, grid, threads, smem, st, p, slots, side, P);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int sms, cudaStream_t st) {
  if (p.c.head_dim == 128) return launch_hd<128>(p, sms, st);
  if (p.c.head_dim == 64) return launch_hd<64>(p, sms, st);
  return launch_hd<32>(p, sms, st);
}

}  // namespace mk
