// Norm of every query and key head, position rotation and append to the paged cache.
//
// Per head x of hd values: x' = R(p)(g * x / sqrt(mean(x^2) + eps)); R rotates the pairs
// (i, i + hd/2) by p * theta^(-2i/hd).  A slot of hd/16 lanes holds a head: lane j the
// values 8j..8j+7 of each half (two 16-byte loads), so that a pair never leaves its
// lane and the mean is a shuffle over hd/16 lanes.  V heads are copied by the same slots.
// A token's cosines and sines are computed once, into shared memory, while its heads'
// loads are in flight.  The angle's fraction of a turn is exact in 64-bit fixed point
// (position * turns, modulo 1), so that positions of any size keep fp32 accuracy.
// Everything is fp32; each result is rounded to bf16 once.
#include "mk_ops.cuh"

namespace mk {
namespace {

constexpr int kRopeThreads = 256;

struct Head8 {  // values 8j..8j+7 of the lower and of the upper half of a head
  uint4 lo, hi;
};

__device__ __forceinline__ void widen(uint4 u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf16x2_to_f2(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint4 narrow(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// HD / 16 lanes a head; `tpb` tokens a block.
template <int HD>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p, int tpb) {
  constexpr int LPH = HD / 16;
  __shared__ float2 cs[8 * (HD / 2)];  // [token of the block][HD / 2] (cos, sin)
  const int n = p.a.n_nodes;
  const long long tokens = (long long)p.c.batch * n;
  const long long t0 = (long long)blockIdx.x * tpb;
  const int heads = p.a.n_q_heads + 2 * p.c.n_kv_heads;
  const int slots = heads * LPH;  // per token
  const uint16_t* q = static_cast<const uint16_t*>(p.a.q);
  const uint16_t* k = static_cast<const uint16_t*>(p.a.k);
  const uint16_t* v = static_cast<const uint16_t*>(p.a.v);

  // cosines and sines of the block's tokens
  for (int i = threadIdx.x; i < tpb * (HD / 2); i += kRopeThreads) {
    const long long t = t0 + i / (HD / 2);
    if (t >= tokens) break;
    const int b = (int)(t / n), node = (int)(t - (long long)b * n);
    const int pos = p.a.positions ? __ldg(p.a.positions + t) : __ldg(p.c.seq_lens + b) + node;
    const unsigned long long u = (unsigned long long)(long long)pos * p.turns[i % (HD / 2)];
    float s, c;
    sincospif((float)(int)(u >> 32) * 4.656612873077393e-10f, &s, &c);  // half turns = signed fraction * 2^-31
    cs[i] = make_float2(c, s);
  }
  __syncthreads();

  // whole groups of LPH lanes take part in the shuffles: the loop bound is rounded up to warps
  const int total = tpb * slots;
  for (int base = 0; base < total; base += kRopeThreads) {
    const int s = base + (int)threadIdx.x;
    const int tl = s / slots, r = s - tl * slots;
    const int head = r / LPH, lane = r % LPH;
    const long long t = t0 + tl;
    const int b = (int)(t / n), node = (int)(t - (long long)b * n);
    bool live = s < total && t < tokens;
    int len = 0, cnt = 0;
    if (live) {
      len = __ldg(p.c.seq_lens + b);
      cnt = p.a.counts ? __ldg(p.a.counts + b) : n;
      live = node < cnt;
    }
    const int kind = head < p.a.n_q_heads ? 0 : head < p.a.n_q_heads + p.c.n_kv_heads ? 1 : 2;
    const int hk = head - p.a.n_q_heads - (kind == 2 ? p.c.n_kv_heads : 0);
    Head8 h = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (live) {
      const uint16_t* src =
          kind == 0 ? q + b * p.a.q_stride[0] + node * p.a.q_stride[1] + head * p.a.q_stride[2]
          : kind == 1 ? k + b * p.a.k_stride[0] + node * p.a.k_stride[1] + hk * p.a.k_stride[2]
                      : v + b * p.a.v_stride[0] + node * p.a.v_stride[1] + hk * p.a.v_stride[2];
      h.lo = *reinterpret_cast<const uint4*>(src + 8 * lane);
      h.hi = *reinterpret_cast<const uint4*>(src + HD / 2 + 8 * lane);
    }
    uint16_t* dst = nullptr;
    if (live && kind == 0) {
      dst = static_cast<uint16_t*>(p.a.q_out) + b * p.a.out_stride[0] + node * p.a.out_stride[1] + head * p.a.out_stride[2];
    } else if (live) {
      const long long at = (long long)len + node;
      if (len < 0 || cnt > n || (long long)len + cnt > 16ll * p.c.max_pages) {
        op_error(p.a.status, MK_ERR_INVALID, b, node, len);
      } else {
        const int page = __ldg(p.c.page_table + (long long)b * p.c.max_pages + at / kOpPage);
        if (page < 0 || page >= p.c.n_pages)
          op_error(p.a.status, MK_ERR_BAD_PAGE, b, (int)(at / kOpPage), page);
        else
          dst = static_cast<uint16_t*>(kind == 1 ? p.c.k : p.c.v) +
                (((long long)page * p.c.n_kv_heads + hk) * kOpPage + at % kOpPage) * HD;
      }
    }
    const void* gain = kind == 0 ? p.a.q_gain : p.a.k_gain;
    float lo[8], hi[8];
    widen(h.lo, lo);
    widen(h.hi, hi);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += lo[i] * lo[i] + hi[i] * hi[i];
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (!dst) continue;
    if (kind != 2) {
      if (gain) {
        const float rs = rsqrtf(ss * (1.f / HD) + p.a.eps);
        float g[8];
        widen(__ldg(reinterpret_cast<const uint4*>(gain) + lane), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) lo[i] *= rs * g[i];
        widen(__ldg(reinterpret_cast<const uint4*>(gain) + LPH + lane), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) hi[i] *= rs * g[i];
      }
      const float2* c = cs + tl * (HD / 2) + 8 * lane;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 w = c[i];
        const float a = lo[i], d = hi[i];
        lo[i] = a * w.x - d * w.y;
        hi[i] = d * w.x + a * w.y;
      }
      h.lo = narrow(lo);
      h.hi = narrow(hi);
    }
    *reinterpret_cast<uint4*>(dst + 8 * lane) = h.lo;
    *reinterpret_cast<uint4*>(dst + HD / 2 + 8 * lane) = h.hi;
  }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t st) {
  const int hd = p.c.head_dim;
  const int slots = (p.a.n_q_heads + 2 * p.c.n_kv_heads) * (hd / 16);
  // small models: several tokens fill a block (at most 8: the shared cosines)
  int tpb = kRopeThreads / slots;
  tpb = tpb < 1 ? 1 : tpb > 8 ? 8 : tpb;
  const long long tokens = (long long)p.c.batch * p.a.n_nodes;
  const unsigned grid = (unsigned)((tokens + tpb - 1) / tpb);
  if (hd == 128)
    rope_kernel<128><<<grid, kRopeThreads, 0, st>>>(p, tpb);
  else if (hd == 64)
    rope_kernel<64><<<grid, kRopeThreads, 0, st>>>(p, tpb);
  else
    rope_kernel<32><<<grid, kRopeThreads, 0, st>>>(p, tpb);
  return cudaGetLastError();
}

}  // namespace mk
