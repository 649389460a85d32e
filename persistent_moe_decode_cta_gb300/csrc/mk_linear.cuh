// The epilogue of the products in mk_linear: bias, activation, residual and the store.
#pragma once

#include "mk_ops.cuh"

namespace mk {

// act(y).  The tanh form is y / (1 + exp(-2 z)), the erf form y/2 erfc(-y / sqrt 2): both keep their relative precision where
// 1 + tanh or 1 + erf would cancel.  Far below zero the exponential overflows and the quotient is zero.
//
// For float32 results, with CUDA's functions:
template <int ACT>
__device__ __forceinline__ float act_exact(float y) {
  if (ACT == MK_ACT_RELU) return y < 0.f ? 0.f : y;  // (NaN stays)
  if (ACT == MK_ACT_GELU) return 0.5f * y * erfcf(-0.70710678118654752f * y);
  const float z = ACT == MK_ACT_SILU ? y : 1.5957691216057308f * fmaf(0.044715f * y * y, y, y);
  return y / (1.f + expf(-z));
}

// For bf16 results, which hide the 2^-18 of approximate exponentials and reciprocals, of two values at once.  One value at a time
// with __expf and __fdividef, whose guards for results below the normal range cost more than the rest, the epilogue of 224 x 256
// results took 8500 cycles in place of 6400.
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint64_t splat2(float v) { return pack2(v, v); }
__device__ __forceinline__ uint64_t ex2_2(uint64_t v) {
  const float2 f = unpack2(v);
  return pack2(ex2(f.x), ex2(f.y));
}
__device__ __forceinline__ uint64_t rcp2(uint64_t v) {
  const float2 f = unpack2(v);
  return pack2(rcp(f.x), rcp(f.y));
}
template <int ACT>
__device__ __forceinline__ void act_pair(float& y0, float& y1) {
  constexpr double kLog2e = 1.4426950408889634, kTanh = -1.5957691216057308 * kLog2e;
  const uint64_t y = pack2(y0, y1);
  if (ACT == MK_ACT_GELU) {
    // erfc(t), t >= 0, to 2^-19 of itself and 2^-22 t^2: s exp(Q(s) - t^2) with s = 1 / (1 + t/2), Q a polynomial of degree 7
    // through the Chebyshev nodes of ln(exp(t^2) erfc(t) / s) on s = 1/16 .. 1.  (With erfcf 2001 x 4096 took 17 us longer.)
    const uint64_t t = pack2(0.70710678118654752f * fabsf(y0), 0.70710678118654752f * fabsf(y1));
    const uint64_t s = rcp2(fma2(splat2(0.5f), t, splat2(1.f)));
    uint64_t q = splat2(-0.185161319f);
    q = fma2(q, s, splat2(0.741661299f));
    q = fma2(q, s, splat2(-0.986141772f));
    q = fma2(q, s, splat2(0.338574501f));
    q = fma2(q, s, splat2(-0.0352274307f));
    q = fma2(q, s, splat2(0.393147085f));
    q = fma2(q, s, splat2(0.998619703f));
    q = fma2(q, s, splat2(-1.26547264f));
    const uint64_t e = ex2_2(mul2(fma2(mul2(t, splat2(-1.f)), t, q), splat2((float)kLog2e)));
    // (y/2 erfc(-t) = y - y/2 erfc(t); an infinite y less 0)
    const float2 half = unpack2(mul2(mul2(pack2(fminf(y0, 1e38f), fminf(y1, 1e38f)), mul2(s, splat2(0.5f))), e));
    y0 = y0 < 0.f ? half.x : y0 - half.x;
    y1 = y1 < 0.f ? half.y : y1 - half.y;
  } else {
    const uint64_t z = ACT == MK_ACT_SILU ? splat2((float)-kLog2e) : fma2(mul2(y, y), splat2((float)(0.044715 * kTanh)), splat2((float)kTanh));
    const float2 r = unpack2(mul2(y, rcp2(add2(ex2_2(mul2(y, z)), splat2(1.f)))));
    y0 = r.x, y1 = r.y;
  }
}

// ... of all of v.  (In registers and unrolled: one value after another through shared memory, 2001 x 4096 with the tanh form
// took 88 us.)
template <int ACT, bool EXACT, int N>
__device__ __forceinline__ void linear_acts(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += EXACT || ACT == MK_ACT_RELU ? 1 : 2) {
    if constexpr (EXACT || ACT == MK_ACT_RELU)
      v[i] = act_exact<ACT>(v[i]);
    else
      act_pair<ACT>(v[i], v[i + 1]);
  }
}
template <bool EXACT, int N>
__device__ __forceinline__ void linear_acts(float (&v)[N], int act) {
  switch (act) {
    case MK_ACT_RELU: linear_acts<MK_ACT_RELU, EXACT>(v); break;
    case MK_ACT_SILU: linear_acts<MK_ACT_SILU, EXACT>(v); break;
    case MK_ACT_GELU: linear_acts<MK_ACT_GELU, EXACT>(v); break;
    case MK_ACT_GELU_TANH: linear_acts<MK_ACT_GELU_TANH, EXACT>(v); break;
  }
}

// Four outputs of a row from column `col` on, `width` of them real (any number): residual, read ahead where it can be, and store.
__device__ __forceinline__ uint2 linear_residual(const LinearEpi& epi, long long row, int col, int width) {
  return epi.vec && epi.residual && width > 0 ? op_ld8(epi.residual + row * epi.residual_stride + col) : make_uint2(0, 0);
}
template <bool WIDE>
__device__ __forceinline__ void linear_put(const LinearEpi& epi, void* out, long long out_stride, const float (&v)[4], uint2 ahead, long long row,
                                           int col, int width) {
  if (width <= 0) return;
  if (epi.vec) {
    float y[4] = {v[0], v[1], v[2], v[3]};
    if (epi.residual) {
      const float2 lo = bf16x2_to_f2(ahead.x), hi = bf16x2_to_f2(ahead.y);
      y[0] += lo.x, y[1] += lo.y, y[2] += hi.x, y[3] += hi.y;
    }
    if (WIDE)
      *reinterpret_cast<float4*>(static_cast<float*>(out) + row * out_stride + col) = make_float4(y[0], y[1], y[2], y[3]);
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + row * out_stride + col) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < width) {
      float y = v[i];
      if (epi.residual) y += bf16_to_f(op_ld2(epi.residual + row * epi.residual_stride + col + i));
      if (WIDE)
        static_cast<float*>(out)[row * out_stride + col + i] = y;
      else
        static_cast<uint16_t*>(out)[row * out_stride + col + i] = to_bf16(y);
    }
}

// Where a lane of a warp that stores 16 rows by 32 outputs at a time has its four pieces (rows lane / 8 + 4 j, outputs 4 (lane % 8)
// on): addresses of the first, bytes from one to the next.  `whole`: 32 outputs that can be read and written four at a time.
struct LinearAt {
  uint8_t* out;
  const uint8_t* res;
  long long out4, res4;
  bool whole;
};
template <bool WIDE>
__device__ __forceinline__ LinearAt linear_at(const mk_expert_args& a, const LinearEpi& epi, long long r0, int w0, int width, int lane) {
  constexpr int kSize = WIDE ? 4 : 2;
  const long long row = r0 + (lane >> 3), col = w0 + 4 * (lane & 7);
  return LinearAt{static_cast<uint8_t*>(a.out) + (row * a.out_stride + col) * kSize,
                  reinterpret_cast<const uint8_t*>(epi.residual + row * epi.residual_stride + col), 4 * a.out_stride * kSize,
                  4 * epi.residual_stride * 2, epi.vec && width >= 32};
}
// the residual of the lane's four pieces
__device__ __forceinline__ void linear_ahead(const LinearEpi& epi, const LinearAt& at, uint2 (&ahead)[4], int rows, int width, int lane) {
  if (!epi.residual || !epi.vec) return;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if ((lane >> 3) + 4 * j < rows && 4 * (lane & 7) < width) ahead[j] = op_ld8(at.res + j * at.res4);
}
// A warp's results v[i] = (row r0 + i, output w0 + lane), i < 16, `rows` and `width` of them real: bias and activation in
// place, then through `stage` (16 x 32 floats of the warp's own) so that eight lanes write 32 outputs of a row side by side.
template <bool WIDE>
__device__ __forceinline__ void linear_store(const mk_expert_args& a, const LinearEpi& epi, const LinearAt& at, float (&v)[16],
                                             const uint2 (&ahead)[4], long long r0, int rows, int w0, int width, float bias, float* stage,
                                             int lane) {
  if (width <= 0) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] += bias;
  linear_acts<WIDE>(v, epi.act);
#pragma unroll
  for (int i = 0; i < 16; ++i) stage[i * 32 + lane] = v[i];
  __syncwarp();
  const float4* const from = reinterpret_cast<const float4*>(stage) + lane;  // (row lane / 8, four outputs)
  if (at.whole && rows >= 16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float4 y = from[j * 32];
      if (epi.residual) {
        const float2 lo = bf16x2_to_f2(ahead[j].x), hi = bf16x2_to_f2(ahead[j].y);
        y.x += lo.x, y.y += lo.y, y.z += hi.x, y.w += hi.y;
      }
      if (WIDE)
        *reinterpret_cast<float4*>(at.out + j * at.out4) = y;
      else
        *reinterpret_cast<uint2*>(at.out + j * at.out4) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
    }
  } else {
    const int col = 4 * (lane & 7);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = (lane >> 3) + 4 * j;
      const float4 y = from[j * 32];
      const float z[4] = {y.x, y.y, y.z, y.w};
      if (r < rows) linear_put<WIDE>(epi, a.out, a.out_stride, z, ahead[j], r0 + r, w0 + col, width - col);
    }
  }
  __syncwarp();
}

}  // namespace mk
