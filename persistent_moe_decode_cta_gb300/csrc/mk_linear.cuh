// The epilogue of the products in mk_linear: bias, activation, residual and the store.
#pragma once

#include "mk_ops.cuh"

namespace mk {

// act(y).  EXACT: for float32 results; a bf16 result hides the 2^-20 of the approximate exponential and division.
// The tanh form is y / (1 + exp(-2 z)), the erf form y/2 erfc(-y / sqrt 2): both keep their relative precision
// where 1 + tanh or 1 + erf would cancel.
// erfc(t), t >= 0, to 2^-19 of itself and 2^-22 t^2: s exp(Q(s) - t^2) with s = 1 / (1 + t/2), Q a polynomial of degree 7 through the
// Chebyshev nodes of ln(exp(t^2) erfc(t) / s) on s = 1/16 .. 1.  (2001 x 4096 with erfcf: 45.5 us, without an activation 29.)
__device__ __forceinline__ float erfc_fast(float t) {
  const float s = __fdividef(1.f, fmaf(0.5f, t, 1.f));
  float q = -0.185161319f;
  q = fmaf(q, s, 0.741661299f);
  q = fmaf(q, s, -0.986141772f);
  q = fmaf(q, s, 0.338574501f);
  q = fmaf(q, s, -0.0352274307f);
  q = fmaf(q, s, 0.393147085f);
  q = fmaf(q, s, 0.998619703f);
  q = fmaf(q, s, -1.26547264f);
  return s * __expf(fmaf(-t, t, q));
}

template <int ACT, bool EXACT>
__device__ __forceinline__ float linear_act(float y) {
  if (ACT == MK_ACT_NONE) return y;
  if (ACT == MK_ACT_RELU) return y < 0.f ? 0.f : y;  // (NaN stays)
  if (ACT == MK_ACT_GELU) {
    if (EXACT) return 0.5f * y * erfcf(-0.70710678118654752f * y);
    const float half = 0.5f * y * erfc_fast(0.70710678118654752f * fabsf(y));  // (y/2 erfc(-t) = y - y/2 erfc(t))
    return y < 0.f ? half : y - half;
  }
  const float z = ACT == MK_ACT_SILU ? y : 1.5957691216057308f * fmaf(0.044715f * y * y, y, y);
  // y / (1 + exp(-z)): far below zero the exponential overflows and the quotient is zero
  const float e = EXACT ? expf(-z) : __expf(-z);
  return EXACT ? y / (1.f + e) : __fdividef(y, 1.f + e);
}
// ... of all of v.  (In registers and unrolled: one value after another through shared memory, 2001 x 4096 with the tanh form
// took 88 us.)
template <int ACT, bool EXACT, int N>
__device__ __forceinline__ void linear_acts(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = linear_act<ACT, EXACT>(v[i]);
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
