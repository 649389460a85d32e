// The epilogue of the products in mk_linear: bias, activation, residual and the store.
#pragma once

#include "mk_ops.cuh"

namespace mk {

// act(y).  EXACT: for float32 results; a bf16 result hides the 2^-20 of the approximate exponential and division.
// The tanh form is y / (1 + exp(-2 z)), the erf form y/2 erfc(-y / sqrt 2): both keep their relative precision
// where 1 + tanh or 1 + erf would cancel.
template <int ACT, bool EXACT>
__device__ __forceinline__ float linear_act(float y) {
  if (ACT == MK_ACT_NONE) return y;
  if (ACT == MK_ACT_RELU) return y < 0.f ? 0.f : y;  // (NaN stays)
  if (ACT == MK_ACT_GELU) return 0.5f * y * erfcf(-0.70710678118654752f * y);
  const float z = ACT == MK_ACT_SILU ? y : 1.5957691216057308f * fmaf(0.044715f * y * y, y, y);
  // y / (1 + exp(-z)): far below zero the exponential overflows and the quotient is zero
  const float e = EXACT ? expf(-z) : __expf(-z);
  return EXACT ? y / (1.f + e) : __fdividef(y, 1.f + e);
}
// ... of all of v + b.  (In registers and unrolled: one value after another, 2001 x 4096 with the tanh form took 88 us.)
template <int ACT, bool EXACT, int N>
__device__ __forceinline__ void linear_acts(float (&v)[N], float b) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = linear_act<ACT, EXACT>(v[i] + b);
}
template <bool EXACT, int N>
__device__ __forceinline__ void linear_acts(float (&v)[N], float b, int act) {
  switch (act) {
    case MK_ACT_RELU: linear_acts<MK_ACT_RELU, EXACT>(v, b); break;
    case MK_ACT_SILU: linear_acts<MK_ACT_SILU, EXACT>(v, b); break;
    case MK_ACT_GELU: linear_acts<MK_ACT_GELU, EXACT>(v, b); break;
    case MK_ACT_GELU_TANH: linear_acts<MK_ACT_GELU_TANH, EXACT>(v, b); break;
    default: linear_acts<MK_ACT_NONE, EXACT>(v, b);
  }
}

// A warp's results v[i] = (row r0 + i, output w0 + lane), i < 32, `rows` and `width` of them real: bias and activation in
// place, then through `stage` (32 x 32 floats of the warp's own) so that eight lanes write 32 outputs of a row side by side.
__device__ __forceinline__ void linear_store(const mk_expert_args& a, const LinearEpi& epi, float (&v)[32], long long r0, int rows, int w0,
                                             int width, float* stage, int lane) {
  if (width <= 0) return;
  const bool wide = epi.out_float != 0;
  const uint16_t* const res = epi.residual + r0 * epi.residual_stride + w0;
  const int col = 4 * (lane & 7), row = lane >> 3;
  uint2 add[8];
  if (epi.vec && epi.residual) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (row + 4 * j < rows && col < width) add[j] = op_ld8(res + (row + 4 * j) * epi.residual_stride + col);
  }
  const float b = epi.bias && lane < width ? bf16_to_f(op_ld2(epi.bias + w0 + lane)) : 0.f;
  if (wide)
    linear_acts<true>(v, b, epi.act);
  else
    linear_acts<false>(v, b, epi.act);
#pragma unroll
  for (int i = 0; i < 32; ++i) stage[i * 32 + lane] = v[i];
  __syncwarp();
  if (epi.vec) {
    if (col < width) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = row + 4 * j;
        if (r >= rows) break;
        float4 y = *reinterpret_cast<const float4*>(stage + r * 32 + col);
        if (epi.residual) {
          const float2 lo = bf16x2_to_f2(add[j].x), hi = bf16x2_to_f2(add[j].y);
          y.x += lo.x, y.y += lo.y, y.z += hi.x, y.w += hi.y;
        }
        const long long at = (r0 + r) * a.out_stride + w0 + col;
        if (wide)
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = y;
        else
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
      }
    }
  } else if (lane < width) {
    for (int r = 0; r < rows; ++r) {
      float y = stage[r * 32 + lane];
      if (epi.residual) y += bf16_to_f(op_ld2(res + r * epi.residual_stride + lane));
      const long long at = (r0 + r) * a.out_stride + w0 + lane;
      if (wide)
        static_cast<float*>(a.out)[at] = y;
      else
        static_cast<uint16_t*>(a.out)[at] = to_bf16(y);
    }
  }
  __syncwarp();
}

}  // namespace mk
