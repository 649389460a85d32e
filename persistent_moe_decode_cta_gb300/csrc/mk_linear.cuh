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
template <int N>
__device__ __forceinline__ void linear_acts(float (&v)[N], int act, bool exact) {
  if (exact)
    linear_acts<true>(v, act);
  else
    linear_acts<false>(v, act);
}

// Four outputs of a row from column `col` on, `width` of them real (any number): residual and store.
__device__ __forceinline__ void linear_put(const LinearEpi& epi, void* out, long long out_stride, const float (&v)[4], long long row, int col,
                                           int width) {
  if (width <= 0) return;
  const uint16_t* const res = epi.residual + row * epi.residual_stride + col;
  float y[4] = {v[0], v[1], v[2], v[3]};
  if (epi.vec) {
    if (epi.residual) {
      const uint2 u = op_ld8(res);
      const float2 lo = bf16x2_to_f2(u.x), hi = bf16x2_to_f2(u.y);
      y[0] += lo.x, y[1] += lo.y, y[2] += hi.x, y[3] += hi.y;
    }
    if (epi.out_float)
      *reinterpret_cast<float4*>(static_cast<float*>(out) + row * out_stride + col) = make_float4(y[0], y[1], y[2], y[3]);
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + row * out_stride + col) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < width) {
      if (epi.residual) y[i] += bf16_to_f(op_ld2(res + i));
      if (epi.out_float)
        static_cast<float*>(out)[row * out_stride + col + i] = y[i];
      else
        static_cast<uint16_t*>(out)[row * out_stride + col + i] = to_bf16(y[i]);
    }
}

// A warp's results v[i] = (row r0 + i, output w0 + lane), i < 16, `rows` and `width` of them real: bias and activation in
// place, then through `stage` (16 x 32 floats of the warp's own) so that eight lanes write 32 outputs of a row side by side.
__device__ __forceinline__ void linear_store(const mk_expert_args& a, const LinearEpi& epi, float (&v)[16], long long r0, int rows, int w0,
                                             int width, float* stage, int lane) {
  if (width <= 0) return;
  const float b = epi.bias && lane < width ? bf16_to_f(op_ld2(epi.bias + w0 + lane)) : 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] += b;
  linear_acts(v, epi.act, epi.out_float != 0);
#pragma unroll
  for (int i = 0; i < 16; ++i) stage[i * 32 + lane] = v[i];
  __syncwarp();
  const int col = 4 * (lane & 7);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = (lane >> 3) + 4 * j;
    const float4 y = *reinterpret_cast<const float4*>(stage + r * 32 + col);
    const float z[4] = {y.x, y.y, y.z, y.w};
    if (r < rows) linear_put(epi, a.out, a.out_stride, z, r0 + r, w0 + col, width - col);
  }
  __syncwarp();
}

}  // namespace mk
