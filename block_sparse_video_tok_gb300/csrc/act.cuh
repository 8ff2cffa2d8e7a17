// act.cuh -- the activations of vsa_linear and their slopes, in fp32, and 16-bit conversions.
//
// The logistic function takes one fast exponential and one fast division: together good to about
// 2^-20 relative where the result is above 2^-20, against the 2^-8 or 2^-11 of the 16-bit results.
// The normal distribution goes through erfc, whose relative precision holds into the lower tail.
#pragma once

#include "block_internal.cuh"

namespace vsa {

constexpr float GELU_C = 0.7978845608028654f, GELU_D = 0.044715f;  // sqrt(2 / pi)

__device__ __forceinline__ float logistic(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }
__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(-0.7071067811865476f * z); }

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if (ACT == VSA_GELU) return z * normal_cdf(z);
  if (ACT == VSA_GELU_TANH) return z * logistic(2.f * GELU_C * fmaf(GELU_D * z * z, z, z));
  if (ACT == VSA_SILU) return z * logistic(z);
  return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if (ACT == VSA_GELU) return fmaf(z * 0.3989422804014327f, __expf(-0.5f * z * z), normal_cdf(z));
  if (ACT == VSA_GELU_TANH) {
    const float zz = z * z, s = logistic(2.f * GELU_C * fmaf(GELU_D * zz, z, z));
    return fmaf(2.f * GELU_C * z * fmaf(3.f * GELU_D, zz, 1.f), s * (1.f - s), s);
  }
  if (ACT == VSA_SILU) {
    const float s = logistic(z);
    return s * fmaf(z, 1.f - s, 1.f);
  }
  return 1.f;
}

// 8 values at once, the activation known at run time only: z = act(z), z *= act'(at).
__device__ __forceinline__ void act8(int act, float* z) {
  if (act == VSA_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = act_value<VSA_GELU_TANH>(z[i]);
  } else if (act == VSA_SILU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = act_value<VSA_SILU>(z[i]);
  } else if (act == VSA_GELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = act_value<VSA_GELU>(z[i]);
  }
}
__device__ __forceinline__ void slope8(int act, const float* at, float* z) {
  if (act == VSA_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] *= act_slope<VSA_GELU_TANH>(at[i]);
  } else if (act == VSA_SILU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] *= act_slope<VSA_SILU>(at[i]);
  } else if (act == VSA_GELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] *= act_slope<VSA_GELU>(at[i]);
  }
}

__device__ __forceinline__ void narrow(float v, __nv_bfloat16* p) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void narrow(float v, __half* p) { *p = __float2half_rn(v); }

}  // namespace vsa
