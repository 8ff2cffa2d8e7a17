// act.cuh -- the activations of vsa_linear and their slopes, in fp32.
//
// The logistic function is one fast exponential and one fast reciprocal.  The normal distribution is
//   Phi(-a) = exp(-a^2 / 2) t P(t),  t = 1 / (1 + 0.36 a),  a >= 0,
// with P a polynomial of degree 6 fitted here to exp(a^2 / 2) Phi(-a) / t by least squares reweighted
// towards the largest relative error (at most 2^-20 for a up to 14, where Phi leaves the range of
// fp32), so its lower tail keeps the results' precision; its slope's exp(-z^2 / 2) is the same one.  All
// are good to about 2^-18 relative, exponents of a size x to x 2^-23 more, against the 2^-8 or 2^-11 of the
// 16-bit results; a logistic function below 2^-126 is 0.  (With the library's erfc in its place the product
// 32760 x 1536 x 6144 took 775 us with gelu, 366 with silu.)
#pragma once

#include "block_internal.cuh"
#include "cross_common.cuh"

namespace vsa {

constexpr float GELU_C = 0.7978845608028654f, GELU_D = 0.044715f;  // sqrt(2 / pi)

__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / (1 + 2^-x): the logistic function of x / log2(e).
__device__ __forceinline__ float logistic2(float x) { return reciprocal(1.f + ex2(-x)); }

// Phi(z), and exp(-z^2 / 2).
__device__ __forceinline__ float normal_cdf(float z, float* bell) {
  const float a = fabsf(z), t = reciprocal(fmaf(0.36f, a, 1.f));
  float q = fmaf(0.047056187f, t, -0.17976487f);
  q = fmaf(q, t, 0.18095505f);
  q = fmaf(q, t, 0.026548008f);
  q = fmaf(q, t, 0.13971997f);
  q = fmaf(q, t, 0.14177228f);
  q = fmaf(q, t, 0.14371306f);
  *bell = ex2(-0.5f * LOG2E_F * z * z);
  const float tail = *bell * (t * q);
  return z < 0.f ? tail : 1.f - tail;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if (ACT == VSA_GELU) {
    float bell;
    return z * normal_cdf(z, &bell);
  }
  if (ACT == VSA_GELU_TANH) return z * logistic2(z * fmaf(2.f * LOG2E_F * GELU_C * GELU_D, z * z, 2.f * LOG2E_F * GELU_C));
  if (ACT == VSA_SILU) return z * logistic2(LOG2E_F * z);
  return z;
}

// The slopes are 0 or 1 from 104 on (the exponentials of all three have left fp32's range), so z is taken
// there from beyond: the polynomials' powers of it would overflow and meet a factor of 0, gelu_tanh's at
// 1.2e13, all at the infinities (which a finite z becomes where pre is rounded to fp16).  NaN stays.  One
// instruction, the smaller magnitude with z's sign: within the noise of every backward measured.
__device__ __forceinline__ float bounded(float z) {
  float y;
  asm("min.NaN.xorsign.abs.f32 %0, %1, 0f42D00000;" : "=f"(y) : "f"(z));
  return y;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  z = bounded(z);
  if (ACT == VSA_GELU) {
    float bell;
    const float cdf = normal_cdf(z, &bell);
    return fmaf(z * 0.3989422804014327f, bell, cdf);
  }
  if (ACT == VSA_GELU_TANH) {
    const float zz = z * z, s = logistic2(z * fmaf(2.f * LOG2E_F * GELU_C * GELU_D, zz, 2.f * LOG2E_F * GELU_C));
    return fmaf(z * fmaf(6.f * GELU_C * GELU_D, zz, 2.f * GELU_C), s * (1.f - s), s);
  }
  if (ACT == VSA_SILU) {
    const float s = logistic2(LOG2E_F * z);
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

__device__ __forceinline__ float widen16(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float widen16(__half v) { return __half2float(v); }
__device__ __forceinline__ void narrow(float v, __nv_bfloat16* p) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void narrow(float v, __half* p) { *p = __float2half_rn(v); }

}  // namespace vsa
