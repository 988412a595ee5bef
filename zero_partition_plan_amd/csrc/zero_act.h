// The linear layer's activations on the device. fp32 arithmetic; the results are rounded to 16 bits by the
// caller, so the hardware's exp2 and reciprocal (about one unit in the last fp32 place each) are far below what
// is kept. Gates are formed so that they keep that accuracy where they are small: (1 + erf u)/2 by the
// upper tail of the normal distribution (the sum has lost every digit at z = -5.75, where the result is still a bf16
// of -2.6e-8), (1 + tanh u)/2 as the sigmoid of 2u.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero_shard.h"

namespace zero {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kGeluC = 0.79788456080286535588f;  // sqrt(2/pi)
constexpr float kGeluA = 0.044715f;

// 1 / (1 + exp(-z)); 0 and 1 at the infinities
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * z));
}

// The normal distribution's (1 + erf(z/sqrt 2))/2, and exp(-z^2/2). The tail beyond a = |z|
// times exp(a^2/2) falls smoothly from 1/2 and as 1/a far out: a polynomial in t = 1/(1 + 0.305 a) without constant term,
// its coefficients fitted for the least relative error on [0, 14] (9.4e-8; past 13.2 exp2 gives 0). One reciprocal, one
// exp2 and no branch: 4096 x 4096 -> 11008 with gelu 328 us, 368 us with the math library's erfc, and 341 us with its
// erf, which cancels.
struct Normal {
  float cdf, e;
};
__device__ __forceinline__ Normal normal(float z) {
  const float a = __builtin_fabsf(z);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.305f, a, 1.0f));
  const float e = __builtin_amdgcn_exp2f(-0.5f * kLog2e * (z * z));
  float p = 0.0366991907f;
  p = __builtin_fmaf(p, t, -0.1529883f);
  p = __builtin_fmaf(p, t, 0.185716867f);
  p = __builtin_fmaf(p, t, -0.0379767939f);
  p = __builtin_fmaf(p, t, 0.121021658f);
  p = __builtin_fmaf(p, t, 0.103420876f);
  p = __builtin_fmaf(p, t, 0.122466817f);
  p = __builtin_fmaf(p, t, 0.121639736f);
  const float q = p * t * e;
  return Normal{z < 0.0f ? q : 1.0f - q, e};
}

template <int ACT>
__device__ __forceinline__ float act(float z) {
  if constexpr (ACT == ZERO_ACT_RELU) return z < 0.0f ? 0.0f : z;  // keeps a NaN
  if constexpr (ACT == ZERO_ACT_GELU) return z * normal(z).cdf;
  // (1 + tanh u)/2 = sigmoid(2u)
  if constexpr (ACT == ZERO_ACT_GELU_TANH)
    return z * sigmoid(2.0f * kGeluC * __builtin_fmaf(kGeluA * z * z, z, z));
  if constexpr (ACT == ZERO_ACT_SILU) return z * sigmoid(z);
  return z;
}

// The slope. Past 1000 every one is 0 or 1 in fp32 already; beyond, and at the infinities that an overflow of the
// stored type leaves, its second term would multiply 0 by an infinity. Keeps a NaN.
constexpr float kFar = 1000.0f;

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  z = z > kFar ? kFar : (z < -kFar ? -kFar : z);
  if constexpr (ACT == ZERO_ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  if constexpr (ACT == ZERO_ACT_GELU) {
    const Normal n = normal(z);
    return __builtin_fmaf(z * 0.39894228040143267794f, n.e, n.cdf);  // density exp(-z^2/2)/sqrt(2 pi)
  }
  if constexpr (ACT == ZERO_ACT_GELU_TANH) {
    const float z2 = z * z;
    const float s = sigmoid(2.0f * kGeluC * __builtin_fmaf(kGeluA * z2, z, z));
    const float du = 2.0f * kGeluC * __builtin_fmaf(3.0f * kGeluA, z2, 1.0f);
    return __builtin_fmaf(z * s * (1.0f - s), du, s);
  }
  if constexpr (ACT == ZERO_ACT_SILU) {
    const float s = sigmoid(z);
    return __builtin_fmaf(z * s, 1.0f - s, s);
  }
  return 1.0f;
}

// The activation chosen at run time (uniform over the launch), for N values at once: one branch, and
// each activation's code once per kernel.
template <int ACT, int N>
__device__ __forceinline__ void act_all(float* z) {
#pragma unroll
  for (int j = 0; j < N; ++j) z[j] = act<ACT>(z[j]);
}

template <int N>
__device__ __forceinline__ void act_rt(float* z, int a) {
  switch (a) {
    case ZERO_ACT_RELU: act_all<ZERO_ACT_RELU, N>(z); break;
    case ZERO_ACT_GELU: act_all<ZERO_ACT_GELU, N>(z); break;
    case ZERO_ACT_GELU_TANH: act_all<ZERO_ACT_GELU_TANH, N>(z); break;
    case ZERO_ACT_SILU: act_all<ZERO_ACT_SILU, N>(z); break;
    default: break;
  }
}

}  // namespace zero
