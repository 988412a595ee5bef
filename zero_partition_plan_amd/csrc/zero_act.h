// The linear layer's activations on the device, and 16-bit conversions. fp32 arithmetic; the results
// are rounded to 16 bits by the caller, so the hardware's exp2 and reciprocal (about one unit in the last
// fp32 place each) are far below what is kept.
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

template <int ACT>
__device__ __forceinline__ float act(float z) {
  if constexpr (ACT == ZERO_ACT_RELU) return z < 0.0f ? 0.0f : z;  // keeps a NaN
  if constexpr (ACT == ZERO_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752440f));
  // (1 + tanh u)/2 = sigmoid(2u)
  if constexpr (ACT == ZERO_ACT_GELU_TANH)
    return z * sigmoid(2.0f * kGeluC * __builtin_fmaf(kGeluA * z * z, z, z));
  if constexpr (ACT == ZERO_ACT_SILU) return z * sigmoid(z);
  return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == ZERO_ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  if constexpr (ACT == ZERO_ACT_GELU) {
    const float cdf = 0.5f * (1.0f + erff(z * 0.70710678118654752440f));
    // density exp(-z^2/2)/sqrt(2 pi)
    return __builtin_fmaf(z * 0.39894228040143267794f,
                          __builtin_amdgcn_exp2f(-0.5f * kLog2e * z * z), cdf);
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
