// Device-side helpers of the kernels that walk rows of logits or activations: reductions over a wave, the
// base-2 exponential, and 16-byte pieces of a row at any element offset.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero_internal.h"

namespace zero {

constexpr float kLowest = -3.402823466e38f;

// 2^x for x <= 0: the instruction itself (about one unit in the last place, 0 below 2^-126)
__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }

// Reductions over a wave in a fixed order, by lane moves inside the vector unit: a row's latency is a
// chain of them, and a move through LDS takes several times as long. The result is in every lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ float moved(float v, float none) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none),
                                                               __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, false));
}

template <typename Op>
__device__ __forceinline__ float wave_reduce(float v, float none, Op op) {
  v = op(v, moved<0x111, 0xf>(v, none));  // lanes 1, 2, 4, 8 before, in rows of 16
  v = op(v, moved<0x112, 0xf>(v, none));
  v = op(v, moved<0x114, 0xf>(v, none));
  v = op(v, moved<0x118, 0xf>(v, none));
  v = op(v, moved<0x142, 0xa>(v, none));  // a row's last lane to the next row
  v = op(v, moved<0x143, 0xc>(v, none));  // lane 31 to the upper rows
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

__device__ __forceinline__ float wave_sum(float v) {
  return wave_reduce(v, 0.0f, [](float x, float y) { return x + y; });
}

// The same sum in fp64.
template <int CTRL, int ROWS>
__device__ __forceinline__ double plus_moved(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xf, false);
  return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double wave_sum(double v) {
  v = plus_moved<0x111, 0xf>(v);
  v = plus_moved<0x112, 0xf>(v);
  v = plus_moved<0x114, 0xf>(v);
  v = plus_moved<0x118, 0xf>(v);
  v = plus_moved<0x142, 0xa>(v);
  v = plus_moved<0x143, 0xc>(v);
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 63);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// 16 bytes of a row at any element offset.
template <typename T>
struct Pack {
  static constexpr int n = 16 / sizeof(T);
  typedef T vec __attribute__((ext_vector_type(16 / sizeof(T)), aligned(sizeof(T))));
  typedef vec type;
};

}  // namespace zero
