// Matrix products of the linear layer on gfx950.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero_act.h"
#include "zero_linear.h"

namespace zero {
namespace {

struct Operand {
  const void* p;
  uint64_t srow, sk;  // strides of the row and of k, in elements
};

template <typename T, typename O>
__global__ __launch_bounds__(256) void k_mm(Operand a, Operand b, GemmArgs g) {
  __shared__ float sa[16][65], sb[16][65];
  const uint32_t tiles_n = (g.n + 63) / 64;
  const uint32_t m0 = blockIdx.x / tiles_n * 64, n0 = blockIdx.x % tiles_n * 64;
  const T* pa = static_cast<const T*>(a.p);
  const T* pb = static_cast<const T*>(b.p);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (uint32_t k0 = 0; k0 < g.k; k0 += 16) {
    for (int i = threadIdx.x; i < 64 * 16; i += 256) {
      const uint32_t r = i / 16, k = i % 16;
      const bool ka = k0 + k < g.k;
      sa[k][r] = ka && m0 + r < g.m ? (float)pa[(m0 + r) * a.srow + (k0 + k) * a.sk] : 0.0f;
      sb[k][r] = ka && n0 + r < g.n ? (float)pb[(n0 + r) * b.srow + (k0 + k) * b.sk] : 0.0f;
    }
    __syncthreads();
    for (int k = 0; k < 16; ++k)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const uint64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m >= g.m || n >= g.n) continue;
      float z = acc[i][j];
      if (g.bias) z += (float)static_cast<const T*>(g.bias)[n];
      if (g.pre) static_cast<T*>(g.pre)[m * g.ldp + n] = (T)z;
      z = act_rt(z, g.act);
      if (g.res) z += (float)static_cast<const T*>(g.res)[m * g.ldr + n];
      O* out = static_cast<O*>(g.out) + m * g.ldo + n;
      if (g.accumulate) z += (float)*out;
      *out = (O)z;
    }
}

template <typename T, typename O>
hipError_t launch(const GemmArgs& g, hipStream_t s) {
  const Operand a{g.a, g.a_kmajor ? 1 : g.lda, g.a_kmajor ? g.lda : 1};
  const Operand b{g.b, g.b_kmajor ? 1 : g.ldb, g.b_kmajor ? g.ldb : 1};
  const uint64_t tiles = (uint64_t)((g.m + 63) / 64) * ((g.n + 63) / 64);
  if (tiles > 0x7fffffffu) return hipErrorInvalidConfiguration;
  k_mm<T, O><<<dim3((unsigned)tiles), dim3(256), 0, s>>>(a, b, g);
  return hipGetLastError();
}

}  // namespace

uint64_t gemm_workspace_bytes(uint64_t, uint64_t, uint64_t) { return 0; }

hipError_t gemm(const GemmArgs& g, hipStream_t s) {
  if (g.dtype == ZERO_BF16)
    return g.out_dtype == ZERO_F32 ? launch<__bf16, float>(g, s) : launch<__bf16, __bf16>(g, s);
  return g.out_dtype == ZERO_F32 ? launch<_Float16, float>(g, s) : launch<_Float16, _Float16>(g, s);
}

}  // namespace zero
