// Matrix products of the linear layer on gfx950: the kernel for a few rows, the join of a product split over
// k, and the launch. Which tile takes a product: zero_gemm_plan.h; the tile kernels: zero_gemm_kernels.hip.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero_gemm.h"

namespace zero {
namespace {

// The workspace's partial sums joined in ascending order, and the epilogue. Bound by memory: 4 bytes a
// split and element.
template <typename T>
__global__ __launch_bounds__(256) void k_join(GemmDev g) {
  const uint32_t groups = (g.n + 7) / 8;
  const uint64_t total = (uint64_t)groups * g.m;
  for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < total; i += gridDim.x * 256ull) {
    const uint64_t m = i / groups;
    const uint32_t n = (uint32_t)(i % groups) * 8;
    typedef float f8 __attribute__((ext_vector_type(8), aligned(4)));
    float z[1][8] = {};
    for (uint32_t s = 0; s < g.splits; ++s) {
      const float* w = g.ws + ((uint64_t)s * g.m + m) * g.n + n;
      if (n + 8 <= g.n) {
        const f8 v = *reinterpret_cast<const f8*>(w);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[0][j] += v[j];
      } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (n + j < g.n) z[0][j] += w[j];
      }
    }
    finish_row<T>(g, z, m, n);
  }
}

// A few rows (16 or 32) times a matrix of k-contiguous rows, where reading that matrix once is all there
// is to do: 16 of its rows a block, straight from memory into the matrix instruction's registers,
// the waves taking turns along k and joined through LDS in their order. No split over blocks, so
// one launch. Any alignment; rows past the end repeat the last one and are not stored. Bound by the
// loads in flight: 8 of a wave and 8 waves a CU on 4096 x 4096, 33.6 MB in 8.9 us (3.8 TB/s; 7.6 us if it was
// read just before); the split tile kernel and its join took 12.
template <typename T, int MT>
__global__ __launch_bounds__(1024) void k_few(GemmDev g) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef T v8 __attribute__((ext_vector_type(8)));
  typedef T v8u __attribute__((ext_vector_type(8), aligned(2)));
  typedef float f4 __attribute__((ext_vector_type(4)));
  constexpr int U = 8;                      // loads in flight per row and wave
  __shared__ float red[16][MT * 16][20];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const uint32_t n0 = blockIdx.x * 16, r = lane & 15;
  const uint32_t kq = (lane >> 4) * 8;
  const uint32_t n = n0 + r < g.n ? n0 + r : g.n - 1;
  const T* w = static_cast<const T*>(g.b) + (uint64_t)n * g.ldb;
  const T* x[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const uint32_t m = t * 16 + r < g.m ? t * 16 + r : g.m - 1;
    x[t] = static_cast<const T*>(g.a) + (uint64_t)m * g.lda;
  }
  f4 acc[MT] = {};
  auto mul = [&](v8 a, const v8* b) {
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      if constexpr (sizeof(T) == 2 && __is_same(T, __bf16))
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[t], acc[t], 0, 0, 0);
      else
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b[t], acc[t], 0, 0, 0);
    }
  };
  for (uint64_t k0 = (uint64_t)wave * (32 * U); k0 < g.k; k0 += (uint64_t)waves * (32 * U)) {
    if (k0 + 32 * U <= g.k) {
      v8 a[U], b[U][MT];
#pragma unroll
      for (int u = 0; u < U; ++u) a[u] = *reinterpret_cast<const v8u*>(w + k0 + u * 32 + kq);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int t = 0; t < MT; ++t) b[u][t] = *reinterpret_cast<const v8u*>(x[t] + k0 + u * 32 + kq);
#pragma unroll
      for (int u = 0; u < U; ++u) mul(a[u], b[u]);
    } else {
      for (uint64_t k1 = k0; k1 < g.k; k1 += 32) {
        const int have = (int)(g.k - k1) - (int)kq;
        v8 a, b[MT];
        if (have >= 8) {
          a = *reinterpret_cast<const v8u*>(w + k1 + kq);
#pragma unroll
          for (int t = 0; t < MT; ++t) b[t] = *reinterpret_cast<const v8u*>(x[t] + k1 + kq);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            a[j] = j < have ? w[k1 + kq + j] : (T)0.0f;
#pragma unroll
            for (int t = 0; t < MT; ++t) b[t][j] = j < have ? x[t][k1 + kq + j] : (T)0.0f;
          }
        }
        mul(a, b);
      }
    }
  }
  // a lane holds 4 neighbouring columns n of row m
#pragma unroll
  for (int t = 0; t < MT; ++t)
    *reinterpret_cast<f4*>(&red[wave][t * 16 + r][(lane >> 4) * 4]) = acc[t];
  __syncthreads();
  for (int i = threadIdx.x; i < MT * 256; i += blockDim.x) {
    float v = red[0][i >> 4][i & 15];
    for (int s = 1; s < waves; ++s) v += red[s][i >> 4][i & 15];
    red[0][i >> 4][i & 15] = v;
  }
  __syncthreads();
  const uint32_t m = threadIdx.x >> 1, nn = n0 + (threadIdx.x & 1) * 8;
  if (m < MT * 16 && m < g.m && nn < g.n) {
    float z[1][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) z[0][j] = red[0][m][(threadIdx.x & 1) * 8 + j];
    finish_row<T>(g, z, m, nn);
  }
#endif
}

constexpr uint32_t kFewRows = 32;
bool few(const GemmArgs& g) { return g.m <= kFewRows && !g.a_kmajor && !g.b_kmajor; }

template <typename T>
hipError_t run_few(const GemmDev& d, hipStream_t s) {
  const uint32_t blocks = (d.n + 15) / 16;
  uint32_t waves = 2048 / blocks;
  const uint32_t most = (d.k + 255) / 256;
  waves = waves > most ? most : waves;
  waves = waves < 4 ? 4 : waves > 16 ? 16 : waves;
  if (d.m <= 16) k_few<T, 1><<<dim3(blocks), dim3(waves * 64), 0, s>>>(d);
  else k_few<T, 2><<<dim3(blocks), dim3(waves * 64), 0, s>>>(d);
  return hipGetLastError();
}

// Whether an operand can be loaded straight to LDS: those loads want whole dwords, not 16 bytes (4096 x
// 4100 x 4100 forward 178 us, 295 through registers). The row pitch keeps a tile's offsets in 32 bits.
bool direct(const void* p, uint64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % 4 == 0 && ld % 2 == 0 && ld <= (1u << 22);
}

}  // namespace

uint64_t gemm_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, bool kmajor) {
  if (!m || !n || (m <= kFewRows && !kmajor)) return 0;
  const Plan p = plan(m, n, k);
  return p.splits > 1 ? p.splits * m * n * 4 : 0;
}

#define ZERO_TILES(d, a, b) hipError_t gemm_tiles_##d##a##b(const GemmDev&, int, bool, hipStream_t);
ZERO_TILES(1, 0, 0) ZERO_TILES(1, 0, 1) ZERO_TILES(1, 1, 1)
ZERO_TILES(2, 0, 0) ZERO_TILES(2, 0, 1) ZERO_TILES(2, 1, 1)

hipError_t gemm(const GemmArgs& g, hipStream_t s) {
  const bool bf = g.dtype == ZERO_BF16;
  GemmDev d{};
  d.a = g.a, d.b = g.b, d.bias = g.bias, d.res = g.res, d.pre = g.pre, d.out = g.out, d.ws = g.ws;
  d.lda = g.lda, d.ldb = g.ldb, d.ldr = g.ldr, d.ldp = g.ldp, d.ldo = g.ldo;
  d.m = g.m, d.n = g.n, d.k = g.k;
  d.splits = 1;
  d.act = g.act, d.accumulate = g.accumulate, d.out_f32 = g.out_dtype == ZERO_F32;
  if (few(g)) return bf ? run_few<__bf16>(d, s) : run_few<_Float16>(d, s);

  const bool dir = direct(g.a, g.lda) && direct(g.b, g.ldb);
  Plan p = plan(g.m, g.n, g.k);
  uint64_t tiles_m, tiles_n;
  if (!place(g.m, g.n, dir, p, tiles_m, tiles_n)) return hipErrorInvalidConfiguration;
  d.tiles_m = (uint32_t)tiles_m, d.tiles_n = (uint32_t)tiles_n;
  d.splits = p.splits, d.k_split = p.k_split;
  hipError_t e;
  if (!g.a_kmajor && !g.b_kmajor) e = bf ? gemm_tiles_200(d, p.shape, dir, s) : gemm_tiles_100(d, p.shape, dir, s);
  else if (!g.a_kmajor) e = bf ? gemm_tiles_201(d, p.shape, dir, s) : gemm_tiles_101(d, p.shape, dir, s);
  else e = bf ? gemm_tiles_211(d, p.shape, dir, s) : gemm_tiles_111(d, p.shape, dir, s);
  if (e != hipSuccess || d.splits == 1) return e;
  const uint64_t work = ((uint64_t)d.n + 7) / 8 * d.m;
  const unsigned blocks = (unsigned)((work + 255) / 256 < 4096 ? (work + 255) / 256 : 4096);
  if (bf) k_join<__bf16><<<dim3(blocks), dim3(256), 0, s>>>(d);
  else k_join<_Float16><<<dim3(blocks), dim3(256), 0, s>>>(d);
  return hipGetLastError();
}

}  // namespace zero
