// Matrix products of the linear layer on gfx950.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero_gemm.h"

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

// The workspace's partial sums joined in ascending order, and the epilogue.
template <typename T>
__global__ __launch_bounds__(256) void k_join(GemmDev g) {
  const uint32_t groups = (g.n + 7) / 8;
  const uint64_t total = (uint64_t)groups * g.m;
  for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < total; i += gridDim.x * 256ull) {
    const uint64_t m = i / groups;
    const uint32_t n = (uint32_t)(i % groups) * 8;
    typedef float f8 __attribute__((ext_vector_type(8), aligned(4)));
    float z[8] = {};
    for (uint32_t s = 0; s < g.splits; ++s) {
      const float* w = g.ws + ((uint64_t)s * g.m + m) * g.n + n;
      if (n + 8 <= g.n) {
        const f8 v = *reinterpret_cast<const f8*>(w);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] += v[j];
      } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (n + j < g.n) z[j] += w[j];
      }
    }
    finish_row<T>(g, z, m, n);
  }
}

struct TileShape {
  uint32_t bm, bn, per_cu;
  float cost;  // time of one step of one tile, relative
};
constexpr TileShape kShapes[] = {{256, 256, 1, 1.0f}, {128, 128, 2, 0.30f}};
constexpr int kNumShapes = sizeof(kShapes) / sizeof(kShapes[0]);
constexpr uint32_t kCus = 256;

struct Plan {
  int shape;
  uint32_t splits, k_split;
};

Plan plan(uint64_t m, uint64_t n, uint64_t k) {
  Plan best{0, 1, 0};
  float best_t = 1e30f;
  const uint64_t steps = k ? (k + kGemmStep - 1) / kGemmStep : 1;
  best.k_split = (uint32_t)(steps * kGemmStep);
  for (int i = 0; i < kNumShapes; ++i) {
    const TileShape& t = kShapes[i];
    const uint64_t tiles = ((m + t.bm - 1) / t.bm) * ((n + t.bn - 1) / t.bn);
    for (uint64_t sp = 1; sp <= 16 && (sp == 1 || steps / sp >= 4); ++sp) {
      const uint64_t per = (steps + sp - 1) / sp;
      const uint64_t slots = kCus * t.per_cu;
      const uint64_t rounds = (tiles * sp + slots - 1) / slots;
      // k_join and the workspace's write and read, in units of a 256 x 256 x 64 step (about 1.2 us)
      const float join = sp > 1 ? 3.0f + (float)(m * n * sp * 8) / 8e6f : 0.0f;
      const float time = (float)(rounds * (per + 4)) * t.cost * t.per_cu + join;
      if (time < best_t) {
        best_t = time;
        best = Plan{i, (uint32_t)((steps + per - 1) / per), (uint32_t)(per * kGemmStep)};
      }
    }
  }
  return best;
}

bool direct(const void* p, uint64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0 && ld <= (1u << 22);
}



}  // namespace

uint64_t gemm_workspace_bytes(uint64_t m, uint64_t n, uint64_t k) {
  if (!m || !n) return 0;
  const Plan p = plan(m, n, k);
  return p.splits > 1 ? p.splits * m * n * 4 : 0;
}

#define ZERO_TILES(d, a, b) hipError_t gemm_tiles_##d##a##b(const GemmDev&, int, hipStream_t);
ZERO_TILES(1, 0, 0) ZERO_TILES(1, 0, 1) ZERO_TILES(1, 1, 1)
ZERO_TILES(2, 0, 0) ZERO_TILES(2, 0, 1) ZERO_TILES(2, 1, 1)

hipError_t gemm(const GemmArgs& g, hipStream_t s) {
  if (!direct(g.a, g.lda) || !direct(g.b, g.ldb)) {
    if (g.dtype == ZERO_BF16)
      return g.out_dtype == ZERO_F32 ? launch<__bf16, float>(g, s) : launch<__bf16, __bf16>(g, s);
    return g.out_dtype == ZERO_F32 ? launch<_Float16, float>(g, s) : launch<_Float16, _Float16>(g, s);
  }
  Plan p = plan(g.m, g.n, g.k);
  GemmDev d{};
  d.a = g.a, d.b = g.b, d.bias = g.bias, d.res = g.res, d.pre = g.pre, d.out = g.out, d.ws = g.ws;
  d.lda = g.lda, d.ldb = g.ldb, d.ldr = g.ldr, d.ldp = g.ldp, d.ldo = g.ldo;
  d.m = g.m, d.n = g.n, d.k = g.k;
  d.tiles_m = (g.m + kShapes[p.shape].bm - 1) / kShapes[p.shape].bm;
  d.tiles_n = (g.n + kShapes[p.shape].bn - 1) / kShapes[p.shape].bn;
  d.splits = p.splits, d.k_split = p.k_split;
  d.act = g.act, d.accumulate = g.accumulate, d.out_f32 = g.out_dtype == ZERO_F32;
  if ((uint64_t)d.tiles_m * d.tiles_n > 0x7fffffffu) return hipErrorInvalidConfiguration;
  const bool bf = g.dtype == ZERO_BF16;
  hipError_t e;
  if (!g.a_kmajor && !g.b_kmajor) e = bf ? gemm_tiles_200(d, p.shape, s) : gemm_tiles_100(d, p.shape, s);
  else if (!g.a_kmajor) e = bf ? gemm_tiles_201(d, p.shape, s) : gemm_tiles_101(d, p.shape, s);
  else e = bf ? gemm_tiles_211(d, p.shape, s) : gemm_tiles_111(d, p.shape, s);
  if (e != hipSuccess || d.splits == 1) return e;
  const uint64_t work = ((uint64_t)d.n + 7) / 8 * d.m;
  const unsigned blocks = (unsigned)((work + 255) / 256 < 4096 ? (work + 255) / 256 : 4096);
  if (bf) k_join<__bf16><<<dim3(blocks), dim3(256), 0, s>>>(d);
  else k_join<_Float16><<<dim3(blocks), dim3(256), 0, s>>>(d);
  return hipGetLastError();
}

}  // namespace zero
