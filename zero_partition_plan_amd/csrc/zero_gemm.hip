// Matrix products of the linear layer on gfx950.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero_gemm.h"

namespace zero {
namespace {

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
constexpr TileShape kShapes[] = {{256, 256, 1, 1.0f},  {128, 256, 1, 0.58f}, {256, 128, 1, 0.58f},
                                 {128, 128, 2, 0.30f}, {64, 256, 2, 0.32f},  {32, 256, 2, 0.22f},
                                 {64, 64, 5, 0.10f}};
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

#define ZERO_TILES(d, a, b) hipError_t gemm_tiles_##d##a##b(const GemmDev&, int, bool, hipStream_t);
ZERO_TILES(1, 0, 0) ZERO_TILES(1, 0, 1) ZERO_TILES(1, 1, 1)
ZERO_TILES(2, 0, 0) ZERO_TILES(2, 0, 1) ZERO_TILES(2, 1, 1)

hipError_t gemm(const GemmArgs& g, hipStream_t s) {
  const bool dir = direct(g.a, g.lda) && direct(g.b, g.ldb);
  Plan p = plan(g.m, g.n, g.k);
  if (!dir && p.shape == 0) p.shape = 1;  // the same splits, so the same workspace
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
