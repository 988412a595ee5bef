// Device side of the matrix product: what its tile kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero_act.h"
#include "zero_gemm_plan.h"
#include "zero_linear.h"

namespace zero {

struct GemmDev {
  const void *a, *b, *bias, *res;
  void *pre, *out;
  float* ws;            // [splits][m][n] partial sums when splits > 1
  uint64_t lda, ldb, ldr, ldp, ldo;
  uint32_t m, n, k;
  uint32_t tiles_m, tiles_n, splits, k_split;
  int32_t act, accumulate, out_f32;
};

// The tile a workgroup takes. Workgroups go round the 8 XCDs in turn, each with its own L2: each
// XCD gets one contiguous run of tiles, and a run walks 8 tile rows at a time down the columns, so
// that the tiles in flight on one XCD share their operands' panels.
__device__ __forceinline__ void tile_of(const GemmDev& g, uint32_t id, uint32_t& mt, uint32_t& nt) {
  const uint32_t total = g.tiles_m * g.tiles_n;
  const uint32_t x = id & 7, q = total >> 3, rem = total & 7;
  id = x * q + (x < rem ? x : rem) + (id >> 3);
  const uint32_t group = 8 * g.tiles_n;
  const uint32_t first = id / group * 8;
  const uint32_t rows = g.tiles_m - first < 8 ? g.tiles_m - first : 8;
  const uint32_t in = id % group;
  mt = first + in % rows;
  nt = in / rows;
}

// Where an operand's next step begins, and the bytes from there to the last element that the tile
// uses of it: what the loads are checked against. Everything but the address fits in 32 bits, as a
// tile spans at most 256 rows of at most 2^22 elements. Sizes are rounded up to whole words, the
// second half of a last word belonging to no row that is used.
template <typename T, bool KM, int R>
struct Cursor {
  const T* p;
  uint32_t fixed, ld2;
  uint64_t by;
  __device__ __forceinline__ Cursor(const void* base, uint64_t ld, uint32_t row0, uint32_t rows,
                                    uint32_t k0) {
    p = static_cast<const T*>(base) + (KM ? (uint64_t)k0 * ld + row0 : (uint64_t)row0 * ld + k0);
    const uint32_t here = rows - row0 < R ? rows - row0 : R;
    fixed = KM ? (here * 2 + 3) & ~3u : (here - 1) * (uint32_t)ld * 2;
    ld2 = (uint32_t)ld * 2;
    by = KM ? kGemmStep * ld : kGemmStep;
  }
  __device__ __forceinline__ void advance() { p += by; }
  // k_left: k from the step's first to the operand's end
  __device__ __forceinline__ uint32_t bytes(int k_left) const {
    if (k_left <= 0) return 0;
    if (KM) return fixed + ((k_left < (int)kGemmStep ? k_left : (int)kGemmStep) - 1) * ld2;
    return fixed + (((uint32_t)k_left * 2 + 3) & ~3u);
  }
};

template <typename T, bool KM, int R>
__device__ __forceinline__ void zero_partial(T* lds, int k_left, int tid, int nt) {
  if constexpr (!KM) {
    for (int row = tid; row < R; row += nt)
      for (int k = k_left; k & 7; ++k) lds[row * 64 + (((k >> 3) ^ (row >> 1 & 7)) << 3) + (k & 7)] = (T)0.0f;
  }
}

// z -> out for 8 neighbouring columns from n of R rows: m, m + dm, ... below m_end. Everything that is read is asked
// for before it is needed, and the R rows' arithmetic stands side by side, as nothing else hides
// its latency. The activation is chosen once for all of them. Vectors may lie at any element.
template <typename T, int R>
__device__ __forceinline__ void finish_rows(const GemmDev& g, float (&z)[R][8], uint64_t m, uint32_t dm,
                                            uint32_t m_end, uint32_t n) {
  typedef T v8 __attribute__((ext_vector_type(8), aligned(2)));
  typedef float f8 __attribute__((ext_vector_type(8), aligned(4)));
  // A tile's results go past the caches: written back in turn they took from the operands' share of the
  // memory side cache (2048 x 768 -> 50257 from cold operands 203 us, 249 without; a chain of 4096 x 4096
  // and 11008 layers forward and backward, each reading the one before, 1 to 4% faster).
  constexpr bool kStream = R > 1;
  const T* res = static_cast<const T*>(g.res) + m * g.ldr + n;
  T* pre = static_cast<T*>(g.pre) + m * g.ldp + n;
  float* out32 = static_cast<float*>(g.out) + m * g.ldo + n;
  T* out16 = static_cast<T*>(g.out) + m * g.ldo + n;
  auto there = [&](int r) { return m + (uint64_t)r * dm < m_end; };
  v8 held[R];
  if (g.res) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (there(r)) held[r] = *reinterpret_cast<const v8*>(res + (uint64_t)r * dm * g.ldr);
  }
  if (g.bias) {
    const v8 b = *reinterpret_cast<const v8*>(static_cast<const T*>(g.bias) + n);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < 8; ++j) z[r][j] += (float)b[j];
  }
  if (g.pre) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      v8 o;
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = (T)z[r][j];
      if (!there(r)) continue;
      if constexpr (kStream) __builtin_nontemporal_store(o, reinterpret_cast<v8*>(pre + (uint64_t)r * dm * g.ldp));
      else *reinterpret_cast<v8*>(pre + (uint64_t)r * dm * g.ldp) = o;
    }
  }
  act_rt<R * 8>(&z[0][0], g.act);
  if (g.res) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < 8; ++j) z[r][j] += (float)held[r][j];
  }
  if (g.out_f32) {
    if (g.accumulate) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (there(r)) {
          const f8 o = *reinterpret_cast<const f8*>(out32 + (uint64_t)r * dm * g.ldo);
#pragma unroll
          for (int j = 0; j < 8; ++j) z[r][j] += o[j];
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      f8 o;
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = z[r][j];
      if (!there(r)) continue;
      if constexpr (kStream) __builtin_nontemporal_store(o, reinterpret_cast<f8*>(out32 + (uint64_t)r * dm * g.ldo));
      else *reinterpret_cast<f8*>(out32 + (uint64_t)r * dm * g.ldo) = o;
    }
  } else {
    if (g.accumulate) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (there(r)) {
          const v8 o = *reinterpret_cast<const v8*>(out16 + (uint64_t)r * dm * g.ldo);
#pragma unroll
          for (int j = 0; j < 8; ++j) z[r][j] += (float)o[j];
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      v8 o;
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = (T)z[r][j];
      if (!there(r)) continue;
      if constexpr (kStream) __builtin_nontemporal_store(o, reinterpret_cast<v8*>(out16 + (uint64_t)r * dm * g.ldo));
      else *reinterpret_cast<v8*>(out16 + (uint64_t)r * dm * g.ldo) = o;
    }
  }
}

// The same for one element, at the right edge.
template <typename T>
__device__ __forceinline__ void finish_one(const GemmDev& g, float z, uint64_t m, uint32_t n) {
  if (g.bias) z += (float)static_cast<const T*>(g.bias)[n];
  if (g.pre) static_cast<T*>(g.pre)[m * g.ldp + n] = (T)z;
  act_rt<1>(&z, g.act);
  if (g.res) z += (float)static_cast<const T*>(g.res)[m * g.ldr + n];
  if (g.out_f32) {
    float* out = static_cast<float*>(g.out) + m * g.ldo + n;
    *out = g.accumulate ? z + *out : z;
  } else {
    T* out = static_cast<T*>(g.out) + m * g.ldo + n;
    *out = (T)(g.accumulate ? z + (float)*out : z);
  }
}

// One row's up to 8 columns from n.
template <typename T>
__device__ __forceinline__ void finish_row(const GemmDev& g, float (&z)[1][8], uint64_t m, uint32_t n) {
  if (n + 8 <= g.n) {
    finish_rows<T, 1>(g, z, m, 1, g.m, n);
    return;
  }
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (n + j < g.n) finish_one<T>(g, z[0][j], m, n + j);
}

// Partial sums to the workspace, for the split's join.
template <int R>
__device__ __forceinline__ void keep_rows(const GemmDev& g, float (&z)[R][8], uint64_t m, uint32_t dm,
                                          uint32_t m_end, uint32_t n) {
  typedef float f8 __attribute__((ext_vector_type(8), aligned(4)));
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint64_t row = m + (uint64_t)r * dm;
    if (row >= m_end) continue;
    float* w = g.ws + ((uint64_t)blockIdx.y * g.m + row) * g.n + n;
    if (n + 8 <= g.n) {
      f8 o;
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = z[r][j];
      *reinterpret_cast<f8*>(w) = o;
    } else {
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (n + j < g.n) w[j] = z[r][j];
    }
  }
}

}  // namespace zero
