// gfx950 row kernels of the block boundaries: post norm, gate, scales and residual sum, and the next block's
// pre norm, forward and backward. Compiled once per 16-bit type (-DZERO_NORM_DT) and stream type
// (-DZERO_NORM_S32).
//
// Memory is the bound (8 to 12 bytes an element forward, 12 to 18 backward; 8192 x 4096 forward with an fp32 stream and a
// gate 75 to 78 us, 5.2 to 5.4 TB/s; backward with a 16-bit stream, a gate and two weights 91, 4.5, of which the join takes 5). A row lies in the registers of
// its waves, 8 columns (16 bytes of a 16-bit type) a lane and vector, so every array is read once.
//
// Backward: with gh = dh*w_pre, base = dy + r_pre*gh, xh and oh the normalised values and
// q = branch_scale*gate*w_post, D = base - r_pre*(m1 + xh*c1), and the post norm's own means of q*D*oh and q*D
// are sums of q*oh*base, q*oh*xh, ... that need no D: every sum of a row is formed in one reduction. Sums over
// rows stay in registers over a block's rows, are joined over the block through LDS, and over the blocks by
// k_join (zero_norm.hip), in a fixed order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "zero_norm.h"
#include "zero_rows.h"

#if !defined(ZERO_NORM_DT) || !defined(ZERO_NORM_S32)
#error "compile once per type pair: -DZERO_NORM_DT=<zero_dtype> -DZERO_NORM_S32=<0|1>"
#endif

namespace zero {
namespace norm {
namespace {

template <int DT>
struct Of;
template <>
struct Of<ZERO_F16> {
  typedef _Float16 type;
};
template <>
struct Of<ZERO_BF16> {
  typedef __bf16 type;
};

// 8 columns of a row at any element offset
template <typename T>
struct Eight {
  typedef T vec __attribute__((ext_vector_type(8), aligned(sizeof(T))));
  vec v;
  __device__ __forceinline__ float operator[](int j) const { return (float)v[j]; }
};
template <>
struct Eight<float> {
  typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
  vec v[2];
  __device__ __forceinline__ float operator[](int j) const { return v[j / 4][j % 4]; }
};

// A row's statistics, which may lie at any multiple of 4 bytes.
typedef float Stats __attribute__((ext_vector_type(4), aligned(4)));

// Columns that exist behind column c of d: 8 but at a row's end.
__device__ __forceinline__ int have_of(uint32_t d, uint32_t c) { return c + 8 <= d ? 8 : c < d ? (int)(d - c) : 0; }

template <typename T, bool PAST = false>
__device__ __forceinline__ Eight<T> load_all(const T* p) {
  typedef typename Eight<T>::vec V;
  Eight<T> r;
  if constexpr (sizeof(T) == 4) {
    if constexpr (PAST) {
      r.v[0] = __builtin_nontemporal_load(reinterpret_cast<const V*>(p));
      r.v[1] = __builtin_nontemporal_load(reinterpret_cast<const V*>(p + 4));
    } else {
      r.v[0] = *reinterpret_cast<const V*>(p);
      r.v[1] = *reinterpret_cast<const V*>(p + 4);
    }
  } else {
    if constexpr (PAST) r.v = __builtin_nontemporal_load(reinterpret_cast<const V*>(p));
    else r.v = *reinterpret_cast<const V*>(p);
  }
  return r;
}

// 8 columns of which `have` exist; the others 0.
template <typename T>
__device__ __forceinline__ Eight<T> load8(const T* p, int have) {
  if (have == 8) return load_all<T>(p);
  Eight<T> r;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const T x = j < have ? p[j] : (T)0.0f;
    if constexpr (sizeof(T) == 4) r.v[j / 4][j % 4] = x;
    else r.v[j] = x;
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, int have, const float (&x)[8], bool past) {
  Eight<T> r;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (sizeof(T) == 4) r.v[j / 4][j % 4] = x[j];
    else r.v[j] = (T)x[j];
  }
  if (have == 8) {
    typedef typename Eight<T>::vec V;
    if constexpr (sizeof(T) == 4) {
      if (past) {
        __builtin_nontemporal_store(r.v[0], reinterpret_cast<V*>(p));
        __builtin_nontemporal_store(r.v[1], reinterpret_cast<V*>(p + 4));
      } else {
        reinterpret_cast<V*>(p)[0] = r.v[0];
        *reinterpret_cast<V*>(p + 4) = r.v[1];
      }
    } else {
      if (past) __builtin_nontemporal_store(r.v, reinterpret_cast<V*>(p));
      else *reinterpret_cast<V*>(p) = r.v;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < have) p[j] = (T)x[j];
  }
}

// The sum of v over the first W lanes of each 16 (W a power of two), in all of them: one read of LDS for each lane and
// moves inside the vector unit, in place of a read for each wave.
template <int CTRL>
__device__ __forceinline__ float plus(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

__device__ __forceinline__ float few_sum(float v, uint32_t W) {
  if (W > 1) v = plus<0xb1>(v);   // lanes 1 apart
  if (W > 2) v = plus<0x4e>(v);   // 2 apart
  if (W > 4) v = plus<0x141>(v);  // the other four of eight
  if (W > 8) v = plus<0x140>(v);  // the other eight
  return v;
}

// A sum over the waves of a block that holds one row. `slot` alternates, so one barrier a sum is enough.
template <int MAXW>
__device__ __forceinline__ float row_sum(float v, float (*lds)[MAXW], int& slot) {
  v = wave_sum(v);
  const uint32_t waves = blockDim.x / 64, l = threadIdx.x % 16;
  if (waves == 1) return v;
  if (threadIdx.x % 64 == 0) lds[slot][threadIdx.x / 64] = v;
  __syncthreads();
  v = l < waves ? lds[slot][l] : 0.0f;
  slot ^= 1;
  return few_sum(v, 16);
}

// Mean and 1/deviation of a row of 8*NV columns a lane.
template <int NV, int MAXW>
__device__ __forceinline__ void moments(const float (&v)[NV][8], const int (&have)[NV], int kind, float inv_n, float eps,
                                        float (*lds)[MAXW], int& slot, float& mean, float& rstd) {
  mean = 0.0f;
  if (kind == ZERO_NORM_LAYER) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[i][j];  // 0 behind the row's end
    mean = row_sum<MAXW>(s, lds, slot) * inv_n;
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float c = j < have[i] ? v[i][j] - mean : 0.0f;
      s += c * c;
    }
  rstd = 1.0f / sqrtf(row_sum<MAXW>(s, lds, slot) * inv_n + eps);
}

// One block a row. WHOLE: the columns are a multiple of 8; then a lane behind the row's end reads the row's start, which
// does not count, and every load goes out without a condition before the first sum waits for one.
template <typename T, typename S, int NV, bool WHOLE>
__global__ __launch_bounds__(1024) void k_forward(ForwardArgs a, uint32_t gate_step, bool past) {
  __shared__ float lds[2][16];
  const zero_norm_block& b = a.b;
  const uint32_t d = (uint32_t)b.features;
  const uint64_t row = (uint64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= b.rows) return;
  const float inv_n = 1.0f / (float)d;
  int slot = 0, have[NV];
  uint32_t col[NV];
  float v[NV][8];
  float mean = 0.0f, rstd = 1.0f, post_mean = 0.0f, post_rstd = 1.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    col[i] = (i * blockDim.x + threadIdx.x) * 8;
    have[i] = have_of(d, col[i]);
  }
  auto load = [&](auto* p, int i) {
    typedef typename std::remove_const<typename std::remove_pointer<decltype(p)>::type>::type E;
    if constexpr (WHOLE) return load_all<E>(p + (have[i] ? col[i] : 0u));
    else return load8<E>(p + (have[i] ? col[i] : 0u), have[i]);
  };
  const T *post_w = static_cast<const T*>(b.post_weight), *post_b = static_cast<const T*>(b.post_bias);
  const T *pre_w = static_cast<const T*>(b.pre_weight), *pre_b = static_cast<const T*>(b.pre_bias);
  const T* gate = b.gate ? static_cast<const T*>(b.gate) + (uint64_t)((uint32_t)row / gate_step) * b.ld_gate : nullptr;
  Eight<S> xs[NV];
  Eight<T> os[NV], w[NV], c[NV], g[NV], u[NV], e[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (b.branch) os[i] = load(static_cast<const T*>(b.branch) + row * b.ld_branch, i);
    xs[i] = load(static_cast<const S*>(a.x) + row * a.ldx, i);
  }
  // the parameters with them, but of two vectors where they are used: 4096 x 12288 112 us, and 133 with all held
  auto post_parameters = [&](int i) {
    if (post_w) w[i] = load(post_w, i);
    if (post_b) c[i] = load(post_b, i);
    if (gate) g[i] = load(gate, i);
  };
  auto pre_parameters = [&](int i) {
    if (pre_w) u[i] = load(pre_w, i);
    if (pre_b) e[i] = load(pre_b, i);
  };
  if constexpr (NV == 1) post_parameters(0), pre_parameters(0);
  if (b.branch) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = j < have[i] ? os[i][j] : 0.0f;
    if (b.post != ZERO_NORM_NONE) moments<NV, 16>(v, have, b.post, inv_n, b.eps, lds, slot, post_mean, post_rstd);
    S* y = static_cast<S*>(a.y) + row * a.ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (NV > 1) post_parameters(i);
      float out[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float t = (v[i][j] - post_mean) * post_rstd;
        if (post_w) t = t * w[i][j];
        if (post_b) t = t + c[i][j];
        if (gate) t = t * g[i][j];
        out[j] = b.residual_scale * xs[i][j] + b.branch_scale * t;
        v[i][j] = j < have[i] ? (float)(S)out[j] : 0.0f;
      }
      store8<S>(y + col[i], have[i], out, past);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = j < have[i] ? xs[i][j] : 0.0f;
  }
  if (b.pre != ZERO_NORM_NONE) {
    moments<NV, 16>(v, have, b.pre, inv_n, b.eps, lds, slot, mean, rstd);
    T* h = static_cast<T*>(a.h) + row * a.ldh;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (NV > 1) pre_parameters(i);
      float out[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        out[j] = (v[i][j] - mean) * rstd;
        if (pre_w) out[j] = out[j] * u[i][j];
        if (pre_b) out[j] = out[j] + e[i][j];
      }
      store8<T>(h + col[i], have[i], out, false);
    }
  }
  if (a.stats && threadIdx.x == 0)
    *reinterpret_cast<Stats*>(a.stats + 4 * row) = Stats{post_mean, post_rstd, mean, rstd};
}

// Keeps what is computed from x from being formed earlier and held in registers.
template <typename T>
__device__ __forceinline__ void again(Eight<T>& x) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  u4 v[sizeof(Eight<T>) / 16];
  __builtin_memcpy(v, &x, sizeof(x));
#pragma unroll
  for (auto& q : v) asm volatile("" : "+v"(q));
  __builtin_memcpy(&x, v, sizeof(x));
}

// What of a row's arrays a lane holds.
template <typename T, typename S, int GATE>
struct Held {
  Eight<S> y, dy;
  Eight<T> dh, o, g;
};

// LN: a mean is taken off in one of the norms, or a bias has a gradient. GATE: as gate_mode. WHOLE: the columns are
// a multiple of 8, so every lane's are all there or none are.
//
// The sums over rows are four at most: of dh*xh and dh, and of E*oh and E with E = D, times the row's gate where
// every row has its own. Where rows share a gate, the gradients of that gate and of the post norm's parameters
// are E*oh's and E's sums times the one or the others.
// NT threads a block. SUMS: forms the sums over rows; else it leaves each row's m1 and c1 for k_columns.
template <typename T, typename S, int NV, bool LN, int GATE, bool WHOLE, int NT, bool SUMS>
__global__ __launch_bounds__(NT) void k_backward(BackwardArgs a) {
  constexpr int kWaves = NT / 64;
  constexpr int kOut = LN ? 8 : 4;  // sums of a row
  __shared__ __attribute__((aligned(16))) float lds[2][kWaves][kOut];
  __shared__ __attribute__((aligned(16))) float cols[LN ? 2 : 1][SUMS ? NT * 8 : 4];
  const zero_norm_block& b = a.b;
  const uint32_t d = (uint32_t)b.features, W = a.plan.waves, groups = kWaves / W;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);  // the same in its lanes: a row's addresses are scalars
  const uint32_t lanes = W * 64, group = wave / W, lane = threadIdx.x % lanes;
  const float inv_n = 1.0f / (float)d;
  const bool pre = b.pre != ZERO_NORM_NONE, post = b.post != ZERO_NORM_NONE, has_o = b.branch != nullptr;
  const float scale = has_o ? b.residual_scale : 1.0f;
  uint32_t col[NV];
  int have[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    col[i] = (i * lanes + lane) * 8;
    have[i] = have_of(d, col[i]);
  }
  // a parameter's columns: 1 without it, and 0 behind the row's end, so that nothing there counts
  auto weight = [&](const void* p, int i) {
    const T* w = static_cast<const T*>(p);
    Eight<T> r = load8<T>(w ? w + (have[i] ? col[i] : 0u) : nullptr, w ? have[i] : 0);
    if (!w) {
#pragma unroll
      for (int j = 0; j < 8; ++j) r.v[j] = j < have[i] ? (T)1.0f : (T)0.0f;
    }
    return r;
  };
  Eight<T> wpre[NV], wpost[NV], gate[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) wpre[i] = weight(b.pre_weight, i), wpost[i] = weight(b.post_weight, i);
  float s_xh[NV][8] = {}, s_oh[NV][8] = {};
  float s_dh[LN ? NV : 1][8] = {}, s_e[LN ? NV : 1][8] = {};

  // The block's sums of one or two arrays, group by group, in column order; `to` takes column c's.
  auto joined = [&](float (&s)[NV][8], float (*s2)[8], auto to) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        const uint32_t at = (group * lanes + lane) * 8 + j;
        *reinterpret_cast<float4*>(cols[0] + at) = make_float4(s[i][j], s[i][j + 1], s[i][j + 2], s[i][j + 3]);
        if (s2) *reinterpret_cast<float4*>(cols[LN ? 1 : 0] + at) = make_float4(s2[i][j], s2[i][j + 1], s2[i][j + 2], s2[i][j + 3]);
      }
      __syncthreads();
      for (uint32_t c = threadIdx.x; c < lanes * 8; c += NT) {
        float t = 0.0f, t2 = 0.0f;
        for (uint32_t g = 0; g < groups; ++g) {
          t += cols[0][g * lanes * 8 + c];
          if (s2) t2 += cols[LN ? 1 : 0][g * lanes * 8 + c];
        }
        const uint32_t at = i * lanes * 8 + c;
        if (at < d) to(at, t, t2);
      }
    }
  };
  float* const part_pw = a.part[kPostW] ? a.part[kPostW] + (uint64_t)blockIdx.x * d : nullptr;
  float* const part_pb = a.part[kPostB] ? a.part[kPostB] + (uint64_t)blockIdx.x * d : nullptr;
  float* const part_g = a.part[kGate] ? a.part[kGate] + (uint64_t)blockIdx.x * d : nullptr;

  const uint64_t part = a.plan.chunks > 1 ? blockIdx.x % a.plan.chunks : 0;
  const uint64_t seg0 = a.plan.chunks > 1 ? blockIdx.x / a.plan.chunks : (uint64_t)blockIdx.x * a.plan.segs;
  const uint64_t seg1 = a.plan.chunks > 1 ? seg0 + 1 : seg0 + a.plan.segs < a.plan.segments ? seg0 + a.plan.segs : a.plan.segments;
  int slot = 0;
  for (uint64_t seg = seg0; seg < seg1; ++seg) {
    const uint64_t first = seg * a.plan.per + part * a.plan.chunk;
    uint64_t end = part + 1 == a.plan.chunks ? (seg + 1) * a.plan.per : first + a.plan.chunk;
    if (end > (seg + 1) * a.plan.per) end = (seg + 1) * a.plan.per;
    if (end > b.rows) end = b.rows;
    const T* seg_gate = GATE == 1 ? static_cast<const T*>(b.gate) + seg * b.ld_gate : nullptr;
    if constexpr (GATE == 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i) gate[i] = weight(seg_gate, i);
    }
    // The parameters' columns of vector i: held, but what is formed of them is formed anew in each pass.
    auto parameters = [&](int i) {
      again(wpre[i]), again(wpost[i]);
      if constexpr (GATE == 1) again(gate[i]);
    };
    // A vector of a row's arrays. Rows behind the end, and lanes behind the row's, read what is there: nothing of it
    // counts (their weights are 0), and loads without conditions go out together, a row ahead of their use.
    auto load = [&](uint64_t row, int i) {
      Held<T, S, GATE> r{};
      row = row < end ? row : end - 1;
      const uint32_t c = have[i] ? col[i] : 0u;
      auto eight = [&](auto* p) {
        typedef typename std::remove_const<typename std::remove_pointer<decltype(p)>::type>::type E;
        // past the caches what is not read again
        if constexpr (WHOLE) return load_all<E, SUMS>(p);
        else return load8<E>(p, have[i]);
      };
      if (a.dy) r.dy = eight(static_cast<const S*>(a.dy) + row * a.lddy + c);
      if (pre) r.dh = eight(static_cast<const T*>(a.dh) + row * a.lddh + c);
      if (pre) r.y = eight(static_cast<const S*>(a.y) + row * a.ldy + c);
      if (has_o) r.o = eight(static_cast<const T*>(b.branch) + row * b.ld_branch + c);
      if constexpr (GATE == 2) r.g = eight(static_cast<const T*>(b.gate) + row * b.ld_gate + c);
      return r;
    };
    // the next row's arrays are asked for before this one's are used, where the registers hold both
    Held<T, S, GATE> ahead[NV];
    Stats st_ahead;
    auto look = [&](uint64_t row) {
#pragma unroll
      for (int i = 0; i < NV; ++i) ahead[i] = load(row, i);
      st_ahead = *reinterpret_cast<const Stats*>(a.stats + 4 * (row < end ? row : end - 1));
    };
    if (SUMS && first < end) look(first + group);
    for (uint64_t base_row = first; base_row < end; base_row += groups) {
      const uint64_t row = base_row + group;
      const bool on = row < end;
      if (!SUMS) look(row);
      Held<T, S, GATE> held[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) held[i] = ahead[i];
      const Stats st = st_ahead;
      if (SUMS && base_row + groups < end) look(row + groups);
      const float mo = post ? st.x : 0.0f, ro = post ? st.y : 1.0f;
      const float mp = pre ? st.z : 0.0f, rp = pre ? st.w : 0.0f;
      float sum[kOut] = {};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        parameters(i);
        const Held<T, S, GATE>& r = held[i];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xh = (r.y[j] - mp) * rp, gh = r.dh[j] * wpre[i][j];
          const float base = r.dy[j] + rp * gh, oh = (r.o[j] - mo) * ro;
          float q = b.branch_scale * wpost[i][j];
          if constexpr (GATE == 1) q *= gate[i][j];
          if constexpr (GATE == 2) q *= r.g[j];
          const float p = q * oh;
          sum[0] += gh * xh;
          sum[1] += p * base;
          sum[2] += p * xh;
          if constexpr (LN) {
            sum[3] += gh;
            sum[4] += q * base;
            sum[5] += q * xh;
            sum[6] += q;
            sum[7] += p;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < (LN ? 8 : 3); ++k) sum[k] = wave_sum(sum[k]);
      if (W > 1) {
        if (threadIdx.x % 64 == 0) {
#pragma unroll
          for (int k = 0; k < kOut; k += 4)
            *reinterpret_cast<float4*>(&lds[slot][wave][k]) = make_float4(sum[k], sum[k + 1], sum[k + 2], sum[k + 3]);
        }
        __syncthreads();
        // a read for each wave up to 8; moves between lanes are the longer chain there (8192 x 4096 with two layer
        // norms 113 us and 121 when that was chosen, but 4096 x 5120 without 73 and 65)
        if (NT > 512 && W > 8) {
#pragma unroll
          for (int k = 0; k < kOut; k += 4) {
            const float4 o = *reinterpret_cast<const float4*>(&lds[slot][group * W + threadIdx.x % W][k]);
            sum[k] = few_sum(o.x, W), sum[k + 1] = few_sum(o.y, W), sum[k + 2] = few_sum(o.z, W);
            sum[k + 3] = few_sum(o.w, W);
          }
        } else {
#pragma unroll
          for (int k = 0; k < kOut; ++k) sum[k] = 0.0f;
          for (uint32_t w = 0; w < W; ++w)
#pragma unroll
            for (int k = 0; k < kOut; k += 4) {
              const float4 o = *reinterpret_cast<const float4*>(&lds[slot][group * W + w][k]);
              sum[k] += o.x, sum[k + 1] += o.y, sum[k + 2] += o.z, sum[k + 3] += o.w;
            }
        }
        slot ^= 1;
      }
      const float c1 = sum[0] * inv_n, m1 = LN && b.pre == ZERO_NORM_LAYER ? sum[3] * inv_n : 0.0f;
      float c2 = 0.0f, m2 = 0.0f;
      if (post) c2 = (sum[1] - rp * ((LN ? m1 * sum[LN ? 7 : 0] : 0.0f) + c1 * sum[2])) * inv_n;
      if (LN && b.post == ZERO_NORM_LAYER) m2 = (sum[LN ? 4 : 0] - rp * (m1 * sum[LN ? 6 : 0] + c1 * sum[LN ? 5 : 0])) * inv_n;
      if (!on) continue;
      if (!SUMS && a.coef && lane == 0) *reinterpret_cast<float2*>(a.coef + 2 * row) = make_float2(m1, c1);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        parameters(i);
        Held<T, S, GATE>& r = held[i];
        again(r.y), again(r.dy), again(r.dh), again(r.o);
        if constexpr (GATE == 2) again(r.g);
        float dx[8], db[8], dg[8], oh[8];
        Eight<T> bias{};
        if (GATE == 2 && a.dgate && b.post_bias) bias = load8<T>(static_cast<const T*>(b.post_bias) + (have[i] ? col[i] : 0u), have[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float dh = r.dh[j];
          const float xh = (r.y[j] - mp) * rp;
          const float D = r.dy[j] + rp * (dh * wpre[i][j]) - rp * (m1 + xh * c1);
          oh[j] = (r.o[j] - mo) * ro;
          float e = D;
          if constexpr (GATE == 2) {
            dg[j] = b.branch_scale * D * (oh[j] * wpost[i][j] + bias[j]);
            e *= r.g[j];
          }
          float u = b.branch_scale * e * wpost[i][j];
          if constexpr (GATE == 1) u *= gate[i][j];
          dx[j] = scale * D;
          db[j] = u;
          if constexpr (SUMS) {
            s_xh[i][j] += dh * xh;
            s_oh[i][j] += e * oh[j];
          }
          if constexpr (SUMS && LN) {
            s_dh[i][j] += dh;
            s_e[i][j] += e;
          }
        }
        // Without a norm the branch has no part in its own gradient, an inf of it neither. The place of this pass is the one that
        // suits the registers (8192 x 4096 with two layer norms 104 us before dx's store, 116 behind it; 4096 x 5120 in blocks of 1024
        // threads 70 and 67).
        auto normed = [&]() {
          if (!post) return;
#pragma unroll
          for (int j = 0; j < 8; ++j) db[j] = ro * (db[j] - m2 - oh[j] * c2);
        };
        if (NT == 512) normed();
        if (a.dx) store8<S>(static_cast<S*>(a.dx) + row * a.lddx + col[i], have[i], dx, false);
        if (NT != 512) normed();
        if (a.dbranch) store8<T>(static_cast<T*>(a.dbranch) + row * a.lddbranch + col[i], have[i], db, false);
        if (GATE == 2 && a.dgate) {
          const uint64_t at = row * a.lddgate + col[i];
          if (a.grad_f32) {
            float* o = static_cast<float*>(a.dgate) + at;
            if (a.accumulate) {
              const Eight<float> was = load8<float>(o, have[i]);
#pragma unroll
              for (int j = 0; j < 8; ++j) dg[j] += was[j];
            }
            store8<float>(o, have[i], dg, false);
          } else {
            T* o = static_cast<T*>(a.dgate) + at;
            if (a.accumulate) {
              const Eight<T> was = load8<T>(o, have[i]);
#pragma unroll
              for (int j = 0; j < 8; ++j) dg[j] += was[j];
            }
            store8<T>(o, have[i], dg, false);
          }
        }
      }
    }
    if constexpr (SUMS && GATE == 1) {
      // the segment's: its gate's gradient or part of it, and its share of the post norm's
      const bool more = seg > seg0;
      joined(s_oh, LN ? s_e : nullptr, [&](uint32_t c, float t, float t2) {
        const float w = b.post_weight ? (float)static_cast<const T*>(b.post_weight)[c] : 1.0f;
        const float bias = b.post_bias ? (float)static_cast<const T*>(b.post_bias)[c] : 0.0f;
        const float g = b.branch_scale * (float)static_cast<const T*>(b.gate)[seg * b.ld_gate + c];
        const float dg = b.branch_scale * (w * t + bias * t2);
        if (part_pw) part_pw[c] = (more ? part_pw[c] : 0.0f) + g * t;
        if (part_pb) part_pb[c] = (more ? part_pb[c] : 0.0f) + g * t2;
        if (part_g) {
          part_g[c] = dg;
        } else if (a.dgate) {
          const uint64_t at = seg * a.lddgate + c;
          if (a.grad_f32) {
            float* o = static_cast<float*>(a.dgate) + at;
            *o = a.accumulate ? *o + dg : dg;
          } else {
            T* o = static_cast<T*>(a.dgate) + at;
            *o = (T)(a.accumulate ? (float)*o + dg : dg);
          }
        }
      });
      if (seg + 1 < seg1) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            s_oh[i][j] = 0.0f;
            if constexpr (LN) s_e[i][j] = 0.0f;
          }
      }
    }
  }
  if constexpr (!SUMS) return;
  if (GATE != 1 && (part_pw || part_pb))
    joined(s_oh, LN ? s_e : nullptr, [&](uint32_t c, float t, float t2) {
      if (part_pw) part_pw[c] = b.branch_scale * t;
      if (part_pb) part_pb[c] = b.branch_scale * t2;
    });
  if (a.part[kPreW] || a.part[kPreB])
    joined(s_xh, LN ? s_dh : nullptr, [&](uint32_t c, float t, float t2) {
      const uint64_t at = (uint64_t)blockIdx.x * d + c;
      if (a.part[kPreW]) a.part[kPreW][at] = t;
      if (a.part[kPreB]) a.part[kPreB][at] = t2;
    });
}

// The sums over rows where a row takes so many registers that k_backward cannot hold them beside it: each thread
// walks its 8 columns down the block's rows, with each row's m1 and c1 from k_backward, and reads the arrays
// again (4096 x 12288 with an fp32 stream and a layer norm 278 us; held in one kernel, and so partly in
// memory, 735).
constexpr int kColumnThreads = 256;

template <typename T, typename S, int GATE>
__global__ __launch_bounds__(kColumnThreads) void k_columns(BackwardArgs a) {
  const zero_norm_block& b = a.b;
  const uint32_t d = (uint32_t)b.features, c = (blockIdx.y * kColumnThreads + threadIdx.x) * 8;
  const int have = have_of(d, c);
  if (!have) return;
  const bool pre = b.pre != ZERO_NORM_NONE, post = b.post != ZERO_NORM_NONE;
  const bool sum_pre = a.part[kPreW] || a.part[kPreB];
  const bool sum_post = a.part[kPostW] || a.part[kPostB] || (GATE == 1 && a.dgate);
  const Eight<T> wpre = load8<T>(static_cast<const T*>(b.pre_weight) + (b.pre_weight ? c : 0u), b.pre_weight ? have : 0);
  float s_xh[8] = {}, s_dh[8] = {}, p_w[8] = {}, p_b[8] = {};
  const uint64_t part = a.plan.chunks > 1 ? blockIdx.x % a.plan.chunks : 0;
  const uint64_t seg0 = a.plan.chunks > 1 ? blockIdx.x / a.plan.chunks : (uint64_t)blockIdx.x * a.plan.segs;
  const uint64_t seg1 = a.plan.chunks > 1 ? seg0 + 1 : seg0 + a.plan.segs < a.plan.segments ? seg0 + a.plan.segs : a.plan.segments;
  for (uint64_t seg = seg0; seg < seg1; ++seg) {
    const uint64_t first = seg * a.plan.per + part * a.plan.chunk;
    uint64_t end = part + 1 == a.plan.chunks ? (seg + 1) * a.plan.per : first + a.plan.chunk;
    if (end > (seg + 1) * a.plan.per) end = (seg + 1) * a.plan.per;
    if (end > b.rows) end = b.rows;
    float s_oh[8] = {}, s_e[8] = {};
#pragma unroll 2
    for (uint64_t row = first; row < end; ++row) {
      const Stats st = *reinterpret_cast<const Stats*>(a.stats + 4 * row);
      const float mo = post ? st.x : 0.0f, ro = post ? st.y : 1.0f;
      const float mp = pre ? st.z : 0.0f, rp = pre ? st.w : 0.0f;
      Eight<S> y{}, dy{};
      Eight<T> dh{}, o{}, g{};
      if (pre) dh = load8<T>(static_cast<const T*>(a.dh) + row * a.lddh + c, have);
      if (pre) y = load8<S>(static_cast<const S*>(a.y) + row * a.ldy + c, have);
      float2 k = make_float2(0.0f, 0.0f);
      if (sum_post) {
        k = *reinterpret_cast<const float2*>(a.coef + 2 * row);
        if (a.dy) dy = load8<S>(static_cast<const S*>(a.dy) + row * a.lddy + c, have);
        o = load8<T>(static_cast<const T*>(b.branch) + row * b.ld_branch + c, have);
        if constexpr (GATE == 2) g = load8<T>(static_cast<const T*>(b.gate) + row * b.ld_gate + c, have);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = (y[j] - mp) * rp;
        s_xh[j] += dh[j] * xh;
        s_dh[j] += dh[j];
        if (sum_post) {
          const float w = b.pre_weight ? wpre[j] : 1.0f;
          float e = dy[j] + rp * (dh[j] * w) - rp * (k.x + xh * k.y);
          if constexpr (GATE == 2) e *= g[j];
          s_oh[j] += e * ((o[j] - mo) * ro);
          s_e[j] += e;
        }
      }
    }
    if (!sum_post) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= have) continue;
      float g = b.branch_scale;
      if constexpr (GATE == 1) {
        const float w = b.post_weight ? (float)static_cast<const T*>(b.post_weight)[c + j] : 1.0f;
        const float bias = b.post_bias ? (float)static_cast<const T*>(b.post_bias)[c + j] : 0.0f;
        const float dg = b.branch_scale * (w * s_oh[j] + bias * s_e[j]);
        g *= (float)static_cast<const T*>(b.gate)[seg * b.ld_gate + c + j];
        const uint64_t at = seg * a.lddgate + c + j;
        if (a.part[kGate]) {
          a.part[kGate][(uint64_t)blockIdx.x * d + c + j] = dg;
        } else if (a.dgate && a.grad_f32) {
          float* out = static_cast<float*>(a.dgate) + at;
          *out = a.accumulate ? *out + dg : dg;
        } else if (a.dgate) {
          T* out = static_cast<T*>(a.dgate) + at;
          *out = (T)(a.accumulate ? (float)*out + dg : dg);
        }
      }
      p_w[j] += g * s_oh[j];
      p_b[j] += g * s_e[j];
    }
  }
  auto leave = [&](int k, const float (&s)[8]) {
    if (!a.part[k]) return;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < have) a.part[k][(uint64_t)blockIdx.x * d + c + j] = s[j];
  };
  leave(kPostW, p_w), leave(kPostB, p_b), leave(kPreW, s_xh), leave(kPreB, s_dh);
}

template <typename T, typename S, int NV, bool LN, int GATE, int NT, bool SUMS>
hipError_t rows_of(const BackwardArgs& a) {
  const dim3 grid((unsigned)a.plan.blocks), block(NT);
  if (a.b.features % 8 == 0) k_backward<T, S, NV, LN, GATE, true, NT, SUMS><<<grid, block, 0, a.stream>>>(a);
  else k_backward<T, S, NV, LN, GATE, false, NT, SUMS><<<grid, block, 0, a.stream>>>(a);
  return hipGetLastError();
}

template <typename T, typename S, bool LN, int GATE>
hipError_t backward_of(const BackwardArgs& a) {
  // as plan_of chose the threads and the vectors
  if (a.plan.apart) {
    const bool post = a.part[kPostW] || a.part[kPostB] || (GATE == 1 && a.dgate);
    const bool sums = post || a.part[kPreW] || a.part[kPreB];
    // dx over dy: the sums read dy first, after a pass that leaves the rows' m1 and c1 alone
    const bool over = post && a.dx && a.dx == a.dy;
    BackwardArgs first = a, last = a;
    if (over) first.dx = first.dbranch = nullptr, first.dgate = GATE == 1 ? first.dgate : nullptr;
    hipError_t e = rows_of<T, S, 2, LN, GATE, 1024, false>(first);
    if (e != hipSuccess || !sums) return e;
    const dim3 grid((unsigned)a.plan.blocks, (unsigned)((a.b.features + kColumnThreads * 8 - 1) / (kColumnThreads * 8)));
    k_columns<T, S, GATE><<<grid, dim3(kColumnThreads), 0, a.stream>>>(a);
    e = hipGetLastError();
    last.coef = nullptr;
    return e == hipSuccess && over ? rows_of<T, S, 2, LN, GATE, 1024, false>(last) : e;
  }
  if constexpr (!LN && GATE != 2) return rows_of<T, S, 1, LN, GATE, 1024, true>(a);
  else return a.plan.vecs == 1 ? rows_of<T, S, 1, LN, GATE, 512, true>(a) : rows_of<T, S, 2, LN, GATE, 512, true>(a);
}

}  // namespace

template <>
hipError_t launch_forward<ZERO_NORM_DT, ZERO_NORM_S32 != 0>(const ForwardArgs& a) {
  typedef Of<ZERO_NORM_DT>::type T;
  typedef std::conditional<ZERO_NORM_S32 != 0, float, T>::type S;
  const uint64_t vecs = (a.b.features + 7) / 8;
  const uint64_t wide = a.b.rows < (1u << 20) ? a.b.rows : (1u << 20);
  const dim3 grid((unsigned)wide, (unsigned)((a.b.rows + wide - 1) / wide));
  const uint32_t step = a.b.gate ? (uint32_t)(a.b.gate_rows < a.b.rows ? a.b.gate_rows : a.b.rows) : 1u;
  const bool past = a.b.rows * a.b.features * sizeof(S) >= (128ull << 20);
  const bool whole = a.b.features % 8 == 0;
  if (vecs <= 1024) {
    const dim3 block((unsigned)((vecs + 63) / 64 * 64));
    if (whole) k_forward<T, S, 1, true><<<grid, block, 0, a.stream>>>(a, step, past);
    else k_forward<T, S, 1, false><<<grid, block, 0, a.stream>>>(a, step, past);
  } else {
    const dim3 block((unsigned)(((vecs + 1) / 2 + 63) / 64 * 64));
    if (whole) k_forward<T, S, 2, true><<<grid, block, 0, a.stream>>>(a, step, past);
    else k_forward<T, S, 2, false><<<grid, block, 0, a.stream>>>(a, step, past);
  }
  return hipGetLastError();
}

template <>
hipError_t launch_backward<ZERO_NORM_DT, ZERO_NORM_S32 != 0>(const BackwardArgs& a) {
  typedef Of<ZERO_NORM_DT>::type T;
  typedef std::conditional<ZERO_NORM_S32 != 0, float, T>::type S;
  if (a.wide) {
    if (a.gate_mode == 0) return backward_of<T, S, true, 0>(a);
    return a.gate_mode == 1 ? backward_of<T, S, true, 1>(a) : backward_of<T, S, true, 2>(a);
  }
  if (a.gate_mode == 0) return backward_of<T, S, false, 0>(a);
  return a.gate_mode == 1 ? backward_of<T, S, false, 1>(a) : backward_of<T, S, false, 2>(a);
}

}  // namespace norm
}  // namespace zero
