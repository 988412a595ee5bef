// gfx950 row kernels of the block boundaries: post norm, gate, scales and residual sum, and the next block's
// pre norm, forward and backward. Compiled once per 16-bit type (-DZERO_NORM_DT) and stream type
// (-DZERO_NORM_S32).
//
// Memory is the bound (8 to 16 bytes an element forward, 12 to 20 backward). A row lies in the registers of
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

// Columns that exist behind column c of d: 8 but at a row's end.
__device__ __forceinline__ int have_of(uint32_t d, uint32_t c) { return c + 8 <= d ? 8 : c < d ? (int)(d - c) : 0; }

template <typename T>
__device__ __forceinline__ Eight<T> load8(const T* p, int have, float fill = 0.0f) {
  Eight<T> r;
  if (have == 8) {
    if constexpr (sizeof(T) == 4) {
      r.v[0] = *reinterpret_cast<const typename Eight<T>::vec*>(p);
      r.v[1] = *reinterpret_cast<const typename Eight<T>::vec*>(p + 4);
    } else {
      r.v = *reinterpret_cast<const typename Eight<T>::vec*>(p);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const T x = j < have ? p[j] : (T)fill;
      if constexpr (sizeof(T) == 4) r.v[j / 4][j % 4] = x;
      else r.v[j] = x;
    }
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

// A sum over the waves of a block that holds one row. `slot` alternates, so one barrier a sum is enough.
template <int MAXW>
__device__ __forceinline__ float row_sum(float v, float (*lds)[MAXW], int& slot) {
  v = wave_sum(v);
  const int waves = blockDim.x / 64;
  if (waves == 1) return v;
  if (threadIdx.x % 64 == 0) lds[slot][threadIdx.x / 64] = v;
  __syncthreads();
  v = 0.0f;
  for (int i = 0; i < waves; ++i) v += lds[slot][i];
  slot ^= 1;
  return v;
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

// One block a row.
template <typename T, typename S, int NV>
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
  const S* x = static_cast<const S*>(a.x) + row * a.ldx;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    col[i] = (i * blockDim.x + threadIdx.x) * 8;
    have[i] = have_of(d, col[i]);
  }
  Eight<S> xs[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) xs[i] = load8<S>(x + col[i], have[i]);
  if (b.branch) {
    const T* o = static_cast<const T*>(b.branch) + row * b.ld_branch;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Eight<T> e = load8<T>(o + col[i], have[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = e[j];
    }
    if (b.post != ZERO_NORM_NONE) {
      moments<NV, 16>(v, have, b.post, inv_n, b.eps, lds, slot, post_mean, post_rstd);
    }
    S* y = static_cast<S*>(a.y) + row * a.ldy;
    const T* gate = b.gate ? static_cast<const T*>(b.gate) + (uint64_t)((uint32_t)row / gate_step) * b.ld_gate : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Eight<T> w = b.post_weight ? load8<T>(static_cast<const T*>(b.post_weight) + col[i], have[i]) : Eight<T>{};
      const Eight<T> c = b.post_bias ? load8<T>(static_cast<const T*>(b.post_bias) + col[i], have[i]) : Eight<T>{};
      const Eight<T> g = gate ? load8<T>(gate + col[i], have[i]) : Eight<T>{};
      float out[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float t = (v[i][j] - post_mean) * post_rstd;
        if (b.post_weight) t = t * w[j];
        if (b.post_bias) t = t + c[j];
        if (gate) t = t * g[j];
        out[j] = b.residual_scale * xs[i][j] + b.branch_scale * t;
        v[i][j] = j < have[i] ? (float)(S)out[j] : 0.0f;
      }
      store8<S>(y + col[i], have[i], out, past);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = xs[i][j];
  }
  if (b.pre != ZERO_NORM_NONE) {
    moments<NV, 16>(v, have, b.pre, inv_n, b.eps, lds, slot, mean, rstd);
    T* h = static_cast<T*>(a.h) + row * a.ldh;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Eight<T> w = b.pre_weight ? load8<T>(static_cast<const T*>(b.pre_weight) + col[i], have[i]) : Eight<T>{};
      const Eight<T> c = b.pre_bias ? load8<T>(static_cast<const T*>(b.pre_bias) + col[i], have[i]) : Eight<T>{};
      float out[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        out[j] = (v[i][j] - mean) * rstd;
        if (b.pre_weight) out[j] = out[j] * w[j];
        if (b.pre_bias) out[j] = out[j] + c[j];
      }
      store8<T>(h + col[i], have[i], out, false);
    }
  }
  if (a.stats && threadIdx.x == 0)
    *reinterpret_cast<float4*>(a.stats + 4 * row) = make_float4(post_mean, post_rstd, mean, rstd);
}

// What of a row's arrays a lane holds.
template <typename T, typename S, int NV, int GATE>
struct Held {
  Eight<S> y[NV], dy[NV];
  Eight<T> dh[NV], o[NV], g[GATE == 2 ? NV : 1];
  float4 st;
};

// LN: a mean is taken off in one of the norms. GATE: as gate_mode.
template <typename T, typename S, int NV, bool LN, int GATE>
__global__ __launch_bounds__(kBackThreads) void k_backward(BackwardArgs a) {
  constexpr int kWaves = kBackThreads / 64;
  constexpr int kOut = LN ? 8 : 4;  // sums of a row
  __shared__ __attribute__((aligned(16))) float lds[2][kWaves][kOut];
  __shared__ __attribute__((aligned(16))) float cols[kBackThreads * 8];
  const zero_norm_block& b = a.b;
  const uint32_t d = (uint32_t)b.features, W = a.plan.waves, groups = kWaves / W;
  const uint32_t lanes = W * 64, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
  const int wave = threadIdx.x / 64;
  const float inv_n = 1.0f / (float)d;
  const bool pre = b.pre != ZERO_NORM_NONE, post = b.post != ZERO_NORM_NONE, has_o = b.branch != nullptr;
  const float scale = has_o ? b.residual_scale : 1.0f;
  uint32_t col[NV];
  int have[NV];
  Eight<T> wpre[NV], wpost[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    col[i] = (i * lanes + lane) * 8;
    have[i] = have_of(d, col[i]);
    // 1 without a weight; 0 behind the row's end, so that nothing there counts
    const T* w = static_cast<const T*>(b.pre_weight);
    wpre[i] = load8<T>(w ? w + col[i] : nullptr, w ? have[i] : 0, 0.0f);
    const T* u = static_cast<const T*>(b.post_weight);
    wpost[i] = load8<T>(u ? u + col[i] : nullptr, u ? have[i] : 0, 0.0f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!w && j < have[i]) wpre[i].v[j] = (T)1.0f;
      if (!u && j < have[i]) wpost[i].v[j] = (T)1.0f;
    }
  }
  float s_post_w[NV][8] = {}, s_pre_w[NV][8] = {}, s_gate[NV][8] = {};
  float s_post_b[LN ? NV : 1][8] = {}, s_pre_b[LN ? NV : 1][8] = {};

  // The block's sums of one array, group by group, in column order; `to` takes column c's sum.
  auto joined = [&](float (&s)[NV][8], auto to) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; j += 4)
        *reinterpret_cast<float4*>(cols + (group * lanes + lane) * 8 + j) = make_float4(s[i][j], s[i][j + 1], s[i][j + 2], s[i][j + 3]);
      __syncthreads();
      for (uint32_t c = threadIdx.x; c < lanes * 8; c += kBackThreads) {
        float t = 0.0f;
        for (uint32_t g = 0; g < groups; ++g) t += cols[g * lanes * 8 + c];
        const uint32_t at = i * lanes * 8 + c;
        if (at < d) to(at, t);
      }
    }
  };

  const uint64_t part = a.plan.chunks > 1 ? blockIdx.x % a.plan.chunks : 0;
  const uint64_t seg0 = a.plan.chunks > 1 ? blockIdx.x / a.plan.chunks : (uint64_t)blockIdx.x * a.plan.segs;
  const uint64_t seg1 = a.plan.chunks > 1 ? seg0 + 1 : seg0 + a.plan.segs < a.plan.segments ? seg0 + a.plan.segs : a.plan.segments;
  int slot = 0;
  for (uint64_t seg = seg0; seg < seg1; ++seg) {
    const uint64_t first = seg * a.plan.per + part * a.plan.chunk;
    uint64_t end = part + 1 == a.plan.chunks ? (seg + 1) * a.plan.per : first + a.plan.chunk;
    if (end > (seg + 1) * a.plan.per) end = (seg + 1) * a.plan.per;
    if (end > b.rows) end = b.rows;
    Eight<T> gate[GATE == 1 ? NV : 1];
    if constexpr (GATE == 1) {
      const T* g = static_cast<const T*>(b.gate) + seg * b.ld_gate;
#pragma unroll
      for (int i = 0; i < NV; ++i) gate[i] = load8<T>(g + col[i], have[i]);
    }
    auto load = [&](uint64_t row) {
      Held<T, S, NV, GATE> r;
      const bool on = row < end;
      if (on) r.st = *reinterpret_cast<const float4*>(a.stats + 4 * row);
      else r.st = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int n = on ? have[i] : 0;
        r.dy[i] = load8<S>(static_cast<const S*>(a.dy) + (a.dy ? row * a.lddy + col[i] : 0), a.dy ? n : 0);
        r.dh[i] = load8<T>(static_cast<const T*>(a.dh) + (pre ? row * a.lddh + col[i] : 0), pre ? n : 0);
        r.y[i] = load8<S>(static_cast<const S*>(a.y) + (pre ? row * a.ldy + col[i] : 0), pre ? n : 0);
        r.o[i] = load8<T>(static_cast<const T*>(b.branch) + (has_o ? row * b.ld_branch + col[i] : 0), has_o ? n : 0);
        if constexpr (GATE == 2) r.g[i] = load8<T>(static_cast<const T*>(b.gate) + row * b.ld_gate + col[i], n);
      }
      return r;
    };
    for (uint64_t base_row = first; base_row < end; base_row += groups) {
      const uint64_t row = base_row + group;
      const bool on = row < end;
      const Held<T, S, NV, GATE> r = load(row);
      const float mo = post ? r.st.x : 0.0f, ro = post ? r.st.y : 1.0f;
      const float mp = pre ? r.st.z : 0.0f, rp = pre ? r.st.w : 0.0f;
      float sum[kOut] = {};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xh = (r.y[i][j] - mp) * rp, gh = r.dh[i][j] * wpre[i][j];
          const float base = r.dy[i][j] + rp * gh, oh = (r.o[i][j] - mo) * ro;
          float q = b.branch_scale * wpost[i][j];
          if constexpr (GATE == 1) q *= gate[i][j];
          if constexpr (GATE == 2) q *= r.g[i][j];
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
#pragma unroll
      for (int k = 0; k < (LN ? 8 : 3); ++k) sum[k] = wave_sum(sum[k]);
      if (W > 1) {
        if (threadIdx.x % 64 == 0) {
#pragma unroll
          for (int k = 0; k < kOut; k += 4)
            *reinterpret_cast<float4*>(&lds[slot][wave][k]) = make_float4(sum[k], sum[k + 1], sum[k + 2], sum[k + 3]);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kOut; ++k) sum[k] = 0.0f;
        for (uint32_t w = 0; w < W; ++w)
#pragma unroll
          for (int k = 0; k < kOut; k += 4) {
            const float4 o = *reinterpret_cast<const float4*>(&lds[slot][group * W + w][k]);
            sum[k] += o.x, sum[k + 1] += o.y, sum[k + 2] += o.z, sum[k + 3] += o.w;
          }
        slot ^= 1;
      }
      const float c1 = sum[0] * inv_n, m1 = LN && b.pre == ZERO_NORM_LAYER ? sum[3] * inv_n : 0.0f;
      float c2 = 0.0f, m2 = 0.0f;
      if (post) c2 = (sum[1] - rp * ((LN ? m1 * sum[LN ? 7 : 0] : 0.0f) + c1 * sum[2])) * inv_n;
      if (LN && b.post == ZERO_NORM_LAYER) m2 = (sum[LN ? 4 : 0] - rp * (m1 * sum[LN ? 6 : 0] + c1 * sum[LN ? 5 : 0])) * inv_n;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float dx[8], db[8], dg[8];
        Eight<T> bias{};
        if (GATE != 0 && b.post_bias) bias = load8<T>(static_cast<const T*>(b.post_bias) + col[i], have[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float dh = r.dh[i][j];
          const float xh = (r.y[i][j] - mp) * rp;
          const float D = r.dy[i][j] + rp * (dh * wpre[i][j]) - rp * (m1 + xh * c1);
          const float oh = (r.o[i][j] - mo) * ro;
          float u = b.branch_scale * D;
          if (GATE != 0) dg[j] = u * (oh * wpost[i][j] + (b.post_bias ? bias[j] : 0.0f));
          if constexpr (GATE == 1) u *= gate[i][j];
          if constexpr (GATE == 2) u *= r.g[i][j];
          dx[j] = scale * D;
          db[j] = ro * (u * wpost[i][j] - m2 - oh * c2);
          if (on) {
            s_pre_w[i][j] += dh * xh;
            s_post_w[i][j] += u * oh;
            if constexpr (LN) {
              s_pre_b[i][j] += dh;
              s_post_b[i][j] += u;
            }
            if constexpr (GATE == 1) s_gate[i][j] += dg[j];
          }
        }
        if (on) {
          if (a.dx) store8<S>(static_cast<S*>(a.dx) + row * a.lddx + col[i], have[i], dx, a.past_caches);
          if (a.dbranch) store8<T>(static_cast<T*>(a.dbranch) + row * a.lddbranch + col[i], have[i], db, a.past_caches);
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
    }
    if constexpr (GATE == 1) {
      if (a.plan.chunks > 1 || a.part[kGate]) {
        if (a.part[kGate])
          joined(s_gate, [&](uint32_t c, float t) { a.part[kGate][(uint64_t)blockIdx.x * d + c] = t; });
      } else if (a.dgate) {
        joined(s_gate, [&](uint32_t c, float t) {
          const uint64_t at = seg * a.lddgate + c;
          if (a.grad_f32) {
            float* o = static_cast<float*>(a.dgate) + at;
            *o = a.accumulate ? *o + t : t;
          } else {
            T* o = static_cast<T*>(a.dgate) + at;
            *o = (T)(a.accumulate ? (float)*o + t : t);
          }
        });
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) s_gate[i][j] = 0.0f;
      }
    }
  }
  auto leave = [&](int k, float (&s)[NV][8]) {
    if (a.part[k]) joined(s, [&](uint32_t c, float t) { a.part[k][(uint64_t)blockIdx.x * d + c] = t; });
  };
  leave(kPostW, s_post_w);
  leave(kPreW, s_pre_w);
  if constexpr (LN) {
    leave(kPostB, s_post_b);
    leave(kPreB, s_pre_b);
  }
}

template <typename T, typename S, int NV>
hipError_t backward_of(const BackwardArgs& a) {
  // biases are summed by the general variant only
  const bool ln = a.b.post == ZERO_NORM_LAYER || a.b.pre == ZERO_NORM_LAYER || a.part[kPostB] || a.part[kPreB];
  const dim3 grid((unsigned)a.plan.blocks), block(kBackThreads);
#define ZERO_GO(LN, GATE) k_backward<T, S, NV, LN, GATE><<<grid, block, 0, a.stream>>>(a)
  if (ln) {
    if (a.gate_mode == 0) ZERO_GO(true, 0);
    else if (a.gate_mode == 1) ZERO_GO(true, 1);
    else ZERO_GO(true, 2);
  } else {
    if (a.gate_mode == 0) ZERO_GO(false, 0);
    else if (a.gate_mode == 1) ZERO_GO(false, 1);
    else ZERO_GO(false, 2);
  }
#undef ZERO_GO
  return hipGetLastError();
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
  if (vecs <= 1024) {
    const dim3 block((unsigned)((vecs + 63) / 64 * 64));
    k_forward<T, S, 1><<<grid, block, 0, a.stream>>>(a, step, past);
  } else {
    const dim3 block((unsigned)(((vecs + 1) / 2 + 63) / 64 * 64));
    k_forward<T, S, 2><<<grid, block, 0, a.stream>>>(a, step, past);
  }
  return hipGetLastError();
}

template <>
hipError_t launch_backward<ZERO_NORM_DT, ZERO_NORM_S32 != 0>(const BackwardArgs& a) {
  typedef Of<ZERO_NORM_DT>::type T;
  typedef std::conditional<ZERO_NORM_S32 != 0, float, T>::type S;
  return a.plan.vecs == 1 ? backward_of<T, S, 1>(a) : backward_of<T, S, 2>(a);
}

}  // namespace norm
}  // namespace zero
