// Losses over tokens on gfx950: the log probability of each row's token, the clipped policy loss with a KL
// term, the preference loss of paired answers, and their gradient in the logits.
//
// One block per row. In base-2 logarithms with c = log2(e)/T, m one of the largest logits and s = sum over v but
// the token of 2^((z_v - m) c): leaving the token out keeps l = -log1p(s exp((m - z_y)/T)) and 1 - q_y = a/(1 + a) exact
// for tokens the model is sure of. Each lane's sum is fp32, the join of lanes and everything behind it fp64: the
// policy's ratio is compared with its clip, where an error in l decides a row's whole gradient. The gradient is
// F * 2^((z_v - M) c) for every entry, and the token's own over it.
//
// Memory is the bound: the loss alone and the gradient alone read the row once, and the policy's step keeps
// it in registers between the two, as far as it fits; longer rows are read twice. Measured on inputs that change
// from pass to pass: 8192 x 32000 bf16 with a tenth of the rows masked, loss and gradient 170 us (5.9 TB/s; a 2:1 stream
// reaches 6.0), loss alone 76 to 83 (5.7 to 6.2), in two calls 241 to 248; 1023 x 50257 fp32 in two calls 117 (its rows
// lie off 16 bytes); one row of 50257 bf16 10.4, which is a chain of loads and one CU's exponentials (two for an entry).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "zero_arrays.h"
#include "zero_internal.h"
#include "zero_rows.h"

namespace zero {
namespace {

constexpr uint64_t kMaxSize = 0x7fffffffu;
constexpr uint64_t kGridRows = 1u << 21;

// A row's stats: the softmax's largest logit and sum, dloss/dl, 1 - q of the token, l in two parts, which
// upstream (as bits), and whether the row has a token.
enum { kTop, kSum, kSlope, kRest, kLHigh, kLLow, kWhich, kOn };

struct Args {
  zero_token_in in;
  zero_policy p;
  int policy;                 // 0: the loss is l, with the derivative `slope`
  float slope;                // 1, or 0 where k_pairs sets it for the rows of its sequences
  double log_low, log_high;   // log of the ratio's range
  float c_hi, c_lo;           // log2(e)/T as a sum of two fp32 numbers
  int two;                    // the second is over 2^-26 of the first
  double inv_t;
  const float* stats_in;
  const float* upstream;
  uint64_t n_up;
  float scale;
  float *loss, *logp, *stats;
  void* dlogits;
  uint64_t ldg;
};

enum { kForward = 1, kBackward = 2, kStep = 3 };  // bit 0: loss, bit 1: gradient

// A place on the base-2 scale that exponentials are taken from: 2^(z c - k) is 2^((z - m) c) up to a factor that is
// the same for every z, k being m c rounded, and z c - k is one fused operation. The factor's exponent is what the
// rounding took: at most 1/2 for |k| up to 2^24, so it is used there. Further out (a row masked by -1e10, say, where it
// would pass fp32's range) k is infinite and differences are formed first; and so where c needs two fp32 numbers, as one
// takes up to 2^-26 of (m - z) c off an exponent, and more by the temperature.
struct From {
  float m, k;
};

__device__ __forceinline__ From from(const Args& a, float m) {
  const float k = m * a.c_hi;
  return From{m, !a.two && fabsf(k) <= 0x1p24f ? k : INFINITY};
}

// m c - k: what a place's rounding took
__device__ __forceinline__ float rounded_off(const Args& a, From f) {
  return f.k < INFINITY ? __builtin_fmaf(f.m, a.c_hi, -f.k) : 0.0f;
}

// c * d to fp32 accuracy. -inf is taken as the lowest finite number (c_lo may be negative or 0, and would
// make a NaN of it).
__device__ __forceinline__ float mul_c(const Args& a, float d) {
  d = d < kLowest ? kLowest : d;
  return __builtin_fmaf(d, a.c_hi, d * a.c_lo);
}

template <int N>
__device__ __forceinline__ void exponentials(const Args& a, From f, const float (&z)[N], float (&e)[N]) {
  if (f.k < INFINITY) {
#pragma unroll
    for (int j = 0; j < N; ++j) e[j] = ex2(__builtin_fmaf(z[j], a.c_hi, -f.k));
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) e[j] = ex2(mul_c(a, z[j] - f.m));
  }
}

__device__ __forceinline__ float exponential(const Args& a, From f, float z) {
  const float in[1] = {z};
  float e[1];
  exponentials<1>(a, f, in, e);
  return e[0];
}

// What a sum counted from `f` is multiplied by to count from `to`.
__device__ __forceinline__ float moved_to(const Args& a, From f, From to) {
  if (f.k < INFINITY && to.k < INFINITY) return ex2(f.k - to.k);
  return ex2(mul_c(a, f.m - to.m) - rounded_off(a, f) + rounded_off(a, to));
}

// A sum of exponentials and the place it counts from, one of the numbers seen. Starts at the lowest finite
// number, so that -inf entries add 0.
struct PlaceSum {
  From f;
  float s;
};

// Adds N values, but the one at `skip`, to a running sum. Its place moves only when the sum leaves the range (at the
// first values, and at values 2^40 over the place): a maximum of every value would cost as much again as the
// argument and the sum of its exponential.
template <int N>
__device__ __forceinline__ void add(const Args& a, PlaceSum& r, float (&z)[N], uint32_t skip) {
  if (skip < N) {
#pragma unroll
    for (int j = 0; j < N; ++j) z[j] = skip == (uint32_t)j ? -INFINITY : z[j];
  }
  float e[N], s = r.s;
  exponentials<N>(a, r.f, z, e);
#pragma unroll
  for (int j = 0; j < N; ++j) s += e[j];
  if (!(s < 0x1p40f)) {
    float m = r.f.m;
#pragma unroll
    for (int j = 0; j < N; ++j) m = z[j] > m ? z[j] : m;
    if (m > r.f.m) {
      const From to = from(a, m);
      if (r.s > 0.0f) r.s *= moved_to(a, r.f, to);
      r.f = to;
    }
    s = r.s;
    exponentials<N>(a, r.f, z, e);
#pragma unroll
    for (int j = 0; j < N; ++j) s += e[j];
  }
  r.s = s;
}

// exp(d) - 1 - d without the digits that cancel near 0; inf for either infinite d
__device__ __forceinline__ float kl_term(float d) {
  if (!(fabsf(d) < 0.5f)) {
    const float e = expm1f(d);
    return e == INFINITY ? e : e - d;
  }
  float s = 1.0f;
#pragma unroll
  for (int k = 9; k >= 3; --k) s = 1.0f + d * (1.0f / (float)k) * s;
  return 0.5f * d * d * s;
}

// fp64 functions to about 1e-11 relative, which is what l needs: the math library's, to the last place, are
// several times as long, and one wave of every row runs them while the row's other waves wait (8192 rows of 4096
// fp16: loss alone 22.3 us against 23.9, in one pass with the gradient 34.2 against 37.6).

// 1/x by two steps of Newton's from the approximate reciprocal
__device__ __forceinline__ double inverse(double x) {
  double r = __builtin_amdgcn_rcp(x);
  r = fma(fma(-x, r, 1.0), r, r);
  return fma(fma(-x, r, 1.0), r, r);
}

// 2^x for x up to 1000, by its series about the nearest whole exponent; 0 below -1100
__device__ __forceinline__ double exp2_of(double x) {
  x = x < -1100.0 ? -1100.0 : x;
  const double k = rint(x), f = (x - k) * 0.69314718055994530942;
  double p = 1.0 / 362880.0;
  p = fma(p, f, 1.0 / 40320.0);
  p = fma(p, f, 1.0 / 5040.0);
  p = fma(p, f, 1.0 / 720.0);
  p = fma(p, f, 1.0 / 120.0);
  p = fma(p, f, 1.0 / 24.0);
  p = fma(p, f, 1.0 / 6.0);
  p = fma(p, f, 0.5);
  p = fma(p, f, 1.0);
  p = fma(p, f, 1.0);
  return __builtin_amdgcn_ldexp(p, (int)k);
}

// log(1 + e) for e > -1/4, as k log 2 + 2 atanh(u): for e under sqrt(2) - 1 u = e/(2 + e), which keeps e's digits,
// else u = (m - 1)/(m + 1) with 1 + e = 2^k m, m about 1. |u| is under 0.172, and the series ends at u^13/13.
__device__ __forceinline__ double log1p_of(double e) {
  const double v = 1.0 + e;
  double k = 0.0, top = e, bottom = 2.0 + e;
  if (!(e < 0.41421356)) {
    double m = __builtin_amdgcn_frexp_mant(v);  // 1/2 to 1
    k = (double)__builtin_amdgcn_frexp_exp(v);
    if (m < 0.70710678) m *= 2.0, k -= 1.0;
    top = m - 1.0;
    bottom = m + 1.0;
  }
  const double u = top * inverse(bottom), q = u * u;
  double p = 1.0 / 13.0;
  p = fma(p, q, 1.0 / 11.0);
  p = fma(p, q, 1.0 / 9.0);
  p = fma(p, q, 1.0 / 7.0);
  p = fma(p, q, 1.0 / 5.0);
  p = fma(p, q, 1.0 / 3.0);
  p = fma(p, q, 1.0);
  return fma(k, 0.69314718055994530942, 2.0 * u * p);
}

// What one wave works out for a row and the others wait for.
struct Row {
  float top, sum;  // softmax: q_v = (exponential of z_v from `top`)/sum
  float slope;     // dloss/dl
  float rest;      // 1 - q of the token
};

// The row's softmax about its token from the other entries' sum s, counted from f, and its loss. Run by one wave,
// every lane alike.
__device__ __forceinline__ Row finish(const Args& a, uint64_t row, float z, From f, double s, float w, float old,
                                      float adv, float ref, int lane) {
  Row r;
  // k is m c rounded; the sum from m itself
  const double off = f.k < INFINITY ? exp2_of((double)f.k - (double)f.m * (double)a.c_hi) : 1.0;
  s *= off;
  const double t = ((double)z - (double)f.m) * a.inv_t;
  const bool above = t >= 0.0;  // of the others' place; below it s is at least 1 but for its rounding
  const double near = exp2_of(-fabs(t) * 1.4426950408889634074);
  const double e = above ? s * near : (s - 1.0) + near;
  const double log_total = log1p_of(e);
  double l = above ? -log_total : t - log_total;
  double rest = (above ? e : s) * inverse(1.0 + e);
  r.top = above ? z : f.m;
  r.sum = above ? (float)(1.0 + e) * exponential(a, from(a, z), z) : (float)((1.0 + e) * inverse(off));
  if (z == INFINITY) l = rest = NAN, r.sum = NAN;
  if (r.sum == 0.0f) l = rest = NAN, r.sum = NAN;
  r.rest = (float)rest;
  float loss = (float)l;
  r.slope = a.slope;
  if (a.policy) {
    const double x = l - (double)old;
    const bool stop = adv > 0.0f ? x > a.log_high : adv < 0.0f && x < a.log_low;
    const float ratio = expf((float)x);
    const float bound = adv > 0.0f ? 1.0f + a.p.clip_high : 1.0f - a.p.clip_low;
    loss = adv == 0.0f ? 0.0f : -(stop ? bound : ratio) * adv;
    r.slope = stop || adv == 0.0f ? 0.0f : -ratio * adv;
    if (a.p.ref_logp) {
      const float d = (float)((double)ref - l);
      loss += a.p.kl_coef * kl_term(d);
      r.slope -= a.p.kl_coef * expm1f(d);
    }
    if (l != l) loss = r.slope = NAN;  // no softmax, whatever the advantage
    loss *= w;
    r.slope *= w;
  }
  if (lane == 0) {
    if (a.loss) a.loss[row] = loss;
    if (a.logp) a.logp[row] = (float)l;
    if (a.stats) {
      float* o = a.stats + row * ZERO_TOKEN_STATS;
      const float high = (float)l;
      o[kTop] = r.top, o[kSum] = r.sum, o[kSlope] = r.slope, o[kRest] = r.rest;
      o[kLHigh] = high, o[kLLow] = isfinite(high) ? (float)(l - (double)high) : 0.0f;
      o[kWhich] = __uint_as_float((uint32_t)row), o[kOn] = 1.0f;
    }
  }
  return r;
}

// What a row without a token or weight leaves.
template <int MODE>
__device__ __forceinline__ void no_loss(const Args& a, uint64_t row, int t) {
  if (!(MODE & 1)) return;
  if (t == 0) {
    if (a.loss) a.loss[row] = 0.0f;
    if (a.logp) a.logp[row] = 0.0f;
  }
  if (a.stats && t < ZERO_TOKEN_STATS) a.stats[row * ZERO_TOKEN_STATS + t] = 0.0f;
}

template <typename T, int NT>
__device__ __forceinline__ void no_gradient(T* dz, uint32_t vocab, int t) {
  using V = typename Pack<T>::type;
  constexpr uint32_t W = Pack<T>::n;
  const uint32_t body = vocab / W, last = body * W + t;
  V zero = {};
  for (uint32_t i = t; i < body; i += NT) *reinterpret_cast<V*>(dz + (uint64_t)i * W) = zero;
  if (last < vocab) dz[last] = (T)0.0f;
}

// NV: 16-byte vectors of the row that a thread of the step holds in registers; 0: reads it again.
// STREAM: the logits are read and the gradient written past the caches.
template <typename T, int MODE, int NV, int NT, bool STREAM>
__global__ __launch_bounds__(NT) void k_token(Args a) {
  __shared__ float s_m[NT / 64];
  __shared__ double s_s[NT / 64];
  __shared__ Row s_row;
  using V = typename Pack<T>::type;
  constexpr int W = Pack<T>::n;
  const zero_token_in& in = a.in;
  const uint32_t vocab = (uint32_t)in.vocab;
  const uint64_t row = (uint64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= in.rows) return;
  const T* z = static_cast<const T*>(in.logits) + row * in.ld_logits;
  T* dz = static_cast<T*>(a.dlogits) + row * a.ldg;
  const int t = threadIdx.x, wave = t / 64;
  const uint32_t body = vocab / W;     // whole vectors
  const uint32_t last = body * W + t;  // a thread's element behind them, if < vocab

  auto load = [&](uint32_t i) -> V {
    const V* p = reinterpret_cast<const V*>(z + (uint64_t)i * W);
    if constexpr (STREAM && !(MODE == kStep && NV == 0)) return __builtin_nontemporal_load(p);
    else return *p;  // (a step whose row is not held reads it again)
  };
  V held[NV ? NV : 1];
  auto hold = [&]() {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * NT + t < (int)body) held[i] = load(i * NT + t);
  };
  // The token and the weight first, and nothing else of the row without them. Asking for the row beside them would take a
  // load's latency off a batch of few rows (256 x 50257 bf16 18.8 us, 19.5 so), but read every masked row (511 x 131072 bf16
  // with 1 row in 20 unmasked 84 us, 58 so).
  const int64_t label = in.label_bytes == 8 ? static_cast<const int64_t*>(in.label)[row]
                                            : static_cast<const int32_t*>(in.label)[row];
  const float w = (MODE & 1) && a.policy && a.p.weight ? a.p.weight[row] : 1.0f;
  float slope = 1.0f;
  if (MODE == kBackward) slope = a.stats_in[row * ZERO_TOKEN_STATS + kSlope];
  if (label < 0 || label >= (int64_t)vocab || w == 0.0f || slope == 0.0f) {
    no_loss<MODE>(a, row, t);
    if (MODE & 2) no_gradient<T, NT>(dz, vocab, t);
    return;
  }
  const uint32_t y = (uint32_t)label;
  hold();

  Row r;
  float up = a.upstream && MODE == kStep ? a.upstream[row] : 1.0f;
  if constexpr ((MODE & 1) != 0) {
    float zy = 0.0f, old = 0.0f, adv = 0.0f, ref = 0.0f;
    if (wave == 0) {
      zy = (float)z[y];
      if (a.policy) {
        old = a.p.old_logp[row], adv = a.p.advantage[row];
        if (a.p.ref_logp) ref = a.p.ref_logp[row];
      }
    }
    PlaceSum rest{from(a, kLowest), 0.0f};
    auto one = [&](V x, uint32_t i) {
      float f[W];
#pragma unroll
      for (int j = 0; j < W; ++j) f[j] = (float)x[j];
      add<W>(a, rest, f, y - i * W);
    };
    if constexpr (NV > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i * NT + t < (int)body) one(held[i], i * NT + t);
    } else {
      for (uint32_t i = t; i < body; i += 4 * NT) {
        V x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (i + u * NT < body) x[u] = load(i + u * NT);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (i + u * NT < body) one(x[u], i + u * NT);
      }
    }
    if (last < vocab && last != y) {
      float f[1] = {(float)z[last]};
      add<1>(a, rest, f, 1);
    }
    const From own = from(a, wave_reduce(rest.f.m, kLowest, [](float p, float q) { return p > q ? p : q; }));
    const double s = wave_sum((double)(rest.s * moved_to(a, rest.f, own)));
    if ((t & 63) == 0) s_m[wave] = own.m, s_s[wave] = s;
    __syncthreads();
    if (wave == 0) {
      float top = s_m[0];
#pragma unroll
      for (int i = 1; i < NT / 64; ++i) top = s_m[i] > top ? s_m[i] : top;
      const From all = from(a, top);
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < NT / 64; ++i) sum += s_s[i] * (double)moved_to(a, from(a, s_m[i]), all);
      r = finish(a, row, zy, all, sum, w, old, adv, ref, t);
      if ((MODE & 2) && t == 0) s_row = r;
    }
    if constexpr ((MODE & 2) != 0) {
      __syncthreads();
      r = s_row;
    }
  } else {
    const float* o = a.stats_in + row * ZERO_TOKEN_STATS;
    r.top = o[kTop], r.sum = o[kSum], r.slope = slope, r.rest = o[kRest];
    if (a.upstream) {
      const uint32_t k = __float_as_uint(o[kWhich]);
      up = k < a.n_up ? a.upstream[k] : NAN;
    }
  }

  if constexpr ((MODE & 2) != 0) {
    const float g = a.scale * up * r.slope * (float)a.inv_t;
    const float out = -g / r.sum;
    const From top = from(a, r.top);
    auto one = [&](V x, uint32_t i) {
      V v;
      float z[W], e[W];
#pragma unroll
      for (int j = 0; j < W; ++j) z[j] = (float)x[j];
      exponentials<W>(a, top, z, e);
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = (T)(out * e[j]);
      const uint32_t at = y - i * W;
      if (at < W) {
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = at == (uint32_t)j ? (T)(g * r.rest) : v[j];
      }
      if constexpr (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<V*>(dz + (uint64_t)i * W));
      else *reinterpret_cast<V*>(dz + (uint64_t)i * W) = v;
    };
    if constexpr (NV > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i * NT + t < (int)body) one(held[i], i * NT + t);
    } else {
      for (uint32_t i = t; i < body; i += 4 * NT) {
        V x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (i + u * NT < body) x[u] = load(i + u * NT);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (i + u * NT < body) one(x[u], i + u * NT);
      }
    }
    if (last < vocab) dz[last] = last == y ? (T)(g * r.rest) : (T)(out * exponential(a, top, (float)z[last]));
  }
}

// ------------------------------------------------------------------------------------------ pairs

constexpr int kPairThreads = 256;

// One block per pair: the sequences' sums from the rows' l, the loss, and each row's derivative.
__global__ __launch_bounds__(kPairThreads) void k_pairs(zero_preference p, uint64_t rows, float* stats, float* loss,
                                                        float* seq_logp) {
  __shared__ double lds[kPairThreads / 64][4];
  const uint64_t pair = blockIdx.x;
  int64_t edge[3];
#pragma unroll
  for (int i = 0; i < 3; ++i)
    edge[i] = p.start_bytes == 8 ? static_cast<const int64_t*>(p.seq_start)[2 * pair + i]
                                 : static_cast<const int32_t*>(p.seq_start)[2 * pair + i];
#pragma unroll
  for (int i = 0; i < 3; ++i) edge[i] = edge[i] < 0 ? 0 : edge[i] > (int64_t)rows ? (int64_t)rows : edge[i];
  const float w32 = p.weight ? p.weight[pair] : 1.0f;
  const float ref = p.ref_logp ? p.ref_logp[2 * pair] : 0.0f, ref2 = p.ref_logp ? p.ref_logp[2 * pair + 1] : 0.0f;
  double sum[4] = {};  // each sequence's l and number of tokens
#pragma unroll
  for (int i = 0; i < 2; ++i)
    for (int64_t r = edge[i] + threadIdx.x; r < edge[i + 1]; r += kPairThreads) {
      const float* o = stats + r * ZERO_TOKEN_STATS;
      sum[2 * i] += (double)o[kLHigh] + (double)o[kLLow];
      sum[2 * i + 1] += (double)o[kOn];
    }
#pragma unroll
  for (int k = 0; k < 4; ++k) sum[k] = wave_sum(sum[k]);
  if (threadIdx.x % 64 == 0)
#pragma unroll
    for (int k = 0; k < 4; ++k) lds[threadIdx.x / 64][k] = sum[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    sum[k] = 0.0;
    for (int i = 0; i < kPairThreads / 64; ++i) sum[k] += lds[i][k];
  }
  double l[2], n[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    n[i] = p.average && sum[2 * i + 1] > 0.0 ? sum[2 * i + 1] : 1.0;
    l[i] = sum[2 * i] / n[i];
  }
  double gap = l[0] - l[1];
  gap -= (double)ref - (double)ref2;
  const double x = (double)p.beta * gap - (double)p.margin, e = p.label_smoothing;
  const double w = (double)w32;
  // log(1 + exp(-|x|)), and the logistic function of -|x| and |x|
  const double far = exp2_of(-fabs(x) * 1.4426950408889634074), both = log1p_of(far);
  const double plus = x > 0.0 ? 0.0 : -x, minus = x > 0.0 ? x : 0.0;  // the rest of log(1 + exp(-x)), log(1 + exp(x))
  const double up = x > 0.0 ? 1.0 / (1.0 + far) : far / (1.0 + far);   // 1/(1 + exp(-x)), a NaN for one
  const double down = x > 0.0 ? far / (1.0 + far) : 1.0 / (1.0 + far);
  const double value = (e < 1.0 ? (1.0 - e) * (plus + both) : 0.0) + (e > 0.0 ? e * (minus + both) : 0.0);
  const double slope = w == 0.0 ? 0.0 : w * (double)p.beta * (e * up - (1.0 - e) * down);
  if (threadIdx.x == 0) {
    loss[pair] = w == 0.0 ? 0.0f : (float)(w * value);
    if (seq_logp) seq_logp[2 * pair] = (float)l[0], seq_logp[2 * pair + 1] = (float)l[1];
  }
  for (int i = 0; i < 2; ++i) {
    const float each = (float)((i ? -slope : slope) / n[i]);
    for (int64_t r = edge[i] + threadIdx.x; r < edge[i + 1]; r += kPairThreads) {
      float* o = stats + r * ZERO_TOKEN_STATS;
      if (o[kOn] != 0.0f) o[kSlope] = each;
      o[kWhich] = __uint_as_float((uint32_t)pair);
    }
  }
}

// -------------------------------------------------------------------------------------- host side

template <typename T, int MODE, int NV, int NT>
hipError_t launch_one(const Args& a, hipStream_t s) {
  // a row a block, over two dimensions, as one holds no more than 2^32 threads
  const uint64_t wide = a.in.rows < kGridRows ? a.in.rows : kGridRows;
  const dim3 grid((unsigned)wide, (unsigned)((a.in.rows + wide - 1) / wide)), block(NT);
  // Logits and a gradient of 128 MiB and more go past the caches, which would hardly hold them until they are next
  // read (8192 x 32000 bf16 loss alone 76 us, 86 through them; 1023 x 50257 fp32 36 and 38); smaller ones stay for
  // whoever reads them next.
  if (a.in.rows * a.in.vocab * sizeof(T) >= (128ull << 20)) {
    k_token<T, MODE, NV, NT, true><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
  }
  k_token<T, MODE, NV, NT, false><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch(const Args& a, int mode, hipStream_t s) {
  const uint64_t v = a.in.vocab / Pack<T>::n;  // vectors of a row
#define ZERO_GO(MODE, NV, NT) return launch_one<T, MODE, NV, NT>(a, s)
  // Few rows: 1024 threads on each, for the latency of one. Many: small blocks, several to a CU, so that one's loads run
  // under another's arithmetic and stores; but the gradient alone, which waits for nothing, in whole CUs' worth (8192 x
  // 32000 bf16 171 us, 256 threads 193), and a row that is read twice, which so stays in the caches (2048 x 131072 bf16
  // 230 us, 512 threads 241, held by 1024 threads 392).
  const bool wide = a.in.rows < 512;
  if (mode == kForward) {
    if (wide) ZERO_GO(kForward, 0, 1024);
    if (v > 4096) ZERO_GO(kForward, 0, 512);
    ZERO_GO(kForward, 0, 256);
  }
  if (mode == kBackward) {
    if (wide || v > 2048) ZERO_GO(kBackward, 0, 1024);
    ZERO_GO(kBackward, 0, 256);
  }
  if (wide) {
    if (v <= 4 * 1024) ZERO_GO(kStep, 4, 1024);
    if (v <= 8 * 1024) ZERO_GO(kStep, 8, 1024);
    if (v <= 16 * 1024) ZERO_GO(kStep, 16, 1024);
  } else {
    if (v <= 4 * 128) ZERO_GO(kStep, 4, 128);
    if (v <= 8 * 128) ZERO_GO(kStep, 8, 128);
    if (v <= 8 * 256) ZERO_GO(kStep, 8, 256);
    if (v <= 8 * 512) ZERO_GO(kStep, 8, 512);
    if (v <= 16 * 512) ZERO_GO(kStep, 16, 512);
    if (v <= 28 * 512) ZERO_GO(kStep, 28, 512);
  }
  ZERO_GO(kStep, 0, 1024);
#undef ZERO_GO
}

hipError_t launch_dtype(const Args& a, int mode, hipStream_t s) {
  switch (a.in.logit_dtype) {
    case ZERO_F32: return launch<float>(a, mode, s);
    case ZERO_F16: return launch<_Float16>(a, mode, s);
    default: return launch<__bf16>(a, mode, s);
  }
}

// The inputs' own checks (no arrays), and what of `a` they give.
zero_status check_in(const char* fn, const zero_token_in* in, Args& a) {
  if (!in) return fail(ZERO_E_INVAL, "%s: in is NULL", fn);
  if (!dtype_valid(in->logit_dtype)) return fail(ZERO_E_UNSUPPORTED, "%s: logits must be fp32, fp16 or bf16", fn);
  if (in->label_bytes != 4 && in->label_bytes != 8)
    return fail(ZERO_E_INVAL, "%s: label_bytes %d is not 4 or 8", fn, in->label_bytes);
  if (in->vocab == 0) return fail(ZERO_E_INVAL, "%s: vocab is 0", fn);
  if (in->rows > kMaxSize || in->vocab > kMaxSize) return fail(ZERO_E_OVERFLOW, "%s: rows or vocab above 2^31 - 1", fn);
  if (!(in->temperature >= 0x1p-20f && in->temperature <= 0x1p20f))
    return fail(ZERO_E_INVAL, "%s: temperature must lie in [2^-20, 2^20]", fn);
  if (in->rows && (!in->logits || !in->label)) return fail(ZERO_E_INVAL, "%s: NULL argument", fn);
  const uint64_t ld = in->rows > 1 ? in->ld_logits : in->vocab;
  if (ld < in->vocab) return fail(ZERO_E_INVAL, "%s: a leading dimension below the columns", fn);
  if (in->rows && ld >= (1ull << 63) / 4 / in->rows)
    return fail(ZERO_E_OVERFLOW, "%s: a byte count does not fit in 63 bits", fn);
  a.in = *in;
  a.slope = 1.0f;
  a.in.ld_logits = ld;
  const double c = 1.4426950408889634074 / (double)in->temperature;
  a.c_hi = (float)c;
  a.c_lo = (float)(c - (double)a.c_hi);
  a.two = fabsf(a.c_lo) > 0x1p-26f * a.c_hi;
  a.inv_t = 1.0 / (double)in->temperature;
  return ZERO_OK;
}

zero_status check_policy(const char* fn, const zero_policy* p, uint64_t rows, Args& a) {
  if (!p) return fail(ZERO_E_INVAL, "%s: p is NULL", fn);
  if (!(p->clip_low >= 0.0f && p->clip_low <= 1.0f && p->clip_high >= 0.0f && isfinite(p->clip_high) &&
        p->kl_coef >= 0.0f && isfinite(p->kl_coef)))
    return fail(ZERO_E_INVAL, "%s: clip_low must lie in [0, 1], clip_high and kl_coef be finite and not negative", fn);
  if (rows && (!p->old_logp || !p->advantage)) return fail(ZERO_E_INVAL, "%s: NULL old_logp or advantage", fn);
  a.policy = 1;
  a.p = *p;
  if (p->kl_coef == 0.0f) a.p.ref_logp = nullptr;
  a.log_low = log1p(-(double)p->clip_low);
  a.log_high = log1p((double)p->clip_high);
  return ZERO_OK;
}

// The arrays of a call, as check_arrays takes them.
Arr logits_of(const Args& a) {
  return Arr{"logits", a.in.logits, a.in.rows, a.in.vocab, a.in.ld_logits, dtype_bytes(a.in.logit_dtype), false};
}

Arr dlogits_of(const Args& a) {
  return Arr{"dlogits", a.dlogits, a.in.rows, a.in.vocab, a.ldg, dtype_bytes(a.in.logit_dtype), true};
}

Arr label_of(const Args& a) {
  return Arr{"label", a.in.label, 1, a.in.rows, a.in.rows, (uint32_t)a.in.label_bytes, false};
}

Arr floats(const char* name, const float* p, uint64_t n, bool written) { return Arr{name, p, 1, n, n, 4, written}; }

zero_status check_dlogits(const char* fn, Args& a, void* dlogits, uint64_t ldg) {
  if (a.in.rows && !dlogits) return fail(ZERO_E_INVAL, "%s: NULL argument", fn);
  const uint64_t ld = a.in.rows > 1 ? ldg : a.in.vocab;
  if (ld < a.in.vocab) return fail(ZERO_E_INVAL, "%s: a leading dimension below the columns", fn);
  if (a.in.rows && ld >= (1ull << 63) / 4 / a.in.rows)
    return fail(ZERO_E_OVERFLOW, "%s: a byte count does not fit in 63 bits", fn);
  a.dlogits = dlogits;
  a.ldg = ld;
  return ZERO_OK;
}

zero_status launched(const char* fn, hipError_t e) {
  if (e != hipSuccess) return fail(ZERO_E_HIP, "%s launch: %s", fn, hipGetErrorString(e));
  return ok();
}

zero_status policy(const char* fn, const zero_token_in* in, const zero_policy* p, const float* upstream, float scale,
                   float* loss, float* logp, float* stats, void* dlogits, uint64_t ldg, int mode, void* stream) {
  Args a{};
  zero_status st = check_in(fn, in, a);
  if (st == ZERO_OK) st = check_policy(fn, p, in->rows, a);
  if (st == ZERO_OK && mode == kStep) st = check_dlogits(fn, a, dlogits, ldg);
  if (st != ZERO_OK) return st;
  if (!isfinite(scale)) return fail(ZERO_E_INVAL, "%s: scale is not finite", fn);
  if (in->rows == 0) return ok();
  if (!loss || (mode == kForward && !stats)) return fail(ZERO_E_INVAL, "%s: NULL argument", fn);
  const uint64_t R = in->rows;
  const Arr arr[] = {logits_of(a),
                     dlogits_of(a),
                     label_of(a),
                     floats("old_logp", p->old_logp, R, false),
                     floats("advantage", p->advantage, R, false),
                     floats("ref_logp", p->ref_logp, R, false),
                     floats("weight", p->weight, R, false),
                     floats("upstream", upstream, R, false),
                     floats("loss", loss, R, true),
                     floats("logp", logp, R, true),
                     floats("stats", stats, R * ZERO_TOKEN_STATS, true)};
  st = check_arrays(fn, arr, sizeof(arr) / sizeof(arr[0]), 1, 0);
  if (st != ZERO_OK) return st;
  a.upstream = upstream;
  a.n_up = R;
  a.scale = scale;
  a.loss = loss;
  a.logp = logp;
  a.stats = stats;
  (void)hipGetLastError();
  return launched(fn, launch_dtype(a, mode, static_cast<hipStream_t>(stream)));
}

}  // namespace
}  // namespace zero

extern "C" {

zero_status zero_token_logp(const zero_token_in* in, float* logp, float* stats, void* stream) {
  const char* fn = "zero_token_logp";
  zero::Args a{};
  zero_status st = zero::check_in(fn, in, a);
  if (st != ZERO_OK) return st;
  if (in->rows == 0) return zero::ok();
  if (!logp) return zero::fail(ZERO_E_INVAL, "%s: NULL argument", fn);
  const uint64_t R = in->rows;
  const zero::Arr arr[] = {zero::logits_of(a), zero::label_of(a), zero::floats("logp", logp, R, true),
                           zero::floats("stats", stats, R * ZERO_TOKEN_STATS, true)};
  st = zero::check_arrays(fn, arr, 4);
  if (st != ZERO_OK) return st;
  a.logp = logp;
  a.stats = stats;
  (void)hipGetLastError();
  return zero::launched(fn, zero::launch_dtype(a, zero::kForward, static_cast<hipStream_t>(stream)));
}

zero_status zero_policy_forward(const zero_token_in* in, const zero_policy* p, float* loss, float* logp, float* stats,
                                void* stream) {
  return zero::policy("zero_policy_forward", in, p, nullptr, 1.0f, loss, logp, stats, nullptr, 0, zero::kForward, stream);
}

zero_status zero_policy_step(const zero_token_in* in, const zero_policy* p, const float* upstream, float scale,
                             float* loss, float* logp, void* dlogits, uint64_t ld_dlogits, void* stream) {
  return zero::policy("zero_policy_step", in, p, upstream, scale, loss, logp, nullptr, dlogits, ld_dlogits, zero::kStep,
                      stream);
}

zero_status zero_preference_forward(const zero_token_in* in, const zero_preference* p, float* loss, float* logp,
                                    float* seq_logp, float* stats, void* stream) {
  const char* fn = "zero_preference_forward";
  zero::Args a{};
  zero_status st = zero::check_in(fn, in, a);
  if (st != ZERO_OK) return st;
  if (!p) return zero::fail(ZERO_E_INVAL, "%s: p is NULL", fn);
  if (p->start_bytes != 4 && p->start_bytes != 8)
    return zero::fail(ZERO_E_INVAL, "%s: start_bytes %d is not 4 or 8", fn, p->start_bytes);
  if (!(isfinite(p->beta) && isfinite(p->margin) && p->label_smoothing >= 0.0f && p->label_smoothing <= 1.0f))
    return zero::fail(ZERO_E_INVAL, "%s: beta and margin must be finite, label_smoothing lie in [0, 1]", fn);
  if (p->pairs > 1ull << 23) return zero::fail(ZERO_E_OVERFLOW, "%s: pairs above 2^23", fn);
  if ((p->pairs && (!p->seq_start || !loss)) || (in->rows && !stats))
    return zero::fail(ZERO_E_INVAL, "%s: NULL argument", fn);
  const uint64_t R = in->rows, P = p->pairs;
  const uint64_t starts = P ? 2 * P + 1 : 0;
  const zero::Arr arr[] = {zero::logits_of(a),
                           zero::label_of(a),
                           {"seq_start", p->seq_start, 1, starts, starts, (uint32_t)p->start_bytes, false},
                           zero::floats("ref_logp", p->ref_logp, 2 * P, false),
                           zero::floats("weight", p->weight, P, false),
                           zero::floats("loss", loss, P, true),
                           zero::floats("logp", logp, R, true),
                           zero::floats("seq_logp", seq_logp, 2 * P, true),
                           zero::floats("stats", stats, R * ZERO_TOKEN_STATS, true)};
  st = zero::check_arrays(fn, arr, sizeof(arr) / sizeof(arr[0]));
  if (st != ZERO_OK) return st;
  if (R == 0 && P == 0) return zero::ok();
  a.logp = logp;
  a.stats = stats;
  a.slope = 0.0f;
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  hipError_t e = hipSuccess;
  if (R) {
    e = zero::launch_dtype(a, zero::kForward, s);
  }
  if (e == hipSuccess && P) {
    zero::k_pairs<<<dim3((unsigned)P), dim3(zero::kPairThreads), 0, s>>>(*p, R, stats, loss, seq_logp);
    e = hipGetLastError();
  }
  return zero::launched(fn, e);
}

zero_status zero_token_backward(const zero_token_in* in, const float* stats, const float* upstream, uint64_t n_upstream,
                                float scale, void* dlogits, uint64_t ld_dlogits, void* stream) {
  const char* fn = "zero_token_backward";
  zero::Args a{};
  zero_status st = zero::check_in(fn, in, a);
  if (st == ZERO_OK) st = zero::check_dlogits(fn, a, dlogits, ld_dlogits);
  if (st != ZERO_OK) return st;
  if (!isfinite(scale)) return zero::fail(ZERO_E_INVAL, "%s: scale is not finite", fn);
  if (in->rows == 0) return zero::ok();
  if (!stats) return zero::fail(ZERO_E_INVAL, "%s: NULL argument", fn);
  if (n_upstream > zero::kMaxSize) return zero::fail(ZERO_E_OVERFLOW, "%s: n_upstream above 2^31 - 1", fn);
  const uint64_t R = in->rows;
  const zero::Arr arr[] = {zero::logits_of(a), zero::dlogits_of(a), zero::label_of(a),
                           zero::floats("stats", stats, R * ZERO_TOKEN_STATS, false),
                           zero::floats("upstream", upstream, n_upstream, false)};
  st = zero::check_arrays(fn, arr, 5, 1, 0);
  if (st != ZERO_OK) return st;
  a.stats_in = stats;
  a.upstream = upstream;
  a.n_up = n_upstream;
  a.scale = scale;
  (void)hipGetLastError();
  return zero::launched(fn, zero::launch_dtype(a, zero::kBackward, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
