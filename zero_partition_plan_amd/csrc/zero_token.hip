// Losses over tokens on gfx950: the log probability of each row's token, the clipped policy loss with a KL
// term, the preference loss of paired answers, and their gradient in the logits.
//
// One block per row. In base-2 logarithms with c = log2(e)/T, m the largest logit but the token's and
// s = sum over v but the token of 2^((z_v - m) c): leaving the token out keeps l = -log1p(s exp((m - z_y)/T)) and
// 1 - q_y = a/(1 + a) exact for tokens the model is sure of. Each lane's sum is fp32, the join of lanes and
// everything behind it fp64: the policy's ratio is compared with its clip, where an error in l decides a
// row's whole gradient. The gradient is F * 2^((z_v - M) c) for every entry, and the token's own over it.
//
// Memory is the bound: the loss alone and the gradient alone read the row once, and the policy's step keeps
// it in registers between the two, as far as it fits; longer rows are read twice.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

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

// c * d to fp32 accuracy: c in one fp32 number is off by up to 2^-25 of it with one sign for every entry,
// which the sum's logarithm would carry into l. -inf is taken as the lowest finite number (c_lo may be
// negative or 0, and would make a NaN of it).
__device__ __forceinline__ float mul_c(const Args& a, float d) {
  d = d < kLowest ? kLowest : d;
  return __builtin_fmaf(d, a.c_hi, d * a.c_lo);
}

// A running maximum and the sum of 2^((z - m) c). Starts at the lowest finite number, so that -inf entries add 0.
struct MaxSum {
  float m, s;
};

// Adds N values, but the one at `skip`, to a running sum.
template <int N>
__device__ __forceinline__ void add(const Args& a, MaxSum& r, float (&f)[N], uint32_t skip) {
  if (skip < N) {
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = skip == (uint32_t)j ? -INFINITY : f[j];
  }
  float m = f[0];
#pragma unroll
  for (int j = 1; j < N; ++j) m = f[j] > m ? f[j] : m;
  if (m > r.m) {
    r.s *= ex2(mul_c(a, r.m - m));
    r.m = m;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) r.s += ex2(mul_c(a, f[j] - r.m));
}

// exp(d) - 1 - d without the digits that cancel near 0
__device__ __forceinline__ float kl_term(float d) {
  if (!(fabsf(d) < 0.5f)) return expm1f(d) - d;
  float s = 1.0f;
#pragma unroll
  for (int k = 9; k >= 3; --k) s = 1.0f + d * (1.0f / (float)k) * s;
  return 0.5f * d * d * s;
}

// What one wave works out for a row and the others wait for.
struct Row {
  float top, sum;  // softmax: q_v = 2^((z_v - top) c)/sum
  float slope;     // dloss/dl
  float rest;      // 1 - q of the token
};

// The row's softmax about its token from the other entries' largest m and sum s, and its loss. Run by one wave,
// every lane alike.
__device__ __forceinline__ Row finish(const Args& a, uint64_t row, float z, float m, double s, float w, float old,
                                      float adv, float ref, int lane) {
  Row r;
  double l, rest;
  const double t = ((double)z - (double)m) * a.inv_t;
  if (t >= 0.0) {
    const double e = s * exp(-t);
    l = -log1p(e);
    rest = e / (1.0 + e);
    r.top = z;
    r.sum = (float)(1.0 + e);
  } else {
    const double total = s + exp(t);
    l = t - log(total);
    rest = s / total;
    r.top = m;
    r.sum = (float)total;
  }
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
// STREAM: the gradient goes past the caches.
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

  // the token and the weight first, and nothing else of the row without them
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
  V held[NV ? NV : 1];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (i * NT + t < (int)body) held[i] = *reinterpret_cast<const V*>(z + (uint64_t)(i * NT + t) * W);

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
    MaxSum rest{kLowest, 0.0f};
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
      uint32_t i = t;
      for (; i + 3 * NT < body; i += 4 * NT) {
        V x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = *reinterpret_cast<const V*>(z + (uint64_t)(i + u * NT) * W);
#pragma unroll
        for (int u = 0; u < 4; ++u) one(x[u], i + u * NT);
      }
      for (; i < body; i += NT) one(*reinterpret_cast<const V*>(z + (uint64_t)i * W), i);
    }
    if (last < vocab && last != y) {
      float f[1] = {(float)z[last]};
      add<1>(a, rest, f, 1);
    }
    const float m = wave_reduce(rest.m, kLowest, [](float p, float q) { return p > q ? p : q; });
    const double s = wave_sum((double)(rest.s * ex2(mul_c(a, rest.m - m))));
    if ((t & 63) == 0) s_m[wave] = m, s_s[wave] = s;
    __syncthreads();
    if (wave == 0) {
      float top = s_m[0];
#pragma unroll
      for (int i = 1; i < NT / 64; ++i) top = s_m[i] > top ? s_m[i] : top;
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < NT / 64; ++i) sum += s_s[i] * (double)ex2(mul_c(a, s_m[i] - top));
      r = finish(a, row, zy, top, sum, w, old, adv, ref, t);
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
    const float out = -g / r.sum, m = r.top;
    auto one = [&](V x, uint32_t i) {
      V v;
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = (T)(out * ex2(mul_c(a, (float)x[j] - m)));
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
      uint32_t i = t;
      for (; i + 3 * NT < body; i += 4 * NT) {
        V x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = *reinterpret_cast<const V*>(z + (uint64_t)(i + u * NT) * W);
#pragma unroll
        for (int u = 0; u < 4; ++u) one(x[u], i + u * NT);
      }
      for (; i < body; i += NT) one(*reinterpret_cast<const V*>(z + (uint64_t)i * W), i);
    }
    if (last < vocab) dz[last] = last == y ? (T)(g * r.rest) : (T)(out * ex2(mul_c(a, (float)z[last] - m)));
  }
}

// ------------------------------------------------------------------------------------------ pairs

constexpr int kPairThreads = 256;

// Sums of two numbers over the block, in a fixed order, in every thread.
__device__ __forceinline__ void block_sums(double& x, double& y, double (*lds)[2]) {
  x = wave_sum(x), y = wave_sum(y);
  const int wave = threadIdx.x / 64;
  __syncthreads();
  if (threadIdx.x % 64 == 0) lds[wave][0] = x, lds[wave][1] = y;
  __syncthreads();
  x = y = 0.0;
  for (int i = 0; i < kPairThreads / 64; ++i) x += lds[i][0], y += lds[i][1];
}

// One block per pair: the sequences' sums from the rows' l, the loss, and each row's derivative.
__global__ __launch_bounds__(kPairThreads) void k_pairs(zero_preference p, uint64_t rows, float* stats, float* loss,
                                                        float* seq_logp) {
  __shared__ double lds[kPairThreads / 64][2];
  const uint64_t pair = blockIdx.x;
  int64_t edge[3];
  for (int i = 0; i < 3; ++i) {
    const int64_t e = p.start_bytes == 8 ? static_cast<const int64_t*>(p.seq_start)[2 * pair + i]
                                         : static_cast<const int32_t*>(p.seq_start)[2 * pair + i];
    edge[i] = e < 0 ? 0 : e > (int64_t)rows ? (int64_t)rows : e;
  }
  double l[2], n[2];
  for (int i = 0; i < 2; ++i) {
    double sum = 0.0, count = 0.0;
    for (int64_t r = edge[i] + threadIdx.x; r < edge[i + 1]; r += kPairThreads) {
      const float* o = stats + r * ZERO_TOKEN_STATS;
      sum += (double)o[kLHigh] + (double)o[kLLow];
      count += (double)o[kOn];
    }
    block_sums(sum, count, lds);
    n[i] = p.average && count > 0.0 ? count : 1.0;
    l[i] = sum / n[i];
  }
  double gap = l[0] - l[1];
  if (p.ref_logp) gap -= (double)p.ref_logp[2 * pair] - (double)p.ref_logp[2 * pair + 1];
  const double x = (double)p.beta * gap - (double)p.margin, e = p.label_smoothing;
  const double w = p.weight ? (double)p.weight[pair] : 1.0;
  // log(1 + exp(-|x|)), and the logistic function of -|x| and |x|
  const double far = exp(-fabs(x)), both = log1p(far);
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
  // a gradient of 128 MiB and more would push the logits out of the memory side cache; a smaller one stays for
  // whoever reads it next
  if constexpr ((MODE & 2) != 0) {
    if (a.in.rows * a.in.vocab * sizeof(T) >= (128ull << 20)) {
      k_token<T, MODE, NV, NT, true><<<grid, block, 0, s>>>(a);
      return hipGetLastError();
    }
  }
  k_token<T, MODE, NV, NT, false><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch(const Args& a, int mode, hipStream_t s) {
  const uint64_t v = a.in.vocab / Pack<T>::n;  // vectors of a row
#define ZERO_GO(MODE, NV, NT) return launch_one<T, MODE, NV, NT>(a, s)
  // Few rows: 1024 threads on each, for the latency of one. Many: small blocks, several to a CU.
  const bool wide = a.in.rows < 512;
  if (mode == kForward) {
    if (wide) ZERO_GO(kForward, 0, 1024);
    if (v > 4096) ZERO_GO(kForward, 0, 512);
    ZERO_GO(kForward, 0, 256);
  }
  if (mode == kBackward) {
    if (wide) ZERO_GO(kBackward, 0, 1024);
    if (v > 4096) ZERO_GO(kBackward, 0, 512);
    ZERO_GO(kBackward, 0, 256);
  }
  if (wide) {
    if (v <= 4 * 1024) ZERO_GO(kStep, 4, 1024);
    if (v <= 8 * 1024) ZERO_GO(kStep, 8, 1024);
  } else {
    if (v <= 4 * 256) ZERO_GO(kStep, 4, 256);
    if (v <= 8 * 256) ZERO_GO(kStep, 8, 256);
    if (v <= 16 * 256) ZERO_GO(kStep, 16, 256);
    if (v <= 28 * 256) ZERO_GO(kStep, 28, 256);
    if (v <= 28 * 512) ZERO_GO(kStep, 28, 512);
  }
  if (v <= 16 * 1024) ZERO_GO(kStep, 16, 1024);
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

struct Arr {
  const char* name;
  const void* p;
  uint64_t bytes;
  uint32_t align;
  bool written;
};

// Alignment of every array and overlaps of the written ones; in_place: arr[x] may be arr[y].
zero_status check_arrays(const char* fn, const Arr* arr, int n, int x0 = -1, int y0 = -1) {
  for (int i = 0; i < n; ++i)
    if (arr[i].p && arr[i].bytes && reinterpret_cast<uintptr_t>(arr[i].p) % arr[i].align)
      return fail(ZERO_E_INVAL, "%s: %s is not aligned to its element size", fn, arr[i].name);
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j) {
      if (!arr[i].written || i == j || !arr[i].p || !arr[j].p) continue;
      if (i == x0 && j == y0 && arr[i].p == arr[j].p) continue;
      if (overlaps(arr[i].p, arr[i].bytes, arr[j].p, arr[j].bytes))
        return fail(ZERO_E_INVAL, "%s: %s overlaps %s", fn, arr[i].name, arr[j].name);
    }
  return ZERO_OK;
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

uint64_t logit_bytes(const Args& a, uint64_t ld) {
  return ((a.in.rows - 1) * ld + a.in.vocab) * dtype_bytes(a.in.logit_dtype);
}

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
  const uint32_t e = dtype_bytes(in->logit_dtype);
  const Arr arr[] = {{"logits", in->logits, logit_bytes(a, a.in.ld_logits), e, false},
                     {"dlogits", mode == kStep ? dlogits : nullptr, mode == kStep ? logit_bytes(a, a.ldg) : 0, e, true},
                     {"label", in->label, R * in->label_bytes, (uint32_t)in->label_bytes, false},
                     {"old_logp", p->old_logp, R * 4, 4, false},
                     {"advantage", p->advantage, R * 4, 4, false},
                     {"ref_logp", p->ref_logp, R * 4, 4, false},
                     {"weight", p->weight, R * 4, 4, false},
                     {"upstream", upstream, R * 4, 4, false},
                     {"loss", loss, R * 4, 4, true},
                     {"logp", logp, R * 4, 4, true},
                     {"stats", stats, R * ZERO_TOKEN_STATS * 4, 4, true}};
  const bool in_place = mode == kStep && a.ldg == a.in.ld_logits;
  st = check_arrays(fn, arr, sizeof(arr) / sizeof(arr[0]), in_place ? 1 : -1, 0);
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
  const zero::Arr arr[] = {
      {"logits", in->logits, zero::logit_bytes(a, a.in.ld_logits), zero::dtype_bytes(in->logit_dtype), false},
      {"label", in->label, R * in->label_bytes, (uint32_t)in->label_bytes, false},
      {"logp", logp, R * 4, 4, true},
      {"stats", stats, R * ZERO_TOKEN_STATS * 4, 4, true}};
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
  const zero::Arr arr[] = {
      {"logits", in->logits, R ? zero::logit_bytes(a, a.in.ld_logits) : 0, zero::dtype_bytes(in->logit_dtype), false},
      {"label", in->label, R * in->label_bytes, (uint32_t)in->label_bytes, false},
      {"seq_start", p->seq_start, P ? (2 * P + 1) * p->start_bytes : 0, (uint32_t)p->start_bytes, false},
      {"ref_logp", p->ref_logp, 2 * P * 4, 4, false},
      {"weight", p->weight, P * 4, 4, false},
      {"loss", loss, P * 4, 4, true},
      {"logp", logp, R * 4, 4, true},
      {"seq_logp", seq_logp, 2 * P * 4, 4, true},
      {"stats", stats, R * ZERO_TOKEN_STATS * 4, 4, true}};
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
  const uint32_t eb = zero::dtype_bytes(in->logit_dtype);
  const zero::Arr arr[] = {
      {"logits", in->logits, zero::logit_bytes(a, a.in.ld_logits), eb, false},
      {"dlogits", dlogits, zero::logit_bytes(a, a.ldg), eb, true},
      {"label", in->label, R * in->label_bytes, (uint32_t)in->label_bytes, false},
      {"stats", stats, R * ZERO_TOKEN_STATS * 4, 4, false},
      {"upstream", upstream, n_upstream * 4, 4, false}};
  st = zero::check_arrays(fn, arr, 5, a.ldg == a.in.ld_logits ? 1 : -1, 0);
  if (st != ZERO_OK) return st;
  a.stats_in = stats;
  a.upstream = upstream;
  a.n_up = n_upstream;
  a.scale = scale;
  (void)hipGetLastError();
  return zero::launched(fn, zero::launch_dtype(a, zero::kBackward, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
