// Distillation from a teacher's top logits on gfx950: loss, gradient, and both.
//
// One block per row. In base-2 logarithms with c = log2(e)/T, m the row's largest logit and
// s = sum over v of 2^((z_v - m) c):  log2 q_v = (z_v - m) c - log2 s. The row's logits are read
// once with a running (m, s) per thread, joined in a fixed order. With a tail, the sum runs over
// the entries that are not listed only (a bitmap in LDS says which), so that the student's
// remaining mass comes from a sum of its own and not from 1 minus a sum close to 1; the listed
// entries, at most 1024, are joined to it afterwards. The gradient is a second pass that writes
// F * 2^((z_v - m) c) for every entry and then the listed ones over it.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "zero_internal.h"

namespace zero {
namespace {

constexpr uint64_t kMaxSize = 0x7fffffffu;
constexpr float kLowest = -3.402823466e38f;
constexpr float kLn2 = 0.69314718055994530942f;

struct Args {
  zero_distill_in in;
  float c_hi, c_lo;  // log2(e)/T as a sum of two fp32 numbers
  float inv_t;
  const float* stats_in;
  const float* upstream;
  float scale;
  float *loss, *stats;
  void* dlogits;
  uint64_t ldg;
};

enum { kForward = 1, kBackward = 2, kStep = 3 };  // bit 0: loss, bit 1: gradient

// c * d for a difference of logits d, to fp32 accuracy: c in one fp32 number would lose up to
// 2^-25 |c d| to its own rounding, seen in the small probabilities of an fp32 gradient. -inf is taken
// as the lowest finite number (c_lo may be negative or 0, and would make a NaN of it); T is at most
// 2^20, so that is still an exponent far below any fp32.
__device__ __forceinline__ float mul_c(const Args& a, float d) {
  d = d < kLowest ? kLowest : d;
  return __builtin_fmaf(d, a.c_hi, d * a.c_lo);
}

// The same inside the pass over the logits: 16-bit logits, whose gradient is rounded to 16 bits,
// take the one-term product.
template <typename T>
__device__ __forceinline__ float mul_s(const Args& a, float d) {
  return sizeof(T) == 4 ? mul_c(a, d) : d * a.c_hi;
}

// A running maximum and the sum of 2^((z - m) c). Starts at the lowest finite number, so that
// -inf entries add 0 and a row of the type's lowest values is an ordinary row.
struct MaxSum {
  float m, s;
};

__device__ __forceinline__ MaxSum join(const Args& a, MaxSum x, MaxSum y) {
  MaxSum r;
  r.m = x.m > y.m ? x.m : y.m;
  r.s = x.s * exp2f(mul_c(a, x.m - r.m)) + y.s * exp2f(mul_c(a, y.m - r.m));
  return r;
}

__device__ __forceinline__ void block_join(const Args& a, MaxSum& v, MaxSum* lds) {
  for (int o = 32; o; o >>= 1) v = join(a, v, MaxSum{__shfl_xor(v.m, o), __shfl_xor(v.s, o)});
  const int wave = threadIdx.x / 64, waves = blockDim.x / 64;
  __syncthreads();
  if (threadIdx.x % 64 == 0) lds[wave] = v;
  __syncthreads();
  v = lds[0];
  for (int w = 1; w < waves; ++w) v = join(a, v, lds[w]);
}

__device__ __forceinline__ float block_sum(float v, float* lds) {
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  const int wave = threadIdx.x / 64, waves = blockDim.x / 64;
  __syncthreads();
  if (threadIdx.x % 64 == 0) lds[wave] = v;
  __syncthreads();
  v = lds[0];
  for (int w = 1; w < waves; ++w) v += lds[w];
  return v;
}

__device__ __forceinline__ float load_as_float(const void* p, int32_t dtype, uint64_t i) {
  if (dtype == ZERO_F32) return static_cast<const float*>(p)[i];
  if (dtype == ZERO_F16) return (float)static_cast<const _Float16*>(p)[i];
  return (float)static_cast<const __bf16*>(p)[i];
}

// 16 bytes of logits at any element offset.
template <typename T>
struct Pack {
  static constexpr int n = 16 / sizeof(T);
  typedef T vec __attribute__((ext_vector_type(16 / sizeof(T)), aligned(sizeof(T))));
  typedef vec type;
};

template <typename T, bool TAIL, int MODE>
__global__ __launch_bounds__(1024) void k_distill(Args a) {
  extern __shared__ uint32_t lds[];
  __shared__ MaxSum s_ms[16];
  __shared__ float s_f[16];
  __shared__ int s_dup;
  using V = typename Pack<T>::type;
  constexpr int W = Pack<T>::n;
  const zero_distill_in& in = a.in;
  const uint32_t K = (uint32_t)in.topk, vocab = (uint32_t)in.vocab;
  const uint64_t row = blockIdx.x;
  const T* z = static_cast<const T*>(in.logits) + row * in.ld_logits;
  T* dz = static_cast<T*>(a.dlogits) + row * a.ldg;
  const int t = threadIdx.x, nt = blockDim.x;

  const float w = in.weight ? in.weight[row] : 1.0f;
  uint32_t* bits = lds;                                              // [ceil(vocab/32)]
  const uint32_t words = (vocab + 31) / 32;
  int* s_idx = reinterpret_cast<int*>(lds + words);                  // [K] -1: no entry
  float* s_p = reinterpret_cast<float*>(lds + words + K);            // [K]
  float* s_z = reinterpret_cast<float*>(lds + words + 2 * K);        // [K]

  // the teacher's distribution: y_k = t_k c, p_k = 2^(y_k - max) / sum
  float tmax = -INFINITY;
  if (w != 0.0f) {
    for (uint32_t i = t; i < words; i += nt) bits[i] = 0;
    if (t == 0) s_dup = 0;
    for (uint32_t k = t; k < K; k += nt) {
      const uint64_t e = row * in.ld_top + k;
      const int64_t id = in.index_bytes == 8 ? static_cast<const int64_t*>(in.top_index)[e]
                                             : static_cast<const int32_t*>(in.top_index)[e];
      const bool valid = id >= 0 && id < (int64_t)vocab;
      const float y = valid ? load_as_float(in.top_logits, in.teacher_dtype, e) : -INFINITY;
      s_idx[k] = valid ? (int)id : -1;
      s_p[k] = y;
      s_z[k] = valid ? (float)z[id] : -INFINITY;
      tmax = y > tmax || y != y ? y : tmax;
    }
  }
  // tail: log of a mass at temperature T, so it is compared as (tail * T) among the logits; kept
  // apart as its own base-2 exponent
  const float ytail = TAIL && w != 0.0f ? in.tail[row] * 1.44269504088896340736f : -INFINITY;
  for (int o = 32; o; o >>= 1) {
    const float x = __shfl_xor(tmax, o);
    tmax = x > tmax || x != x ? x : tmax;
  }
  __syncthreads();
  if (t % 64 == 0) s_f[t / 64] = tmax;
  __syncthreads();
  for (int i = 0; i < nt / 64; ++i) tmax = s_f[i] > tmax || s_f[i] != s_f[i] ? s_f[i] : tmax;
  if (w == 0.0f || (tmax == -INFINITY && ytail == -INFINITY)) {
    if ((MODE & 1) && t == 0) {
      a.loss[row] = 0.0f;
      if (a.stats) a.stats[2 * row] = a.stats[2 * row + 1] = 0.0f;
    }
    if (MODE & 2)
      for (uint32_t v = t; v < vocab; v += nt) dz[v] = (T)0.0f;
    return;
  }
  // exponents relative to the larger of the listed entries and the tail
  const float listed_over_tail = mul_c(a, tmax) - ytail;  // +inf without a tail
  const bool tail_first = listed_over_tail < 0.0f;
  float tsum = 0.0f;
  for (uint32_t k = t; k < K; k += nt) {
    float y = s_p[k] == -INFINITY ? -INFINITY : mul_c(a, s_p[k] - tmax);
    if (tail_first) y += listed_over_tail;
    s_p[k] = y;
    tsum += exp2f(y);
    if (s_idx[k] >= 0) {
      const uint32_t bit = 1u << (s_idx[k] & 31);
      if (atomicOr(&bits[s_idx[k] >> 5], bit) & bit) s_dup = 1;
    }
  }
  tsum = block_sum(tsum, s_f);
  const float ytail_rel = tail_first ? 0.0f : -listed_over_tail;
  const float etail = TAIL ? exp2f(ytail_rel) : 0.0f;
  tsum += etail;
  const float log_tsum = log2f(tsum), ptail = etail / tsum;
  __syncthreads();

  // the student's (m, s): of every entry, or with a tail of the entries not listed
  MaxSum rest{kLowest, 0.0f};
  if (MODE & 1) {
    const uint32_t body = vocab / W;
    for (uint32_t i = t; i < body; i += nt) {
      const V x = *reinterpret_cast<const V*>(z + (uint64_t)i * W);
      float f[W];
      for (int j = 0; j < W; ++j) f[j] = (float)x[j];
      if (TAIL) {
        const uint32_t mask = bits[i * W / 32] >> (i * W % 32);
        for (int j = 0; j < W; ++j) f[j] = mask >> j & 1 ? -INFINITY : f[j];
      }
      float m = f[0];
      for (int j = 1; j < W; ++j) m = f[j] > m ? f[j] : m;
      if (m > rest.m) {
        rest.s *= exp2f(mul_c(a, rest.m - m));
        rest.m = m;
      }
      float s = 0.0f;
      for (int j = 0; j < W; ++j) s += __builtin_amdgcn_exp2f(mul_s<T>(a, f[j] - rest.m));
      rest.s += s;
    }
    for (uint32_t v = body * W + t; v < vocab; v += nt) {
      float f = (float)z[v];
      if (TAIL && bits[v >> 5] >> (v & 31) & 1) f = -INFINITY;
      if (f > rest.m) {
        rest.s *= exp2f(mul_c(a, rest.m - f));
        rest.m = f;
      }
      rest.s += __builtin_amdgcn_exp2f(mul_s<T>(a, f - rest.m));
    }
    block_join(a, rest, s_ms);
    if (a.stats && t == 0) a.stats[2 * row] = rest.m, a.stats[2 * row + 1] = rest.s;
  } else {
    rest.m = a.stats_in[2 * row], rest.s = a.stats_in[2 * row + 1];
  }

  // Entries listed twice: the first of them (its leader) takes the sum of their p for the
  // gradient and stands for them in the student's mass.
  const bool dup = s_dup;
  MaxSum all = rest;
  if (TAIL) {
    MaxSum top{kLowest, 0.0f};
    for (uint32_t k = t; k < K; k += nt) {
      bool leader = s_idx[k] >= 0;
      if (dup && leader)
        for (uint32_t j = 0; j < k; ++j) leader &= s_idx[j] != s_idx[k];
      if (leader) top = join(a, top, MaxSum{s_z[k] > kLowest ? s_z[k] : kLowest, s_z[k] == -INFINITY ? 0.0f : 1.0f});
      if (s_z[k] != s_z[k]) top.s = s_z[k];
    }
    block_join(a, top, s_ms);
    all = join(a, rest, top);
  }
  const float bad = all.s > 0.0f ? 0.0f : NAN;   // no softmax: NaN, or nothing but -inf
  const float log_s = log2f(all.s) + bad;
  const float qrest = exp2f(mul_c(a, rest.m - all.m)) * rest.s / all.s;

  if (MODE & 1) {
    // in natural logarithms: (z - m)/T stays finite where its base-2 form would overflow
    const float ln_s = kLn2 * log_s;
    float kl = 0.0f;
    for (uint32_t k = t; k < K; k += nt) {
      const float lp = s_p[k] - log_tsum, p = exp2f(lp);
      if (!(p == 0.0f)) kl += p * (kLn2 * lp - ((s_z[k] - all.m) * a.inv_t - ln_s));
    }
    kl = block_sum(kl, s_f);
    if (TAIL && ptail > 0.0f) {
      const float lq = rest.s == 0.0f
                           ? -INFINITY
                           : (rest.m - all.m) * a.inv_t + kLn2 * log2f(rest.s) - ln_s;
      kl += ptail * (kLn2 * (ytail_rel - log_tsum) - lq);
    }
    if (t == 0) a.loss[row] = w * kl + bad;
  }
  if (MODE & 2) {
    const float g = a.scale * (a.upstream ? a.upstream[row] : 1.0f) * w * a.inv_t;
    const float inv = g / all.s;
    const float fout = TAIL ? (rest.s == 0.0f ? bad : g * (qrest - ptail) / rest.s) : inv;
    const float m = rest.m;
    const uint32_t body = vocab / W;
    for (uint32_t i = t; i < body; i += nt) {
      const V x = *reinterpret_cast<const V*>(z + (uint64_t)i * W);
      V y;
      for (int j = 0; j < W; ++j) y[j] = (T)(fout * __builtin_amdgcn_exp2f(mul_s<T>(a, (float)x[j] - m)));
      *reinterpret_cast<V*>(dz + (uint64_t)i * W) = y;
    }
    for (uint32_t v = body * W + t; v < vocab; v += nt)
      dz[v] = (T)(fout * __builtin_amdgcn_exp2f(mul_s<T>(a, (float)z[v] - m)));
    __syncthreads();
    for (uint32_t k = t; k < K; k += nt) {
      bool leader = s_idx[k] >= 0;
      float p = exp2f(s_p[k] - log_tsum);
      if (dup && leader) {
        for (uint32_t j = 0; j < k; ++j) leader &= s_idx[j] != s_idx[k];
        for (uint32_t j = k + 1; j < K && leader; ++j)
          if (s_idx[j] == s_idx[k]) p += exp2f(s_p[j] - log_tsum);
      }
      if (leader) dz[s_idx[k]] = (T)(inv * exp2f(mul_c(a, s_z[k] - all.m)) - g * p + bad);
    }
  }
}

template <typename T, bool TAIL>
hipError_t launch(const Args& a, int mode, hipStream_t s) {
  const uint64_t words = (a.in.vocab + 31) / 32 + 3 * a.in.topk;
  const dim3 grid((unsigned)a.in.rows), block(256);
  const size_t lds = words * 4;
  if (mode == kForward) k_distill<T, TAIL, kForward><<<grid, block, lds, s>>>(a);
  if (mode == kBackward) k_distill<T, TAIL, kBackward><<<grid, block, lds, s>>>(a);
  if (mode == kStep) k_distill<T, TAIL, kStep><<<grid, block, lds, s>>>(a);
  return hipGetLastError();
}

struct Arr {
  const char* name;
  const void* p;
  uint64_t bytes;
  uint32_t align;
  bool written;
};

zero_status run(const char* fn, const zero_distill_in* in, const float* upstream, float scale,
                float* loss, const float* stats_in, float* stats, void* dlogits, uint64_t ldg,
                int mode, void* stream) {
  if (!in) return fail(ZERO_E_INVAL, "%s: in is NULL", fn);
  if (!dtype_valid(in->logit_dtype) || !dtype_valid(in->teacher_dtype))
    return fail(ZERO_E_UNSUPPORTED, "%s: dtypes must be fp32, fp16 or bf16", fn);
  if (in->index_bytes != 4 && in->index_bytes != 8)
    return fail(ZERO_E_INVAL, "%s: index_bytes %d is not 4 or 8", fn, in->index_bytes);
  if (in->vocab == 0 || in->topk == 0) return fail(ZERO_E_INVAL, "%s: vocab or topk is 0", fn);
  if (in->vocab > ZERO_DISTILL_MAX_VOCAB || in->topk > ZERO_DISTILL_MAX_TOPK)
    return fail(ZERO_E_UNSUPPORTED, "%s: vocab %llu or topk %llu above %d and %d", fn,
                (unsigned long long)in->vocab, (unsigned long long)in->topk, ZERO_DISTILL_MAX_VOCAB,
                ZERO_DISTILL_MAX_TOPK);
  if (in->rows > kMaxSize) return fail(ZERO_E_OVERFLOW, "%s: rows above 2^31 - 1", fn);
  if (!(in->temperature >= 0x1p-20f && in->temperature <= 0x1p20f))
    return fail(ZERO_E_INVAL, "%s: temperature must lie in [2^-20, 2^20]", fn);
  if (!isfinite(scale)) return fail(ZERO_E_INVAL, "%s: scale is not finite", fn);
  if (in->rows == 0) return ok();
  if (!in->logits || !in->top_index || !in->top_logits || ((mode & 1) && !loss) ||
      (mode == kForward && !stats) || (mode == kBackward && !stats_in) || ((mode & 2) && !dlogits))
    return fail(ZERO_E_INVAL, "%s: NULL argument", fn);
  const uint64_t rows = in->rows;
  const uint64_t ldl = rows > 1 ? in->ld_logits : in->vocab, ldt = rows > 1 ? in->ld_top : in->topk;
  const uint64_t ldd = rows > 1 ? ldg : in->vocab;
  if (ldl < in->vocab || ldt < in->topk || ((mode & 2) && ldd < in->vocab))
    return fail(ZERO_E_INVAL, "%s: a leading dimension below the columns", fn);
  const uint64_t most = (1ull << 63) / 8 / rows;
  if (ldl >= most || ldt >= most || ((mode & 2) && ldd >= most))
    return fail(ZERO_E_OVERFLOW, "%s: a byte count does not fit in 63 bits", fn);
  const uint32_t le = dtype_bytes(in->logit_dtype), te = dtype_bytes(in->teacher_dtype);
  const Arr arr[] = {
      {"logits", in->logits, ((rows - 1) * ldl + in->vocab) * le, le, false},
      {"top_index", in->top_index, ((rows - 1) * ldt + in->topk) * in->index_bytes,
       (uint32_t)in->index_bytes, false},
      {"top_logits", in->top_logits, ((rows - 1) * ldt + in->topk) * te, te, false},
      {"tail", in->tail, rows * 4, 4, false},
      {"weight", in->weight, rows * 4, 4, false},
      {"upstream", upstream, rows * 4, 4, false},
      {"loss", loss, rows * 4, 4, true},
      {"stats", stats ? stats : stats_in, rows * 8, 4, stats != nullptr},
      {"dlogits", dlogits, ((rows - 1) * ldd + in->vocab) * le, le, true}};
  for (const Arr& x : arr)
    if (x.p && reinterpret_cast<uintptr_t>(x.p) % x.align)
      return fail(ZERO_E_INVAL, "%s: %s is not aligned to its element size", fn, x.name);
  for (const Arr& x : arr)
    for (const Arr& y : arr) {
      if (!x.written || &x == &y || !x.p || !y.p) continue;
      if (&x == &arr[8] && &y == &arr[0] && x.p == y.p && ldd == ldl) continue;  // in place
      if (overlaps(x.p, x.bytes, y.p, y.bytes))
        return fail(ZERO_E_INVAL, "%s: %s overlaps %s", fn, x.name, y.name);
    }

  Args a{};
  a.in = *in;
  a.in.ld_logits = ldl;
  a.in.ld_top = ldt;
  const double c = 1.4426950408889634074 / (double)in->temperature;
  a.c_hi = (float)c;
  a.c_lo = (float)(c - (double)a.c_hi);
  a.inv_t = (float)(1.0 / (double)in->temperature);
  a.stats_in = stats_in;
  a.upstream = upstream;
  a.scale = scale;
  a.loss = loss;
  a.stats = stats;
  a.dlogits = dlogits;
  a.ldg = ldd;
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  hipError_t e;
  const bool tail = in->tail != nullptr;
  switch (in->logit_dtype) {
    case ZERO_F32: e = tail ? launch<float, true>(a, mode, s) : launch<float, false>(a, mode, s); break;
    case ZERO_F16:
      e = tail ? launch<_Float16, true>(a, mode, s) : launch<_Float16, false>(a, mode, s);
      break;
    default: e = tail ? launch<__bf16, true>(a, mode, s) : launch<__bf16, false>(a, mode, s); break;
  }
  if (e != hipSuccess) return fail(ZERO_E_HIP, "%s launch: %s", fn, hipGetErrorString(e));
  return ok();
}

}  // namespace
}  // namespace zero

extern "C" {

zero_status zero_distill_forward(const zero_distill_in* in, float* loss, float* stats, void* stream) {
  return zero::run("zero_distill_forward", in, nullptr, 1.0f, loss, nullptr, stats, nullptr, 0,
                   zero::kForward, stream);
}

zero_status zero_distill_backward(const zero_distill_in* in, const float* stats,
                                  const float* upstream, float scale, void* dlogits,
                                  uint64_t ld_dlogits, void* stream) {
  return zero::run("zero_distill_backward", in, upstream, scale, nullptr, stats, nullptr, dlogits,
                   ld_dlogits, zero::kBackward, stream);
}

zero_status zero_distill_step(const zero_distill_in* in, const float* upstream, float scale,
                              float* loss, void* dlogits, uint64_t ld_dlogits, void* stream) {
  return zero::run("zero_distill_step", in, upstream, scale, loss, nullptr, nullptr, dlogits,
                   ld_dlogits, zero::kStep, stream);
}

}  // extern "C"
