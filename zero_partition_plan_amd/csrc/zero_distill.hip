// Distillation from a teacher's top logits on gfx950: loss, gradient, and both.
//
// One block per row. In base-2 logarithms with c = log2(e)/T, m the row's largest logit and
// s = sum over v of 2^((z_v - m) c):  log2 q_v = (z_v - m) c - log2 s. The first wave looks after the
// teacher's entries while the others sum. With a tail, the sum runs over the entries that are not
// listed only (a bitmap in LDS says which), so that the student's remaining mass comes from a
// sum of its own and not from 1 minus a sum close to 1; the listed entries, at most 1024, are
// joined to it afterwards. The gradient writes F * 2^((z_v - m) c) for every entry and then the
// listed ones over it.
//
// Memory is the bound: the loss alone and the gradient alone read the row once, and the step keeps the
// row in registers between the two, as far as it fits (a row of 131072 16-bit or 65536 fp32 logits);
// longer rows are read twice, the second time mostly from cache. Measured on inputs that change from pass to
// pass, where a large copy reaches 6.1 TB/s and reading alone 7.1: 8192 x 32000 bf16 loss and gradient 204 us (5.1 TB/s),
// 4096 x 50257 bf16 191 us (4.3, its rows lie off 16 bytes), 4096 x 32000 bf16 loss alone 52 us (5.1), 2048 x
// 131072 fp16 loss alone 99 us (5.4), 1024 x 50257 fp32 with a tail 116 us (3.5: rows of 201 kB leave one or two
// to a CU, so loads, arithmetic and stores overlap less), one row of 50257 9.3 us, which is its chain of loads and reductions.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "zero_internal.h"
#include "zero_rows.h"

namespace zero {
namespace {

constexpr uint64_t kMaxSize = 0x7fffffffu;
constexpr uint64_t kGridRows = 1u << 21;
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
// 2^-24 |c d| to its own rounding, seen in the small probabilities of an fp32 gradient. -inf is taken
// as the lowest finite number (c_lo may be negative or 0, and would make a NaN of it); T is at most
// 2^20, so that is still an exponent far below any fp32.
__device__ __forceinline__ float mul_c(const Args& a, float d) {
  d = d < kLowest ? kLowest : d;
  return __builtin_fmaf(d, a.c_hi, d * a.c_lo);
}

// The same inside the pass over the logits. 16-bit logits take the one-term product: their gradient is rounded to
// 16 bits, far above it, and the fp32 loss of such a row is off by at most 2^-24 of the mean of (m - z)/T
// under q, 6e-7 at a mean of 10, about what the roundings of its logarithms are. The two terms cost 8% of the loss
// alone (2048 x 131072 fp16 100.5 us against 93.1) and 2 us of the step on one row (11.4 against 9.4).
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
  r.s = x.s * ex2(mul_c(a, x.m - r.m)) + y.s * ex2(mul_c(a, y.m - r.m));
  return r;
}

// the larger, or a NaN if there is one
__device__ __forceinline__ float larger(float x, float y) { return y > x || y != y ? y : x; }

__device__ __forceinline__ MaxSum wave_join(const Args& a, MaxSum v) {
  const float m = wave_reduce(v.m, kLowest, [](float x, float y) { return x > y ? x : y; });
  return MaxSum{m, wave_sum(v.s * ex2(mul_c(a, v.m - m)))};
}

__device__ __forceinline__ float load_as_float(const void* p, int32_t dtype, uint64_t i) {
  if (dtype == ZERO_F32) return static_cast<const float*>(p)[i];
  if (dtype == ZERO_F16) return (float)static_cast<const _Float16*>(p)[i];
  return (float)static_cast<const __bf16*>(p)[i];
}

// What the first wave leaves for the others.
struct Teacher {
  MaxSum top;       // the listed entries' logits, each index once (tail only)
  float log_sum;    // log2 of the teacher's sum, in the entries' own base-2 exponents s_y
  float log_tail;   // log2 p_tail
  float p_tail;
  int dup;          // some index is listed twice
  int none;         // no teacher mass
};

// An entry of the teacher as it lies in memory.
struct Entry {
  int64_t id;
  float y;
};

__device__ __forceinline__ Entry load_entry(const zero_distill_in& in, uint64_t row, uint32_t k) {
  const uint64_t e = row * in.ld_top + k;
  Entry r;
  r.id = in.index_bytes == 8 ? static_cast<const int64_t*>(in.top_index)[e]
                             : static_cast<const int32_t*>(in.top_index)[e];
  r.y = load_as_float(in.top_logits, in.teacher_dtype, e);
  return r;
}

// The teacher's entries, by one wave (`first`: its lanes' first ones): exponents s_y[k] (-inf: no mass), indices s_idx[k] (-1: no
// entry) and the student's logits there.
template <typename T, bool TAIL>
__device__ __forceinline__ void teach(const Args& a, uint64_t row, Entry first, const T* z, uint32_t* bits,
                                      int* s_idx, float* s_y, float* s_z, Teacher* out) {
  const zero_distill_in& in = a.in;
  const uint32_t K = (uint32_t)in.topk;
  const int lane = threadIdx.x;
  float tmax = -INFINITY;
  for (uint32_t k = lane; k < K; k += 64) {
    const Entry e = k < 64 ? first : load_entry(in, row, k);
    const bool valid = e.id >= 0 && e.id < (int64_t)in.vocab;
    const float y = valid ? e.y : -INFINITY;
    s_idx[k] = valid ? (int)e.id : -1;
    s_y[k] = y;
    s_z[k] = valid ? (float)z[e.id] : -INFINITY;
    tmax = larger(tmax, y);
  }
  tmax = wave_reduce(tmax, -INFINITY, larger);
  // the tail is given as a logarithm at temperature T; exponents are relative to the larger of the
  // listed entries and the tail
  const float ytail = TAIL ? in.tail[row] * 1.44269504088896340736f : -INFINITY;
  const float over = mul_c(a, tmax) - ytail;  // +inf without a tail
  const bool tail_first = over < 0.0f;
  float sum = 0.0f;
  int dup = 0;
  for (uint32_t k = lane; k < K; k += 64) {
    float y = s_y[k] == -INFINITY ? -INFINITY : mul_c(a, s_y[k] - tmax);
    if (tail_first) y += over;
    s_y[k] = y;
    sum += ex2(y);
    if (s_idx[k] >= 0) {
      const uint32_t bit = 1u << (s_idx[k] & 31);
      if (atomicOr(&bits[s_idx[k] >> 5], bit) & bit) dup = 1;
    }
  }
  dup = __any(dup);
  const float y_rel = tail_first ? 0.0f : -over;
  const float e_tail = TAIL ? ex2(y_rel) : 0.0f;
  sum = wave_sum(sum) + e_tail;
  MaxSum top{kLowest, 0.0f};
  if (TAIL) {
    for (uint32_t k = lane; k < K; k += 64) {
      bool leader = s_idx[k] >= 0;  // the first entry of its index
      if (dup && leader)
        for (uint32_t j = 0; j < k; ++j) leader &= s_idx[j] != s_idx[k];
      if (leader)
        top = join(a, top, MaxSum{s_z[k] > kLowest ? s_z[k] : kLowest, s_z[k] == -INFINITY ? 0.0f : 1.0f});
      if (s_z[k] != s_z[k]) top.s = s_z[k];
    }
    top = wave_join(a, top);
  }
  if (lane == 0) {
    out->top = top;
    out->log_sum = log2f(sum);
    out->log_tail = y_rel - log2f(sum);
    out->p_tail = e_tail / sum;
    out->dup = dup;
    out->none = tmax == -INFINITY && ytail == -INFINITY;
  }
}

// Adds n values to a running sum; those whose bit in `skip` is set are left out.
template <typename T, int N>
__device__ __forceinline__ void add(const Args& a, MaxSum& r, float (&f)[N], uint32_t skip) {
  if (skip & ((1u << N) - 1)) {
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = skip >> j & 1 ? -INFINITY : f[j];
  }
  float m = f[0];
#pragma unroll
  for (int j = 1; j < N; ++j) m = f[j] > m ? f[j] : m;
  if (m > r.m) {
    r.s *= ex2(mul_c(a, r.m - m));
    r.m = m;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) r.s += ex2(mul_s<T>(a, f[j] - r.m));
}

// What a row without weight or teacher leaves.
template <int MODE>
__device__ __forceinline__ void no_loss(const Args& a, uint64_t row, int t) {
  if (!(MODE & 1) || t) return;
  a.loss[row] = 0.0f;
  if (a.stats) a.stats[2 * row] = a.stats[2 * row + 1] = 0.0f;
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
template <typename T, bool TAIL, int MODE, int NV, int NT, bool STREAM>
__global__ __launch_bounds__(NT) void k_distill(Args a) {
  extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
  __shared__ MaxSum s_ms[NT / 64];
  __shared__ Teacher teacher;
  using V = typename Pack<T>::type;
  constexpr int W = Pack<T>::n;
  const zero_distill_in& in = a.in;
  const uint32_t K = (uint32_t)in.topk, vocab = (uint32_t)in.vocab;
  const uint64_t row = (uint64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= in.rows) return;
  const T* z = static_cast<const T*>(in.logits) + row * in.ld_logits;
  T* dz = static_cast<T*>(a.dlogits) + row * a.ldg;
  const int t = threadIdx.x, wave = t / 64;
  const uint32_t body = vocab / W;               // whole vectors
  const uint32_t last = body * W + t;            // a thread's element behind them, if < vocab
  const uint32_t words = (vocab + 127) / 128 * 4;
  uint32_t* bits = lds;
  int* s_idx = reinterpret_cast<int*>(lds + words);
  float* s_y = reinterpret_cast<float*>(lds + words + K);
  float* s_z = reinterpret_cast<float*>(lds + words + 2 * K);

  // the weight first, and nothing else of the row if it is 0
  const float w = in.weight ? in.weight[row] : 1.0f;
  if (w == 0.0f) {
    no_loss<MODE>(a, row, t);
    if (MODE & 2) no_gradient<T, NT>(dz, vocab, t);
    return;
  }
  // in the order of need: the teacher's entries, the row
  Entry first{-1, 0.0f};
  if (t < 64 && t < (int)K) first = load_entry(in, row, t);
  V held[NV ? NV : 1];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (i * NT + t < (int)body) held[i] = *reinterpret_cast<const V*>(z + (uint64_t)(i * NT + t) * W);
  for (uint32_t i = t; i < words / 4; i += NT)
    reinterpret_cast<uint4*>(bits)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  if (wave == 0) teach<T, TAIL>(a, row, first, z, bits, s_idx, s_y, s_z, &teacher);
  if (TAIL) __syncthreads();  // the sum needs to know what is listed

  // the student's (m, s): of every entry, or with a tail of the entries not listed
  auto skip = [&](uint32_t i) -> uint32_t {
    return TAIL ? bits[i * W / 32] >> (i * W % 32) : 0;  // W bits from bit 0
  };
  MaxSum rest{kLowest, 0.0f};
  if (MODE & 1) {
    auto one = [&](V x, uint32_t i) {
      float f[W];
#pragma unroll
      for (int j = 0; j < W; ++j) f[j] = (float)x[j];
      add<T, W>(a, rest, f, skip(i));
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
    if (last < vocab) {
      float f[1] = {(float)z[last]};
      add<T, 1>(a, rest, f, TAIL ? bits[last >> 5] >> (last & 31) : 0);
    }
    rest = wave_join(a, rest);
    if ((t & 63) == 0) s_ms[wave] = rest;
  } else {
    rest.m = a.stats_in[2 * row], rest.s = a.stats_in[2 * row + 1];
  }
  __syncthreads();
  if (teacher.none) {
    no_loss<MODE>(a, row, t);
    if (MODE & 2) no_gradient<T, NT>(dz, vocab, t);
    return;
  }
  if (MODE & 1) {
    rest = s_ms[0];
#pragma unroll
    for (int i = 1; i < NT / 64; ++i) rest.m = s_ms[i].m > rest.m ? s_ms[i].m : rest.m;
    rest.s = 0.0f;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) rest.s += s_ms[i].s * ex2(mul_c(a, s_ms[i].m - rest.m));
    if (a.stats && t == 0) a.stats[2 * row] = rest.m, a.stats[2 * row + 1] = rest.s;
  }
  const MaxSum all = TAIL ? join(a, rest, teacher.top) : rest;
  const float bad = all.s > 0.0f ? 0.0f : NAN;   // no softmax: NaN, or nothing but -inf
  const float p_tail = teacher.p_tail;

  if ((MODE & 1) && wave == 0) {
    // in natural logarithms: (z - m)/T stays finite where its base-2 form would overflow
    const float ln_s = kLn2 * (log2f(all.s) + bad);
    float kl = 0.0f;
    for (uint32_t k = t; k < K; k += 64) {
      const float lp = s_y[k] - teacher.log_sum, p = ex2(lp);
      if (!(p == 0.0f)) kl += p * (kLn2 * lp - ((s_z[k] - all.m) * a.inv_t - ln_s));
    }
    kl = wave_sum(kl);
    if (TAIL && !(p_tail == 0.0f)) {
      const float lq = rest.s == 0.0f
                           ? -INFINITY
                           : (rest.m - all.m) * a.inv_t + kLn2 * log2f(rest.s) - ln_s;
      kl += p_tail * (kLn2 * teacher.log_tail - lq);
    }
    if (t == 0) a.loss[row] = w * kl + bad;
  }
  if (MODE & 2) {
    const float g = a.scale * (a.upstream ? a.upstream[row] : 1.0f) * w * a.inv_t;
    const float inv = g / all.s;
    float fout = inv;
    if (TAIL) {
      const float q_rest = ex2(mul_c(a, rest.m - all.m)) * rest.s / all.s;
      fout = rest.s == 0.0f ? bad : g * (q_rest - p_tail) / rest.s;
    }
    const float m = rest.m;
    auto one = [&](V x, uint32_t i) {
      V y;
#pragma unroll
      for (int j = 0; j < W; ++j) y[j] = (T)(fout * ex2(mul_s<T>(a, (float)x[j] - m)));
      if constexpr (STREAM) __builtin_nontemporal_store(y, reinterpret_cast<V*>(dz + (uint64_t)i * W));
      else *reinterpret_cast<V*>(dz + (uint64_t)i * W) = y;
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
    if (last < vocab) dz[last] = (T)(fout * ex2(mul_s<T>(a, (float)z[last] - m)));
    __syncthreads();
    // over the listed entries, one thread per index: entries of one index add their p, in order
    for (uint32_t k = t; k < K; k += NT) {
      bool leader = s_idx[k] >= 0;
      float p = ex2(s_y[k] - teacher.log_sum);
      if (teacher.dup && leader) {
        for (uint32_t j = 0; j < k; ++j) leader &= s_idx[j] != s_idx[k];
        for (uint32_t j = k + 1; j < K && leader; ++j)
          if (s_idx[j] == s_idx[k]) p += ex2(s_y[j] - teacher.log_sum);
      }
      if (leader) dz[s_idx[k]] = (T)(inv * ex2(mul_c(a, s_z[k] - all.m)) - g * p + bad);
    }
  }
}

template <typename T, bool TAIL, int MODE, int NV, int NT>
hipError_t launch_one(const Args& a, hipStream_t s) {
  const size_t lds = ((a.in.vocab + 127) / 128 * 4 + 3 * a.in.topk) * 4;
  // a row a block, over two dimensions, as one holds no more than 2^32 threads
  const uint64_t wide = a.in.rows < kGridRows ? a.in.rows : kGridRows;
  const dim3 grid((unsigned)wide, (unsigned)((a.in.rows + wide - 1) / wide)), block(NT);
  // A gradient of 128 MiB and more would push the logits out of the memory side cache, whether the
  // forward or the head's product left them there (4096 x 32000 bf16 two calls 157 us past the caches,
  // 174 through them); a smaller one stays for whoever reads it next (8192 x 4096 bf16 28 and 26 us).
  if constexpr ((MODE & 2) != 0) {
    if (a.in.rows * a.in.vocab * sizeof(T) >= (128ull << 20)) {
      k_distill<T, TAIL, MODE, NV, NT, true><<<grid, block, lds, s>>>(a);
      return hipGetLastError();
    }
  }
  k_distill<T, TAIL, MODE, NV, NT, false><<<grid, block, lds, s>>>(a);
  return hipGetLastError();
}

template <typename T, bool TAIL>
hipError_t launch(const Args& a, int mode, hipStream_t s) {
  const uint64_t v = a.in.vocab / Pack<T>::n;  // vectors of a row
#define ZERO_GO(MODE, NV, NT) return launch_one<T, TAIL, MODE, NV, NT>(a, s)
  // Few rows: 1024 threads on each, for the latency of one. Many: small blocks, several to a CU, so
  // that one's loads run under another's arithmetic and stores (8192 x 32000 bf16).
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
