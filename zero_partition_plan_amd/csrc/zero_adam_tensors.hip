// The AdamW step over many tensors on gfx950, with moments in 32 bits or in 8, and the conversions
// between an 8-bit moment and its numbers. ("ZeRO 优化器的三个阶段深度对比", section 二: a rank updates its own
// parameters with its own state.)
//
// One wave takes 256 consecutive elements of one tensor, 4 a lane, which is also the run that shares a scale
// in an 8-bit moment. The tensors of a launch are a table in the kernel's arguments, so nothing is copied to
// the device and a captured launch holds its own table; a block finds its tensor by halving over the tensors'
// first blocks. Elementwise streaming, bound by memory. The arithmetic is k_adam_step's, every operation
// rounded on its own. Measured: the 148 tensors of GPT-2 small (124M elements, 28 bytes each) 563 us, 6.2 TB/s; the 9 of
// a Llama-7B block (202M, 16 bytes with 8-bit moments) 581, 556 at best, 5.6 to 5.8, where a 2:1 stream reaches 6.0; 48 tensors of
// 7007 elements 6.5, a launch and its chain of loads. That block's codes as numbers 160 us, 6.3 TB/s; numbers as codes 208, 4.9.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <new>

#include "zero_adam.h"
#include "zero_device.h"
#include "zero_internal.h"
#include "zero_rows.h"

namespace zero {
namespace {

constexpr uint32_t kTile = ZERO_STATE8_BLOCK;  // elements of a block: one wave, 4 a lane
constexpr uint32_t kPer = 48;                  // tensors of a launch: the table stays under 4 KiB
constexpr uint64_t kMaxTiles = 1u << 24;       // blocks of a launch

// A tensor, or a run of its tiles, in a launch.
struct Row {
  float* p;
  const void* g;
  void* out;
  void *m, *v;
  float *ms, *vs;
  uint64_t n;
};

struct Launch {
  Row row[kPer];
  zero_adam_scalars sc[ZERO_ADAM_MAX_GROUPS];
  const float* d_gs;               // NULL: gs
  const zero_adam_scalars* table;  // NULL: sc
  const int64_t* d_step;
  const int32_t* skip;
  uint32_t first[kPer];            // each row's first block
  uint32_t count, table_len;
  float gs;
  int32_t out_dtype;
  uint8_t group[kPer];
};
static_assert(sizeof(Launch) <= 4096, "the table is a kernel argument");

// ------------------------------------------------------------------------------------ device side

typedef f32x4 f32x4u __attribute__((aligned(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef u16x4 u16x4u __attribute__((aligned(2)));
typedef uint32_t u32u __attribute__((aligned(1)));

template <int DT>
__device__ __forceinline__ float widen(uint16_t h) {
  if constexpr (DT == ZERO_BF16) return __uint_as_float((uint32_t)h << 16);
  else return (float)__builtin_bit_cast(_Float16, h);
}

__device__ __forceinline__ uint16_t narrow(float x, int32_t dtype) {
  return dtype == ZERO_BF16 ? __builtin_bit_cast(uint16_t, (__bf16)x) : __builtin_bit_cast(uint16_t, (_Float16)x);
}

// The largest of a wave's magnitudes, in every lane, by their bit patterns: for patterns without a sign the order of
// unsigned numbers is that of the values, with a NaN above all.
__device__ __forceinline__ float wave_largest(float v) {
  return wave_reduce(v, 0.0f, [](float x, float y) { return __float_as_uint(y) > __float_as_uint(x) ? y : x; });
}

// What of 4 elements' codes and their block's scale is stored.
struct Coded {
  uint32_t codes;  // 4 bytes, element 0 lowest
  float scale;
};

// 4 elements a lane of one block: T = 127 with a sign, T = 255 without (x = root of the second moment).
// q = ceil(sqrt(t) - 1/2) from the approximate root, taken a little low so that it is q or one less,
// and one exact comparison ((q + 1/2)^2 has at most 18 bits).
template <int T>
__device__ __forceinline__ Coded encode(const float (&x)[4]) {
  constexpr float kSq = (float)(T * T);
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t mag = __float_as_uint(x[j]) & 0x7fffffffu;
    top = mag > top ? mag : top;
  }
  const float s = wave_largest(__uint_as_float(top));
  Coded r{0, s};
  if (!(s >= 0x1p-126f && s < INFINITY)) {  // the same in all lanes
    r.scale = s < 0x1p-126f ? 0.0f : NAN;
    return r;
  }
  const float inv = 1.0f / s;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float t = (fabsf(x[j]) * inv) * kSq;
    float q = ceilf(__builtin_amdgcn_sqrtf(t) - (0.5f + 0x1p-13f));
    const float half = q + 0.5f;
    q = half * half < t ? q + 1.0f : q;
    if (T == 255) q = x[j] > 0.0f && q < 1.0f ? 1.0f : q;
    if (T == 127) q = x[j] < 0.0f ? -q : q;
    r.codes |= ((uint32_t)(int)q & 0xffu) << (8 * j);
  }
  return r;
}

// The values of 4 codes; `unit` = f32(s * f32(1/T^2)).
template <int T>
__device__ __forceinline__ void decode(uint32_t codes, float unit, float (&x)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float q = T == 127 ? (float)(int8_t)(codes >> (8 * j)) : (float)(uint8_t)(codes >> (8 * j));
    x[j] = (q * fabsf(q)) * unit;
  }
}

template <int T>
__device__ __forceinline__ float unit_of(float s) {
  return s * (float)(1.0 / (double)(T * T));
}

__device__ __forceinline__ uint32_t load_codes(const uint8_t* c, int have) {
  if (have == 4) return __builtin_nontemporal_load(reinterpret_cast<const u32u*>(c));
  uint32_t r = 0;
  for (int j = 0; j < have; ++j) r |= (uint32_t)c[j] << (8 * j);
  return r;
}

__device__ __forceinline__ void store_codes(uint8_t* c, uint32_t v, int have) {
  if (have == 4) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32u*>(c));
    return;
  }
  for (int j = 0; j < have; ++j) c[j] = (uint8_t)(v >> (8 * j));
}

// 4 floats of which `have` exist; the others 0.
__device__ __forceinline__ void load4(const float* a, int have, float (&x)[4]) {
  if (have == 4) {
    const f32x4 v = __builtin_nontemporal_load(reinterpret_cast<const f32x4u*>(a));
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = v[j];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = j < have ? a[j] : 0.0f;
  }
}

__device__ __forceinline__ void store4(float* a, int have, const float (&x)[4]) {
  if (have == 4) {
    __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, reinterpret_cast<f32x4u*>(a));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < have) a[j] = x[j];
  }
}

template <int DT>
__device__ __forceinline__ void load_grad(const void* base, uint64_t i, int have, float (&x)[4]) {
  if constexpr (DT == ZERO_F32) {
    load4(static_cast<const float*>(base) + i, have, x);
  } else {
    const uint16_t* a = static_cast<const uint16_t*>(base) + i;
    if (have == 4) {
      const u16x4 v = __builtin_nontemporal_load(reinterpret_cast<const u16x4u*>(a));
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = widen<DT>(v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = j < have ? widen<DT>(a[j]) : 0.0f;
    }
  }
}

// Elements a lane has of n behind element i: 4 but at a tensor's end.
__device__ __forceinline__ int have_of(uint64_t n, uint64_t i) {
  return i + 4 <= n ? 4 : i < n ? (int)(n - i) : 0;
}

template <int GDT, bool S8, bool L2>
__global__ __launch_bounds__(64) void k_tensors(Launch a) {
  if (a.skip != nullptr && *a.skip != 0) return;
  uint32_t e = 0, end = a.count;
  while (end - e > 1) {
    const uint32_t mid = (e + end) / 2;
    if (a.first[mid] <= blockIdx.x) e = mid;
    else end = mid;
  }
  const Row r = a.row[e];
  const uint32_t tile = blockIdx.x - a.first[e];
  const uint64_t i = (uint64_t)tile * kTile + threadIdx.x * 4;
  const int have = have_of(r.n, i);

  float g[4], p[4], m[4], v[4];
  load_grad<GDT>(r.g, i, have, g);
  load4(r.p + i, have, p);
  uint8_t *mc = static_cast<uint8_t*>(r.m) + i, *vc = static_cast<uint8_t*>(r.v) + i;
  float *mf = static_cast<float*>(r.m) + i, *vf = static_cast<float*>(r.v) + i;
  if constexpr (S8) {
    const uint32_t cm = load_codes(mc, have), cv = load_codes(vc, have);
    decode<127>(cm, unit_of<127>(r.ms[tile]), m);
    decode<255>(cv, unit_of<255>(r.vs[tile]), v);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = v[j] * v[j];
  } else {
    load4(mf, have, m);
    load4(vf, have, v);
  }

  zero_adam_scalars s = a.sc[a.group[e]];
  float gs = a.gs;
  if (a.d_gs != nullptr) gs = *a.d_gs;
  if (a.table != nullptr) {
    const int64_t t = *a.d_step;
    if (t < 1 || t > (int64_t)a.table_len) return;  // refused: nothing is written
    s = a.table[(uint64_t)a.group[e] * a.table_len + (t - 1)];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float x = g[j] * gs;
    if (L2) x = x + s.w * p[j];
    m[j] = s.b1 * m[j] + s.c1 * x;
    v[j] = s.b2 * v[j] + s.c2 * (x * x);
    const float root = sqrtf(v[j]);
    const float den = root / s.bc + s.e;
    if (!L2) p[j] = p[j] * s.dec;
    p[j] = p[j] - s.ss * (m[j] / den);
    if (S8) v[j] = root;
  }

  store4(r.p + i, have, p);
  if constexpr (S8) {
    if (have < 4) {  // behind the tensor's end there is no element to count
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j >= have) m[j] = v[j] = 0.0f;
    }
    const Coded cm = encode<127>(m), cv = encode<255>(v);
    store_codes(mc, cm.codes, have);
    store_codes(vc, cv.codes, have);
    if (threadIdx.x == 0) r.ms[tile] = cm.scale, r.vs[tile] = cv.scale;
  } else {
    store4(mf, have, m);
    store4(vf, have, v);
  }
  if (r.out != nullptr) {
    uint16_t* o = static_cast<uint16_t*>(r.out) + i;
    const u16x4 w = {narrow(p[0], a.out_dtype), narrow(p[1], a.out_dtype), narrow(p[2], a.out_dtype),
                     narrow(p[3], a.out_dtype)};
    if (have == 4) {
      __builtin_nontemporal_store(w, reinterpret_cast<u16x4u*>(o));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < have) o[j] = w[j];
    }
  }
}

// Two blocks' codes a wave, both asked for first: the codes are a fifth of the bytes, and one block's are too few in
// flight (202M codes 160 us, one block a wave 194, four 172).
constexpr int kValueTiles = 2;

template <int T>
__global__ __launch_bounds__(64) void k_values(const uint8_t* codes, const float* scale, uint64_t n,
                                               uint64_t first, float* values) {
  uint32_t c[kValueTiles];
  float unit[kValueTiles];
  const uint64_t tile = first + (uint64_t)blockIdx.x * kValueTiles;
#pragma unroll
  for (int u = 0; u < kValueTiles; ++u) {
    const uint64_t i = (tile + u) * kTile + threadIdx.x * 4;
    c[u] = load_codes(codes + i, have_of(n, i));
    unit[u] = unit_of<T>((tile + u) * kTile < n ? scale[tile + u] : 0.0f);
  }
#pragma unroll
  for (int u = 0; u < kValueTiles; ++u) {
    const uint64_t i = (tile + u) * kTile + threadIdx.x * 4;
    float x[4];
    decode<T>(c[u], unit[u], x);
    if (T == 255) {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = x[j] * x[j];
    }
    store4(values + i, have_of(n, i), x);
  }
}

template <int T>
__global__ __launch_bounds__(64) void k_codes(const float* values, uint64_t n, uint64_t first,
                                              uint8_t* codes, float* scale) {
  const uint64_t tile = first + blockIdx.x, i = tile * kTile + threadIdx.x * 4;
  const int have = have_of(n, i);
  float x[4];
  load4(values + i, have, x);
  if (T == 255) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = sqrtf(x[j]);  // NaN below 0
  }
  const Coded c = encode<T>(x);
  store_codes(codes + i, c.codes, have);
  if (threadIdx.x == 0) scale[tile] = c.scale;
}

// -------------------------------------------------------------------------------------- host side

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

uint64_t tiles_of(uint64_t n) { return n / kTile + (n % kTile != 0); }

struct Span {
  uintptr_t begin, end;
  uint32_t id;  // 8 * tensor + array, or a word's
  bool written;
};

constexpr int kArrays = 7;
const char* const kNames[8] = {"param", "grad", "out_param", "m", "v", "m_scale", "v_scale", "a word"};

// No written span may share a byte with another span. Spans of one kind mostly lie in ascending order
// (tensors of a flat space), so they are merged from sorted runs; a run that is not is sorted first.
bool spans_clear(Span* all, const uint32_t* run, int runs, uint32_t* x, uint32_t* y) {
  auto less = [](const Span& p, const Span& q) { return p.begin < q.begin; };
  uint32_t head[kArrays + 1];
  for (int k = 0; k < runs; ++k) {
    head[k] = run[k];
    if (!std::is_sorted(all + run[k], all + run[k + 1], less)) std::sort(all + run[k], all + run[k + 1], less);
  }
  const Span *any = nullptr, *wrote = nullptr;  // those that reach furthest so far
  for (;;) {
    int k = -1;
    for (int j = 0; j < runs; ++j)
      if (head[j] < run[j + 1] && (k < 0 || all[head[j]].begin < all[head[k]].begin)) k = j;
    if (k < 0) return true;
    const Span& s = all[head[k]++];
    const Span* hit = s.written ? any : wrote;
    if (hit && s.begin < hit->end) {
      *x = s.id, *y = hit->id;
      return false;
    }
    if (!any || s.end > any->end) any = &s;
    if (s.written && (!wrote || s.end > wrote->end)) wrote = &s;
  }
}

struct Word {
  const void* p;
  uint64_t bytes;
  bool written;
};

zero_status check_tensors(const char* fn, const zero_adam_tensor* t, uint32_t count, int32_t gdt, int32_t odt,
                          uint32_t ngroups, const Word* words, int nwords) {
  if (ngroups == 0 || ngroups > ZERO_ADAM_MAX_GROUPS)
    return fail(ZERO_E_INVAL, "%s: %u groups, 1 to %d expected", fn, ngroups, ZERO_ADAM_MAX_GROUPS);
  if (count > ZERO_ADAM_MAX_TENSORS)
    return fail(ZERO_E_UNSUPPORTED, "%s: %u tensors, at most %d a call", fn, count, ZERO_ADAM_MAX_TENSORS);
  if (count && !t) return fail(ZERO_E_INVAL, "%s: tensors is NULL", fn);
  if (!dtype_valid(gdt)) return fail(ZERO_E_INVAL, "%s: unknown grad_dtype %d", fn, gdt);
  const uint32_t gb = dtype_bytes(gdt);
  for (uint32_t i = 0; i < count; ++i) {
    const zero_adam_tensor& x = t[i];
    if (x.state_bits != 32 && x.state_bits != 8)
      return fail(ZERO_E_INVAL, "%s: tensor %u: state_bits %u is not 32 or 8", fn, i, x.state_bits);
    if (x.group >= ngroups) return fail(ZERO_E_INVAL, "%s: tensor %u: group %u of %u", fn, i, x.group, ngroups);
    if (x.n == 0) continue;
    if (x.n >= 1ull << 61) return fail(ZERO_E_OVERFLOW, "%s: tensor %u: n*8 does not fit in 64 bits", fn, i);
    const bool eight = x.state_bits == 8;
    if (!x.param || !x.grad || !x.m || !x.v || (eight && (!x.m_scale || !x.v_scale)))
      return fail(ZERO_E_INVAL, "%s: tensor %u: NULL array", fn, i);
    if (!eight && (x.m_scale || x.v_scale))
      return fail(ZERO_E_INVAL, "%s: tensor %u: scales with 32-bit state", fn, i);
    if (x.out_param && odt != ZERO_BF16 && odt != ZERO_F16)
      return fail(odt == ZERO_F32 ? ZERO_E_UNSUPPORTED : ZERO_E_INVAL, "%s: out_param must be bf16 or fp16", fn);
    if (!aligned(x.param, 4) || !aligned(x.grad, gb) || !aligned(x.out_param, 2) || !aligned(x.m_scale, 4) ||
        !aligned(x.v_scale, 4) || (!eight && (!aligned(x.m, 4) || !aligned(x.v, 4))))
      return fail(ZERO_E_INVAL, "%s: tensor %u: an array is not aligned to its elements", fn, i);
  }
  Span* all = new (std::nothrow) Span[(size_t)count * kArrays + nwords + 1];
  if (!all) return fail(ZERO_E_INVAL, "%s: no host memory for the checks of %u tensors", fn, count);
  uint32_t run[kArrays + 2], at = 0;
  for (int k = 0; k < kArrays; ++k) {
    run[k] = at;
    for (uint32_t i = 0; i < count; ++i) {
      const zero_adam_tensor& x = t[i];
      const bool eight = x.state_bits == 8;
      const void* const arr[kArrays] = {x.param, x.grad, x.out_param, x.m, x.v, x.m_scale, x.v_scale};
      const uint64_t sb = eight ? x.n : 4 * x.n;
      const uint64_t bytes[kArrays] = {4 * x.n, gb * x.n, 2 * x.n, sb, sb, 4 * tiles_of(x.n), 4 * tiles_of(x.n)};
      if (x.n == 0 || !arr[k]) continue;
      const uintptr_t b = reinterpret_cast<uintptr_t>(arr[k]);
      all[at++] = Span{b, b + bytes[k], 8 * i + k, k != 1};
    }
  }
  run[kArrays] = at;
  for (int k = 0; k < nwords; ++k) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(words[k].p);
    if (b) all[at++] = Span{b, b + words[k].bytes, 8 * count + 7, words[k].written};
  }
  run[kArrays + 1] = at;
  uint32_t x = 0, y = 0;
  const bool clear = spans_clear(all, run, kArrays + 1, &x, &y);
  delete[] all;
  if (clear) return ZERO_OK;
  return fail(ZERO_E_INVAL, "%s: %s of tensor %u overlaps %s of tensor %u", fn, kNames[x % 8], x / 8, kNames[y % 8],
              y / 8);
}

template <bool S8, bool L2>
void launch_one(const Launch& a, uint32_t blocks, int32_t gdt, hipStream_t s) {
  switch (gdt) {
    case ZERO_F32: k_tensors<ZERO_F32, S8, L2><<<dim3(blocks), dim3(64), 0, s>>>(a); break;
    case ZERO_F16: k_tensors<ZERO_F16, S8, L2><<<dim3(blocks), dim3(64), 0, s>>>(a); break;
    default: k_tensors<ZERO_BF16, S8, L2><<<dim3(blocks), dim3(64), 0, s>>>(a); break;
  }
}

// arguments already checked; `a` holds everything but its rows
hipError_t launch_all(Launch& a, const zero_adam_tensor* t, uint32_t count, int32_t gdt, bool l2, hipStream_t s) {
  const uint32_t gb = dtype_bytes(gdt);
  bool any = false;
  for (const uint32_t bits : {32u, 8u}) {
    uint64_t blocks = 0;
    a.count = 0;
    auto flush = [&]() {
      if (!a.count) return;
      if (!any) (void)hipGetLastError();
      any = true;
      if (bits == 8) l2 ? launch_one<true, true>(a, (uint32_t)blocks, gdt, s) : launch_one<true, false>(a, (uint32_t)blocks, gdt, s);
      else l2 ? launch_one<false, true>(a, (uint32_t)blocks, gdt, s) : launch_one<false, false>(a, (uint32_t)blocks, gdt, s);
      blocks = 0, a.count = 0;
    };
    for (uint32_t i = 0; i < count; ++i) {
      const zero_adam_tensor& x = t[i];
      if (x.state_bits != bits) continue;
      const uint64_t all = tiles_of(x.n), sb = bits / 8;
      for (uint64_t done = 0; done < all;) {  // one row, unless the launch's grid ends inside the tensor
        if (a.count == kPer || blocks == kMaxTiles) flush();
        const uint64_t take = std::min(all - done, kMaxTiles - blocks), e = done * kTile;
        a.row[a.count] = Row{x.param + e,
                             static_cast<const char*>(x.grad) + e * gb,
                             x.out_param ? static_cast<char*>(x.out_param) + 2 * e : nullptr,
                             static_cast<char*>(x.m) + e * sb,
                             static_cast<char*>(x.v) + e * sb,
                             x.m_scale ? x.m_scale + done : nullptr,
                             x.v_scale ? x.v_scale + done : nullptr,
                             std::min(x.n - e, take * kTile)};
        a.first[a.count] = (uint32_t)blocks;
        a.group[a.count] = (uint8_t)x.group;
        ++a.count;
        blocks += take, done += take;
      }
    }
    flush();
  }
  return any ? hipGetLastError() : hipSuccess;
}

zero_status state_args(const char* fn, const void* codes, const float* scale, uint64_t n, int32_t moment,
                       const float* values) {
  if (moment != 1 && moment != 2) return fail(ZERO_E_INVAL, "%s: moment %d is not 1 or 2", fn, moment);
  if (n == 0) return ZERO_OK;
  if (n >= 1ull << 61) return fail(ZERO_E_OVERFLOW, "%s: n*8 does not fit in 64 bits", fn);
  if (!codes || !scale || !values) return fail(ZERO_E_INVAL, "%s: NULL argument", fn);
  if (!aligned(scale, 4) || !aligned(values, 4))
    return fail(ZERO_E_INVAL, "%s: scale or values is not aligned to its elements", fn);
  const uint64_t sb = 4 * tiles_of(n);
  if (overlaps(codes, n, scale, sb) || overlaps(codes, n, values, 4 * n) || overlaps(scale, sb, values, 4 * n))
    return fail(ZERO_E_INVAL, "%s: codes, scale and values overlap", fn);
  return ZERO_OK;
}

}  // namespace
}  // namespace zero

extern "C" {

zero_status zero_adam_tensors_step(const zero_adam_tensor* tensors, uint32_t count, int32_t grad_dtype,
                                   int32_t out_dtype, const zero_adam_hparams* groups, uint32_t ngroups,
                                   float grad_scale, const float* d_grad_scale, const int32_t* d_skip,
                                   void* stream) {
  const char* fn = "zero_adam_tensors_step";
  const zero::Word words[] = {{d_grad_scale, 4, false}, {d_skip, 4, false}};
  zero_status st = zero::check_tensors(fn, tensors, count, grad_dtype, out_dtype, ngroups, words, 2);
  if (st != ZERO_OK) return st;
  if (!groups) return zero::fail(ZERO_E_INVAL, "%s: groups is NULL", fn);
  if (!zero::aligned(d_grad_scale, 4) || !zero::aligned(d_skip, 4))
    return zero::fail(ZERO_E_INVAL, "%s: d_grad_scale or d_skip is not aligned to its element", fn);
  zero::Launch a{};
  for (uint32_t k = 0; k < ngroups; ++k) {
    st = zero_adam_derive(&groups[k], &a.sc[k]);
    if (st != ZERO_OK) return st;
    if (groups[k].wd_mode != groups[0].wd_mode)
      return zero::fail(ZERO_E_INVAL, "%s: groups of different wd_mode", fn);
  }
  a.gs = grad_scale;
  a.d_gs = d_grad_scale;
  a.skip = d_skip;
  a.out_dtype = out_dtype;
  const hipError_t e = zero::launch_all(a, tensors, count, grad_dtype, groups[0].wd_mode == ZERO_ADAM_L2,
                                        static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return zero::fail(ZERO_E_HIP, "%s launch: %s", fn, hipGetErrorString(e));
  return zero::ok();
}

zero_status zero_adam_tensors_step_dev_t(const zero_adam_tensor* tensors, uint32_t count, int32_t grad_dtype,
                                         int32_t out_dtype, const float* d_grad_scale,
                                         const zero_adam_scalars* d_table, uint32_t ngroups,
                                         uint32_t table_len, int64_t* d_step, int32_t* d_status,
                                         int32_t wd_mode, const int32_t* d_skip, void* stream) {
  const char* fn = "zero_adam_tensors_step_dev_t";
  if (!d_grad_scale || !d_table || !d_step || !d_status)
    return zero::fail(ZERO_E_INVAL, "%s: d_grad_scale, d_table, d_step or d_status is NULL", fn);
  if (table_len == 0) return zero::fail(ZERO_E_INVAL, "%s: empty constants table", fn);
  if (wd_mode != ZERO_ADAMW && wd_mode != ZERO_ADAM_L2)
    return zero::fail(ZERO_E_INVAL, "%s: unknown wd_mode %d", fn, wd_mode);
  if (!zero::aligned(d_grad_scale, 4) || !zero::aligned(d_table, 4) || !zero::aligned(d_step, 8) ||
      !zero::aligned(d_status, 4) || !zero::aligned(d_skip, 4))
    return zero::fail(ZERO_E_INVAL, "%s: a device word or the table is not aligned to its elements", fn);
  const uint64_t tb = (uint64_t)ngroups * table_len * sizeof(zero_adam_scalars);
  const zero::Word words[] = {{d_grad_scale, 4, false}, {d_skip, 4, false}, {d_table, tb, false},
                              {d_step, 8, true}, {d_status, 4, true}};
  const zero_status st = zero::check_tensors(fn, tensors, count, grad_dtype, out_dtype, ngroups, words, 5);
  if (st != ZERO_OK) return st;
  zero::Launch a{};
  a.d_gs = d_grad_scale;
  a.table = d_table;
  a.d_step = d_step;
  a.table_len = table_len;
  a.skip = d_skip;
  a.out_dtype = out_dtype;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = zero::launch_all(a, tensors, count, grad_dtype, wd_mode == ZERO_ADAM_L2, s);
  (void)hipGetLastError();
  if (e == hipSuccess) e = zero::step::advance_step(d_step, d_skip, d_status, table_len, s);
  if (e != hipSuccess) return zero::fail(ZERO_E_HIP, "%s launch: %s", fn, hipGetErrorString(e));
  return zero::ok();
}

zero_status zero_adam_state_values(const void* codes, const float* scale, uint64_t n, int32_t moment,
                                   float* values, void* stream) {
  const char* fn = "zero_adam_state_values";
  const zero_status st = zero::state_args(fn, codes, scale, n, moment, values);
  if (st != ZERO_OK) return st;
  if (n == 0) return zero::ok();
  const uint8_t* c = static_cast<const uint8_t*>(codes);
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  for (uint64_t f = 0, all = zero::tiles_of(n); f < all; f += zero::kMaxTiles) {
    const dim3 grid((unsigned)((std::min(all - f, zero::kMaxTiles) + zero::kValueTiles - 1) / zero::kValueTiles));
    if (moment == 1) zero::k_values<127><<<grid, dim3(64), 0, s>>>(c, scale, n, f, values);
    else zero::k_values<255><<<grid, dim3(64), 0, s>>>(c, scale, n, f, values);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return zero::fail(ZERO_E_HIP, "%s launch: %s", fn, hipGetErrorString(e));
  return zero::ok();
}

zero_status zero_adam_state_codes(const float* values, uint64_t n, int32_t moment, void* codes, float* scale,
                                  void* stream) {
  const char* fn = "zero_adam_state_codes";
  const zero_status st = zero::state_args(fn, codes, scale, n, moment, values);
  if (st != ZERO_OK) return st;
  if (n == 0) return zero::ok();
  uint8_t* c = static_cast<uint8_t*>(codes);
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  for (uint64_t f = 0, all = zero::tiles_of(n); f < all; f += zero::kMaxTiles) {
    const dim3 grid((unsigned)std::min(all - f, zero::kMaxTiles));
    if (moment == 1) zero::k_codes<127><<<grid, dim3(64), 0, s>>>(values, n, f, c, scale);
    else zero::k_codes<255><<<grid, dim3(64), 0, s>>>(values, n, f, c, scale);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return zero::fail(ZERO_E_HIP, "%s launch: %s", fn, hipGetErrorString(e));
  return zero::ok();
}

}  // extern "C"
