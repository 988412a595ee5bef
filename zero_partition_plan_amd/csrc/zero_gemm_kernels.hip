// Tile kernels of the matrix product, for one 16-bit type and one pair of operand orders (set by
// ZERO_GEMM_DT, ZERO_GEMM_AK, ZERO_GEMM_BK when this file is compiled).
//
// out[i, j] = epilogue(sum_k A(i, k) B(j, k)), the sum in fp32 by the 16x16x32 matrix instruction. A
// workgroup takes a tile of out and walks k in stages of 64, two stages in LDS: one is read into
// fragments while the other is loaded, straight from memory to LDS (16 bytes a lane, bounds by the
// buffer descriptor, so ragged edges read zeros). One barrier a stage; the fragments of the next 32
// k are read behind the matrix instructions of these, across the barrier too. A k-contiguous operand is
// read from LDS as it lies, a k-major one (dz and the weight in dz W, both operands of dz^T x) by the transposing
// LDS read, so no operand is ever transposed in memory.
//
// What bounds it is the clock under load and the waits between products: on 8192^3 random bf16 the 256 x 256 tile reaches 1360 to 1420 (x W^T), 1380 to
// 1510 (dz W) and 1440 to 1520 TFLOP/s (dz^T x), from card to card, at 1.5 to
// 1.6 GHz with the matrix units busy in 72, 73 and 78% of the cycles, on zeros 1540 to 1710; hence the instruction with the
// fewest trips of the sums through the matrix unit (the 32x32x16 one: 5 to 9% less), and two stages of
// 64 k rather than more of 32 (a second barrier per 64 k: 14 to 23% less). 8 waves of 128 x 64 sums
// each read LDS conflict-free at half its rate; 4 waves of 128 x 128 would read less but do not fit the registers.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "zero_gemm.h"

#ifndef ZERO_GEMM_DT
#define ZERO_GEMM_DT 2
#define ZERO_GEMM_AK 0
#define ZERO_GEMM_BK 0
#endif

namespace zero {
namespace {

#if ZERO_GEMM_DT == 2
typedef __bf16 T;
#else
typedef _Float16 T;
#endif
constexpr bool kAK = ZERO_GEMM_AK, kBK = ZERO_GEMM_BK;

typedef T t8 __attribute__((ext_vector_type(8)));
typedef T t4 __attribute__((ext_vector_type(4)));
typedef T t8u __attribute__((ext_vector_type(8), aligned(2)));
typedef float f4 __attribute__((ext_vector_type(4)));

constexpr int kStepK = kGemmStep;
constexpr int kStages = 2;  // 3 and 4, where they fit, measured the same

[[maybe_unused]] __device__ __forceinline__ f4 mfma(t8 a, t8 b, f4 c) {
#if ZERO_GEMM_DT == 2
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
#else
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
#endif
}

template <int V>
struct Int {
  static constexpr int value = V;
};

// s_waitcnt for every load into LDS and every LDS access of this wave, and for the LDS accesses alone
[[maybe_unused]] constexpr int kWaitAll = 0x0070, kWaitLds = 0xc07f;

typedef short s4 __attribute__((ext_vector_type(4)));

[[maybe_unused]] __device__ __forceinline__ t4 read_tr(const T* p) {
  typedef __attribute__((address_space(3))) s4 lds_s4;
  const s4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)p);
  return __builtin_bit_cast(t4, v);
}

// One operand's tile of R rows by 64 k in LDS, and how it gets there and into fragments.
// k-contiguous operand: rows of 128 bytes, the 16-byte chunk c of row r at place c ^ (r >> 1 & 7):
// the LDS answers 16 lanes of a 16-byte read at once from 256 bytes of banks, and 16 neighbouring
// rows' chunks of one k then lie in its 16 different places.
// k-major operand: 64 rows of R elements, the 32-byte granule g of row k at place g ^ swz(k): a
// transposing read takes 32 lanes at once, 4 and 4 k (8 apart) of one granule, again in 256 bytes' different places.
template <bool KM, int R, int NT>
struct Tile {
  static constexpr int kChunks = R * kStepK / 8;
  static constexpr int kRounds = kChunks / NT;
  static_assert(kChunks % NT == 0, "whole rounds");
  static constexpr int kElems = R * kStepK;

  static __device__ __forceinline__ int swz(int k) {
    static_assert(R % 128 == 0 || R % 128 == 64 || R == 32, "whole granules, apart in 256 bytes");
    const int half = k >> 3 & 1;
    return R % 128 == 0 ? (k & 3) << 1 | half : R % 64 == 0 ? (k & 2) | half : half;
  }

  // (row, k) of the chunk that lies at place q of the tile
  static __device__ __forceinline__ void chunk_at(int q, int& row, int& k) {
    if constexpr (!KM) {
      row = q / 8;
      k = ((q % 8) ^ (row >> 1 & 7)) * 8;
    } else {
      k = q / (R / 8);
      const int p = q % (R / 8);
      row = (((p >> 1) ^ swz(k)) << 4) + (p & 1) * 8;
    }
  }

  uint32_t voff[kRounds];
  int k0;  // the first k of this thread's chunks (k-contiguous: the same in every round)

  __device__ __forceinline__ void init(uint64_t ld, int tid) {
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      int row, k;
      chunk_at(r * NT + tid, row, k);
      voff[r] = (uint32_t)((KM ? (uint64_t)k * ld + row : (uint64_t)row * ld + k) * 2);
      k0 = k;
    }
  }

  // From the step on whose k end within it (k_left of them): chunks past the end read zeros.
  __device__ __forceinline__ void clip(int k_left) {
    if (KM || k0 < k_left) return;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) voff[r] = 0xfffffff0u;
  }

  // Straight to LDS: `base` is the address of (first row, first k of this step), `bytes` what
  // lies behind it; a load past that gives 0.
  __device__ __forceinline__ void dma(const T* base, uint32_t bytes, T* lds, int wave) const {
    auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(base), 0, bytes, 0x00027000);
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rsrc, (__attribute__((address_space(3))) void*)(lds + (r * NT + wave * 64) * 8), 16,
          voff[r], 0, 0, 0);
  }

  // By way of registers, for operands off the 4 bytes that the direct loads need: chunks at any
  // element, and single elements at the edges.
  t8 held[kRounds];
  __device__ __forceinline__ void fetch(const T* base, uint64_t ld, uint32_t rows_left, int k_left, int tid) {
    // whole steps, which is all but the last: plain loads (rows past the end repeat the last one)
    if (k_left >= kStepK && (!KM || rows_left >= R)) {
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        int row, k;
        chunk_at(r * NT + tid, row, k);
        if (!KM) row = row < (int)rows_left ? row : (int)rows_left - 1;
        held[r] = *reinterpret_cast<const t8u*>(base + (KM ? (uint64_t)k * ld + row : (uint64_t)row * ld + k));
      }
      return;
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      int row, k;
      chunk_at(r * NT + tid, row, k);
      const T* p = base + (KM ? (uint64_t)k * ld + row : (uint64_t)row * ld + k);
      const int have = KM ? (k < k_left ? (int)rows_left - row : 0)
                          : (row < (int)rows_left ? k_left - k : 0);
      if (have >= 8) {
        held[r] = *reinterpret_cast<const t8u*>(p);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) held[r][j] = j < have ? p[j] : (T)0.0f;
      }
    }
  }
  __device__ __forceinline__ void put(T* lds, int tid) const {
#pragma unroll
    for (int r = 0; r < kRounds; ++r) *reinterpret_cast<t8*>(lds + (r * NT + tid) * 8) = held[r];
  }

  // Fragment for 16 rows from row0 and 32 k from kk*32, read from LDS.
  static __device__ __forceinline__ t8 frag(const T* lds, int row0, int kk, int lane) {
    if constexpr (!KM) {
      const int row = row0 + (lane & 15);
      const int c = (kk * 4 + (lane >> 4)) ^ (lane >> 1 & 7);
      return *reinterpret_cast<const t8*>(lds + row * kStepK + c * 8);
    } else {
      const int i = lane & 15;
      const int k = kk * 32 + (lane >> 4) * 8 + (i >> 2);
      const T* p = lds + k * R + (((row0 >> 4) ^ swz(k)) << 4) + (i & 3) * 4;
      const t4 lo = read_tr(p), hi = read_tr(p + 4 * R);
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// Stages of one operand lie side by side, A's before B's: the reads of both stages are then
// immediate offsets from the same addresses.
template <int BM, int BN, int WM, int WN>
struct Shape {
  static constexpr int NT = WM * WN * 64;
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
  using A = Tile<kAK, BM, NT>;
  using B = Tile<kBK, BN, NT>;
  static constexpr int kB = kStages * A::kElems;
  static constexpr int kElems = kB + kStages * B::kElems;
};

template <typename S>
struct Frags {
  t8 a[S::TM], b[S::TN];
};

// The products of the fragments in hand, 32 k, and in their places those of the 32 k after: a row
// fragment is read again as soon as its products are issued, so one set of them is enough; the
// column fragments, used to the end, take a second set.
template <typename S>
__device__ __forceinline__ void half(const T* sa, const T* sb, int kk, Frags<S>& f, f4 (&acc)[S::TM][S::TN],
                                     int wm0, int wn0, int lane) {
  t8 b[S::TN];
#pragma unroll
  for (int i = 0; i < S::TM; ++i) {
#pragma unroll
    for (int j = 0; j < S::TN; ++j) acc[i][j] = mfma(f.b[j], f.a[i], acc[i][j]);
    f.a[i] = S::A::frag(sa, wm0 + i * 16, kk, lane);
#pragma unroll
    for (int j = i * S::TN / S::TM; j < (i + 1) * S::TN / S::TM; ++j)
      b[j] = S::B::frag(sb, wn0 + j * 16, kk, lane);
  }
#pragma unroll
  for (int j = 0; j < S::TN; ++j) f.b[j] = b[j];
}

// From the second half of one step to the first of the next. On entry f holds the last
// fragments of the stage at da and db, which no wave reads any more: the loads of the step after
// the next go there, while the products run through the stage at sa and sb. The stages are declared
// apart, so that the reads of one need not wait for what is on its way into the other.
template <typename S, bool DIRECT>
__device__ __forceinline__ void step(const T* __restrict__ sa, const T* __restrict__ sb,
                                     T* __restrict__ da, T* __restrict__ db, const typename S::A& ta,
                                     const typename S::B& tb, const T* pa, uint32_t abytes, const T* pb,
                                     uint32_t bbytes, Frags<S>& f, f4 (&acc)[S::TM][S::TN],
                                     int wm0, int wn0, int wave, int lane) {
  if (DIRECT) {
    ta.dma(pa, abytes, da, wave);
    tb.dma(pb, bbytes, db, wave);
  }
  half<S>(sa, sb, 0, f, acc, wm0, wn0, lane);
  half<S>(sa, sb, 1, f, acc, wm0, wn0, lane);
  // behind each row of matrix instructions its share of the LDS reads, and of the loads
  constexpr int reads = (S::TM * (kAK ? 2 : 1) + S::TN * (kBK ? 2 : 1) + S::TM - 1) / S::TM;
  constexpr int loads = (S::A::kRounds + S::B::kRounds + S::TM - 1) / S::TM;
#pragma unroll
  for (int i = 0; i < S::TM; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x8, S::TN, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, reads, 0);
    __builtin_amdgcn_sched_group_barrier(0x20, loads, 0);
  }
#pragma unroll
  for (int i = 0; i < S::TM; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x8, S::TN, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, reads, 0);
  }
}

// G groups of waves take the k steps of a tile between them, each with stages of its own, and are
// joined through LDS in their order: where there are few tiles, the time is the chain of their steps.
template <typename S, bool DIRECT, int BM, int BN, int WM, int WN, int G>
__global__ __launch_bounds__(WM* WN * 64 * G, 2) void k_gemm(GemmDev g) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host's pass has no use for the body
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int group = G == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / S::NT);
  T* lds = reinterpret_cast<T*>(smem) + group * S::kElems;
  const int tid = G == 1 ? threadIdx.x : threadIdx.x % S::NT, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  uint32_t mt, nt;
  tile_of(g, blockIdx.x, mt, nt);
  const uint32_t m0 = mt * BM, n0 = nt * BN;
  const uint32_t k_begin = blockIdx.y * g.k_split;
  const uint32_t k_end = k_begin + g.k_split < g.k ? k_begin + g.k_split : g.k;
  const int wm0 = (wave / WN) * (BM / WM), wn0 = (wave % WN) * (BN / WN);

  typename S::A ta;
  typename S::B tb;
  if (DIRECT) {
    ta.init(g.lda, tid);
    tb.init(g.ldb, tid);
  }
  // steps of the workgroup, and of each of its groups: a split that is not the last has a multiple of G, and
  // what lies past the last one's end reads zeros
  const int all = (int)((k_end - k_begin + kStepK - 1) / kStepK);
  const int steps = (all + G - 1) / G;
  const uint32_t k_first = k_begin + (uint32_t)(group * steps) * kStepK;
  Cursor<T, kAK, BM> ca(g.a, g.lda, m0, g.m, k_first);
  Cursor<T, kBK, BN> cb(g.b, g.ldb, n0, g.n, k_first);

  f4 acc[S::TM][S::TN] = {};
  int k_left = (int)g.k - (int)k_first;
  // k's last, partial chunk of a k-contiguous row comes with what lies behind the row
  const int part = DIRECT && k_end == g.k && (!kAK || !kBK) ? (int)(g.k & 7) : 0;
  const int k_last = (int)(k_end - k_begin) - (all - 1) * kStepK;
  // the group and the step of that chunk
  const int g_last = G == 1 || !all ? 0 : (all - 1) / steps, s_last = all - 1 - g_last * steps;
  Frags<S> f = {};
  if (DIRECT) {
    if (k_left < kStepK) ta.clip(k_left), tb.clip(k_left);
    ta.dma(ca.p, ca.bytes(k_left), lds, wave);
    tb.dma(cb.p, cb.bytes(k_left), lds + S::kB, wave);
  } else {
    ta.fetch(ca.p, g.lda, g.m - m0, k_left, tid);
    tb.fetch(cb.p, g.ldb, g.n - n0, k_left, tid);
    ta.put(lds, tid);
    tb.put(lds + S::kB, tid);
  }
  // Held operands run two steps ahead: a step first puts what was asked for during the one before into
  // the free stage, and asks for the next.
  auto next = [&]() __attribute__((always_inline)) {
    ca.advance();
    cb.advance();
    k_left -= kStepK;
  };
  auto fetch = [&]() __attribute__((always_inline)) {
    ta.fetch(ca.p, g.lda, g.m - m0, k_left, tid);
    tb.fetch(cb.p, g.ldb, g.n - n0, k_left, tid);
  };
  if (!DIRECT) {
    next();
    fetch();
  }
  auto body = [&](auto place, bool last) __attribute__((always_inline)) {
    constexpr int P = decltype(place)::value, D = 1 - P;
    T *sa = lds + P * S::A::kElems, *sb = lds + S::kB + P * S::B::kElems;
    T *da = lds + D * S::A::kElems, *db = lds + S::kB + D * S::B::kElems;
    if (DIRECT) next();
    const uint32_t abytes = ca.bytes(k_left), bbytes = cb.bytes(k_left);
    if (DIRECT && k_left < kStepK) ta.clip(k_left), tb.clip(k_left);
    // what the next stage needs has landed, and this wave's reads of the stage that is to be loaded
    // over are done: the barrier makes both true of all waves
    __builtin_amdgcn_s_waitcnt(DIRECT ? kWaitAll : kWaitLds);
    __syncthreads();
    if (part && last) {
      if (G == 1 || group == g_last) {
        zero_partial<T, kAK, BM>(sa, k_last, tid, S::NT);
        zero_partial<T, kBK, BN>(sb, k_last, tid, S::NT);
      }
      __syncthreads();
    }
    if (!DIRECT) {
      ta.put(da, tid);
      tb.put(db, tid);
      next();
      fetch();
    }
    step<S, DIRECT>(sa, sb, da, db, ta, tb, ca.p, abytes, cb.p, bbytes, f, acc, wm0, wn0, wave, lane);
  };
  for (int s = 0; s < steps; s += 2) {
    body(Int<0>{}, s == s_last);
    if (s + 1 < steps) body(Int<1>{}, s + 1 == s_last);
  }
#pragma unroll
  for (int i = 0; i < S::TM; ++i)
#pragma unroll
    for (int j = 0; j < S::TN; ++j) acc[i][j] = mfma(f.b[j], f.a[i], acc[i][j]);
  __builtin_amdgcn_s_waitcnt(kWaitAll);  // the last step's loads past the end land before LDS is reused
  __syncthreads();
  // 32 rows at a time through LDS: the matrix instruction leaves a lane 4 neighbouring columns of
  // one row; the epilogue wants 8 columns a lane, and a row's lanes side by side. One copy of its
  // code for all (it would be the larger part of the kernel, fetched cold by every launch).
  constexpr int kRow = S::TN * 16 + 4;
  constexpr int kLanes = S::TN * 16 / 8;  // lanes on a row
  float* stage = reinterpret_cast<float*>(smem) + (group * (WM * WN) + wave) * (32 * kRow);
  if constexpr (G > 1) {
    static_assert(S::TM == 2 && 64 / kLanes >= 32 / G, "one turn");
#pragma unroll
    for (int c = 0; c < S::TM; ++c)
#pragma unroll
      for (int j = 0; j < S::TN; ++j)
        *reinterpret_cast<f4*>(stage + (c * 16 + (lane & 15)) * kRow + j * 16 + (lane >> 4) * 4) = acc[c][j];
    __syncthreads();
    // each group finishes its share of the rows
    const int r = group * (32 / G) + lane / kLanes, col = (lane % kLanes) * 8;
    const uint32_t m = m0 + wm0 + r, n = n0 + wn0 + col;
    if (lane / kLanes < 32 / G && m < g.m && n < g.n) {
      const float* at = reinterpret_cast<const float*>(smem) + wave * (32 * kRow) + r * kRow + col;
      float z[1][8] = {};
#pragma unroll
      for (int h = 0; h < G; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j) z[0][j] += at[h * (WM * WN * 32 * kRow) + j];
      if (g.splits > 1) keep_rows<1>(g, z, m, 1, g.m, n);
      else finish_row<T>(g, z, m, n);
    }
    return;
  }
#pragma unroll 1
  for (int i = 0; i < S::TM / 2; ++i) {
#pragma unroll
    for (int c = 0; c < S::TM; ++c)
      if (c / 2 == i) {
#pragma unroll
        for (int j = 0; j < S::TN; ++j)
          *reinterpret_cast<f4*>(stage + (c % 2 * 16 + (lane & 15)) * kRow + j * 16 + (lane >> 4) * 4) = acc[c][j];
      }
    __builtin_amdgcn_wave_barrier();
    // two rows of a lane at a time: more in flight would spill the 256 x 256 tile's sums
    constexpr int kPer = 64 / kLanes, R = 2;
    const uint32_t first = m0 + wm0 + i * 32, m_end = first + 32 < g.m ? first + 32 : g.m;
#pragma unroll 1
    for (int r0 = lane / kLanes; r0 < (64 % kLanes && lane >= kPer * kLanes ? 0 : 32); r0 += R * kPer) {
      const uint32_t m = first + r0, n = n0 + wn0 + (lane % kLanes) * 8;
      const float* at = stage + r0 * kRow + (lane % kLanes) * 8;
      float z[R][8];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        *reinterpret_cast<float4*>(&z[r][0]) = *reinterpret_cast<const float4*>(at + r * kPer * kRow);
        *reinterpret_cast<float4*>(&z[r][4]) = *reinterpret_cast<const float4*>(at + r * kPer * kRow + 4);
      }
      if (m >= m_end || n >= g.n) continue;
      if (g.splits > 1) {
        keep_rows<R>(g, z, m, kPer, m_end, n);
      } else if (n + 8 <= g.n) {
        finish_rows<T, R>(g, z, m, kPer, m_end, n);
      } else {
#pragma unroll 1
        for (int r = 0; r < R; ++r)
#pragma unroll 1
          for (int j = 0; n + j < g.n; ++j)
            if (m + r * kPer < m_end) finish_one<T>(g, at[r * kPer * kRow + j], m + r * kPer, n + j);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
#endif
}

template <bool DIRECT, int BM, int BN, int WM, int WN, int G>
hipError_t launch(const GemmDev& g, hipStream_t s) {
  using S = Shape<BM, BN, WM, WN>;
  constexpr int epi = WM * WN * 32 * (S::TN * 16 + 4) * 4;
  constexpr int lds = G * (S::kElems * 2 > epi ? S::kElems * 2 : epi);
  auto fn = k_gemm<S, DIRECT, BM, BN, WM, WN, G>;
  if (lds > 64 * 1024) {
    static std::atomic<uint64_t> allowed{0};  // one bit a device
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(allowed.load(std::memory_order_relaxed) & bit)) {
      e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
      if (e != hipSuccess) return e;
      allowed.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  fn<<<dim3(g.tiles_m * g.tiles_n, g.splits), dim3(S::NT * G), lds, s>>>(g);
  return hipGetLastError();
}

}  // namespace

#define ZERO_CAT_(a, b, c, d) a##b##c##d
#define ZERO_CAT(a, b, c, d) ZERO_CAT_(a, b, c, d)
hipError_t ZERO_CAT(gemm_tiles_, ZERO_GEMM_DT, ZERO_GEMM_AK, ZERO_GEMM_BK)(const GemmDev& g, int shape,
                                                                           bool direct, hipStream_t s) {
  // `held`: whether there is a kernel for operands that go through registers; the largest tiles would
  // spill with them
#define ZERO_SHAPE(id, held, ...) \
  case id: return direct ? launch<true, __VA_ARGS__>(g, s) : launch<!held, __VA_ARGS__>(g, s);
  switch (shape) {
    ZERO_GEMM_SHAPES
    default: return hipErrorInvalidValue;
  }
#undef ZERO_SHAPE
}

}  // namespace zero
