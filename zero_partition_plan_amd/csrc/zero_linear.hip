// The linear layer's entry points: argument checks, the pre-activation gradient and the bias
// gradient. The products themselves are in zero_gemm.hip. ("ZeRO 优化器的三个阶段深度对比", section 三,
// and "ZeRO：把显存“分”着用", ZeRO Stage 3: a gathered layer runs forward, and again for its backward.)
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero_act.h"
#include "zero_internal.h"
#include "zero_linear.h"

namespace zero {
namespace {

constexpr uint64_t kMaxSize = 1u << 27;  // keeps every grid below 2^32 threads a dimension

// dz = round16(dy * act'(pre)), 8 columns a thread, and the bias gradient's partial sums of the
// stored dz: a block takes 256 columns and `chunk` rows, its 8 threads on a column every eighth row,
// joined through LDS in a fixed order. One pass over dy and pre: memory is the bound. Without an
// activation only the sums are formed. 333 x 2304 fp16 with gelu_tanh and its join: 4.3 to 5.1 and 2.0 to 2.9 us (one
// thread a column over all rows took 80).
constexpr int kColsPerBlock = 256, kRowLanes = 8;

template <typename T, int ACT>
__global__ __launch_bounds__(256) void k_dz(const T* dy, uint64_t lddy, const T* pre, uint64_t ldp,
                                            T* dz, uint64_t lddz, uint32_t rows, uint32_t cols,
                                            uint32_t chunk, float* sums, void* db, int db_f32,
                                            int accumulate) {
  typedef T v8 __attribute__((ext_vector_type(8), aligned(2)));
  __shared__ float part[kRowLanes][kColsPerBlock + 4];
  const int cl = threadIdx.x % 32, rl = threadIdx.x / 32;
  const uint32_t c = blockIdx.x * kColsPerBlock + cl * 8;
  const uint64_t first = (uint64_t)blockIdx.y * chunk;
  const uint64_t end = first + chunk < rows ? first + chunk : rows;
  float s[8] = {};
  if (c + 8 <= cols) {
#pragma unroll 2
    for (uint64_t r = first + rl; r < end; r += kRowLanes) {
      v8 d = *reinterpret_cast<const v8*>(dy + r * lddy + c);
      if constexpr (ACT != ZERO_ACT_NONE) {
        const v8 z = *reinterpret_cast<const v8*>(pre + r * ldp + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = (T)((float)d[j] * act_slope<ACT>((float)z[j]));
        *reinterpret_cast<v8*>(dz + r * lddz + c) = d;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += (float)d[j];
    }
  } else {
    for (uint64_t r = first + rl; r < end; r += kRowLanes)
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (c + j < cols) {
          T d = dy[r * lddy + c + j];
          if constexpr (ACT != ZERO_ACT_NONE) {
            d = (T)((float)d * act_slope<ACT>((float)pre[r * ldp + c + j]));
            dz[r * lddz + c + j] = d;
          }
          s[j] += (float)d;
        }
  }
  if (!sums && !db) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) part[rl][cl * 8 + j] = s[j];
  __syncthreads();
  const uint32_t col = blockIdx.x * kColsPerBlock + threadIdx.x;
  if (col >= cols) return;
  float v = 0.0f;
#pragma unroll
  for (int l = 0; l < kRowLanes; ++l) v += part[l][threadIdx.x];
  if (sums) {
    sums[(uint64_t)blockIdx.y * cols + col] = v;
  } else if (db_f32) {  // the only chunk
    float* o = static_cast<float*>(db) + col;
    *o = accumulate ? v + *o : v;
  } else {
    T* o = static_cast<T*>(db) + col;
    *o = (T)(accumulate ? v + (float)*o : v);
  }
}

// dbias from the chunks' sums: 4 threads on a column, every fourth chunk each.
template <typename O>
__global__ __launch_bounds__(256) void k_db(const float* sums, uint32_t chunks, uint32_t cols, O* db,
                                            int accumulate) {
  __shared__ float part[4][64];
  const int cl = threadIdx.x % 64, l = threadIdx.x / 64;
  const uint32_t c = blockIdx.x * 64 + cl;
  float v = 0.0f;
  if (c < cols)
#pragma unroll 4
    for (uint32_t i = l; i < chunks; i += 4) v += sums[(uint64_t)i * cols + c];
  part[l][cl] = v;
  __syncthreads();
  if (l || c >= cols) return;
  v = (part[0][cl] + part[1][cl]) + (part[2][cl] + part[3][cl]);
  if (accumulate) v += (float)db[c];
  db[c] = (O)v;
}

// Row chunks of the pass: enough blocks to fill the card several times, 32 rows a chunk at least where
// there are 24 chunks of that (1000 x 2304 with the join 7.7 us, 9.3 with 8 rows), 8 rows below (333 x 2304 6.3
// us against 7.2, 128 x 4096 5.2 against 6.4), and at most 128 chunks, which the join still reads in a few microseconds.
// A single chunk needs no join: up to 32 rows the join's launch costs more than the chunks save (16 x 2304 3.5
// us in one chunk, 4.9 in two and the join; 64 x 768 6.0 and 5.0).
constexpr uint64_t kOneChunk = 32;
uint32_t dz_chunks(uint64_t rows, uint64_t cols) {
  if (rows <= kOneChunk) return 1;
  const uint64_t groups = (cols + kColsPerBlock - 1) / kColsPerBlock;
  const uint64_t eighths = (rows + 7) / 8 < 24 ? (rows + 7) / 8 : 24;
  uint64_t n = (rows + 31) / 32 > eighths ? (rows + 31) / 32 : eighths;
  const uint64_t most = groups < 16 ? 128 : 2048 / groups;
  if (n > most) n = most ? most : 1;
  return n ? (uint32_t)n : 1u;
}

template <typename T>
hipError_t run_dz(int act, const void* dy, uint64_t lddy, const void* pre, uint64_t ldp, void* dz,
                  uint64_t lddz, uint64_t rows, uint64_t cols, float* sums, void* db, int db_f32, int accumulate,
                  hipStream_t s) {
  const uint32_t chunks = dz_chunks(rows, cols);
  const uint32_t chunk = (uint32_t)((rows + chunks - 1) / chunks);
  const dim3 grid((unsigned)((cols + kColsPerBlock - 1) / kColsPerBlock), chunks);
#define ZERO_DZ(A)                                                                             \
  k_dz<T, A><<<grid, dim3(256), 0, s>>>(static_cast<const T*>(dy), lddy,                       \
                                        static_cast<const T*>(pre), ldp, static_cast<T*>(dz), \
                                        lddz, (uint32_t)rows, (uint32_t)cols, chunk, sums, db, db_f32, accumulate)
  switch (act) {
    case ZERO_ACT_NONE: ZERO_DZ(ZERO_ACT_NONE); break;
    case ZERO_ACT_RELU: ZERO_DZ(ZERO_ACT_RELU); break;
    case ZERO_ACT_GELU: ZERO_DZ(ZERO_ACT_GELU); break;
    case ZERO_ACT_GELU_TANH: ZERO_DZ(ZERO_ACT_GELU_TANH); break;
    default: ZERO_DZ(ZERO_ACT_SILU); break;
  }
#undef ZERO_DZ
  return hipGetLastError();
}

template <typename O>
hipError_t run_db(const float* sums, uint64_t rows, uint64_t cols, void* db, int accumulate,
                  hipStream_t s) {
  k_db<O><<<dim3((unsigned)((cols + 63) / 64)), dim3(256), 0, s>>>(
      sums, dz_chunks(rows, cols), (uint32_t)cols, static_cast<O*>(db), accumulate);
  return hipGetLastError();
}

// Copies a matrix to rows that start on 16 bytes, the columns up to a multiple of 8 filled with zeros.
// Rows off 4 bytes reach the products through registers, in smaller tiles; where a product is large,
// copying first is shorter (4096 x 4097 x 4097 forward 207 us against 254, backward 354 against 600).
// Bound by memory, read and written once.
template <typename T>
__global__ __launch_bounds__(256) void k_pack(const T* src, uint64_t ld, uint32_t rows, uint32_t cols,
                                              T* dst, uint32_t ldd) {
  typedef T v8 __attribute__((ext_vector_type(8)));
  typedef T v8u __attribute__((ext_vector_type(8), aligned(2)));
  const uint32_t c = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (c >= ldd) return;
  for (uint32_t r = blockIdx.y; r < rows; r += gridDim.y) {
    const T* p = src + (uint64_t)r * ld + c;
    v8 v = {};
    if (c + 8 <= cols) {
      v = *reinterpret_cast<const v8u*>(p);
    } else {
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (c + j < cols) v[j] = p[j];
    }
    *reinterpret_cast<v8*>(dst + (uint64_t)r * ldd + c) = v;
  }
}

uint64_t pad8(uint64_t n) { return (n + 7) & ~7ull; }

// Room in the workspace for such copies, in bytes (multiples of 16): of dz, and of x and W (in the backward
// one after the other, so the larger of the two). By sizes alone: rows are off 4 bytes where the features are
// odd (arrays at an odd place besides go through registers; rows on 4 bytes are loaded directly, 4096 x 4100 x
// 4100 forward 178 us against 202 with copies). Zero where the copies would cost more than the 3/4 of
// the product's time they save, at 1.2 PFLOP/s and 3.5 TB/s.
struct Room {
  uint64_t dz, x, w;
};

Room pack_room(uint64_t M, uint64_t K, uint64_t N, bool backward) {
  Room r{0, 0, 0};
  if (!backward && M <= 32) return r;  // taken by a kernel that needs no alignment
  const float product = 2.0f * (float)M * (float)N * (float)K / 1.2e9f;  // us
  const float gain = 0.75f * product * (backward ? 2.0f : 1.0f);
  float cost = 0.0f;
  const bool odd_k = K % 2 != 0, odd_n = backward && N % 2 != 0;
  if (odd_k) cost += 4.0f * (float)K * ((float)M + (float)N) / 3.5e6f + 6.0f;
  if (odd_n) cost += 4.0f * (float)M * (float)N / 3.5e6f + 3.0f;
  if (gain <= cost) return r;
  if (odd_n) r.dz = M * pad8(N) * 2;
  if (odd_k) r.x = M * pad8(K) * 2, r.w = N * pad8(K) * 2;
  return r;
}

bool on16(const void* p, uint64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0; }

// The matrix itself, or its copy at `to` if there is room for one and use.
hipError_t pack(const void*& p, uint64_t& ld, uint64_t rows, uint64_t cols, uint64_t room, char* to,
                hipStream_t s) {
  if (!room || !rows || !cols || on16(p, ld)) return hipSuccess;
  const uint32_t ldd = (uint32_t)pad8(cols);
  const dim3 grid((ldd / 8 + 255) / 256, (unsigned)(rows < 65535 ? rows : 65535));
  k_pack<uint16_t><<<grid, dim3(256), 0, s>>>(static_cast<const uint16_t*>(p), ld, (uint32_t)rows,
                                              (uint32_t)cols, reinterpret_cast<uint16_t*>(to), ldd);
  p = to;
  ld = ldd;
  return hipGetLastError();
}

// One array of a call, as its checks see it.
struct Mat {
  const char* name;
  const void* p;
  uint64_t rows, cols, ld;
  uint32_t eb;
  bool written;

  bool empty() const { return !p || rows == 0 || cols == 0; }
  uint64_t bytes() const { return empty() ? 0 : ((rows - 1) * ld + cols) * eb; }
};

// Whether two arrays share an element. Two matrices of one leading dimension that interleave
// without meeting (column slices of one buffer) do not.
bool meet(const Mat& a, const Mat& b) {
  if (!overlaps(a.p, a.bytes(), b.p, b.bytes())) return false;
  if (a.eb != b.eb || a.rows < 2 || b.rows < 2 || a.ld != b.ld) return true;
  const uintptr_t lo = reinterpret_cast<uintptr_t>(a.p), hi = reinterpret_cast<uintptr_t>(b.p);
  const Mat& first = lo <= hi ? a : b;
  const Mat& second = lo <= hi ? b : a;
  const uint64_t d = lo <= hi ? hi - lo : lo - hi;
  if (d % a.eb) return true;
  const uint64_t q = d / a.eb % a.ld;  // the second's first column in the first's rows
  return q < first.cols || q + second.cols > a.ld;
}

// Shapes and alignment of every array, then that nothing written meets anything else.
// `same[i]` >= 0 names an array that array i may be, element for element.
zero_status check_mats(const char* fn, Mat* m, int count, const int* same0, const int* same1) {
  for (int i = 0; i < count; ++i) {
    if (m[i].empty()) continue;
    if (m[i].rows == 1) m[i].ld = m[i].cols;
    if (m[i].ld < m[i].cols)
      return fail(ZERO_E_INVAL, "%s: %s: leading dimension %llu below its %llu columns", fn, m[i].name,
                  (unsigned long long)m[i].ld, (unsigned long long)m[i].cols);
    uint64_t e;
    if (__builtin_mul_overflow(m[i].rows, m[i].ld, &e) || e >= (1ull << 63) / 8)
      return fail(ZERO_E_OVERFLOW, "%s: %s does not fit in 63 bits", fn, m[i].name);
    if (reinterpret_cast<uintptr_t>(m[i].p) % m[i].eb)
      return fail(ZERO_E_INVAL, "%s: %s is not aligned to its element size", fn, m[i].name);
  }
  for (int i = 0; i < count; ++i) {
    if (!m[i].written || m[i].empty()) continue;
    for (int j = 0; j < count; ++j) {
      if (j == i || m[j].empty() || (m[j].written && j < i)) continue;
      if ((same0[i] == j || same1[i] == j) && m[i].p == m[j].p && m[i].ld == m[j].ld) continue;
      if (meet(m[i], m[j]))
        return fail(ZERO_E_INVAL, "%s: %s overlaps %s", fn, m[i].name, m[j].name);
    }
  }
  return ZERO_OK;
}

// The workspace's first part: partial sums of the products or of the bias gradient, whichever runs.
uint64_t sums_bytes(uint64_t M, uint64_t K, uint64_t N, bool backward) {
  if (!backward) return (gemm_workspace_bytes(M, N, K, false) + 15) & ~15ull;
  const uint64_t dx = gemm_workspace_bytes(M, K, N, true), dw = gemm_workspace_bytes(N, K, M, true);
  const uint64_t db = N * dz_chunks(M, N) * 4;
  const uint64_t most = dx > dw ? dx : dw;
  return ((most > db ? most : db) + 15) & ~15ull;
}

zero_status check_shape(const char* fn, const zero_linear_shape* s) {
  if (!s) return fail(ZERO_E_INVAL, "%s: shape is NULL", fn);
  if (!dtype_valid(s->dtype)) return fail(ZERO_E_INVAL, "%s: unknown dtype %d", fn, s->dtype);
  if (s->dtype == ZERO_F32)
    return fail(ZERO_E_UNSUPPORTED, "%s: dtype must be bf16 or fp16", fn);
  if (s->act < ZERO_ACT_NONE || s->act > ZERO_ACT_SILU)
    return fail(ZERO_E_INVAL, "%s: unknown activation %d", fn, s->act);
  if (s->rows > kMaxSize || s->in_features > kMaxSize || s->out_features > kMaxSize)
    return fail(ZERO_E_OVERFLOW, "%s: a size above 2^27", fn);
  return ZERO_OK;
}

zero_status check_workspace(const char* fn, const zero_linear_shape* s, bool backward, void* ws,
                            uint64_t bytes) {
  const uint64_t need =
      zero_linear_workspace_bytes(s->rows, s->in_features, s->out_features, backward);
  if (need == 0) return ZERO_OK;
  if (!ws || bytes < need)
    return fail(ZERO_E_INVAL, "%s: workspace of %llu bytes, %llu needed", fn,
                (unsigned long long)(ws ? bytes : 0), (unsigned long long)need);
  if (reinterpret_cast<uintptr_t>(ws) % 16)
    return fail(ZERO_E_INVAL, "%s: workspace is not aligned to 16 bytes", fn);
  return ZERO_OK;
}

zero_status hip_result(const char* fn, hipError_t e) {
  if (e != hipSuccess) return fail(ZERO_E_HIP, "%s launch: %s", fn, hipGetErrorString(e));
  return ok();
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" {

uint64_t zero_linear_workspace_bytes(uint64_t rows, uint64_t in_features, uint64_t out_features,
                                     int32_t backward) {
  if (rows > kMaxSize || in_features > kMaxSize || out_features > kMaxSize) return 0;
  const Room r = pack_room(rows, in_features, out_features, backward != 0);
  if (!backward)
    return sums_bytes(rows, in_features, out_features, false) + r.x + r.w;
  return sums_bytes(rows, in_features, out_features, true) + r.dz + (r.x > r.w ? r.x : r.w);
}

zero_status zero_linear_forward(const zero_linear_shape* s, const void* x, uint64_t ldx,
                                const void* weight, const void* bias, const void* residual,
                                uint64_t ldr, void* pre, uint64_t ldp, void* y, uint64_t ldy,
                                void* workspace, uint64_t workspace_bytes, void* stream) {
  const char* fn = "zero_linear_forward";
  if (zero_status st = check_shape(fn, s)) return st;
  const uint64_t M = s->rows, K = s->in_features, N = s->out_features;
  if (M == 0 || N == 0) return ok();
  if (!y) return fail(ZERO_E_INVAL, "%s: y is NULL", fn);
  if (K && (!x || !weight)) return fail(ZERO_E_INVAL, "%s: x or weight is NULL", fn);
  if (zero_status st = check_workspace(fn, s, false, workspace, workspace_bytes)) return st;
  const uint64_t need = zero_linear_workspace_bytes(M, K, N, 0);
  Mat m[] = {{"x", x, M, K, ldx, 2, false},
             {"weight", weight, N, K, K, 2, false},
             {"bias", bias, 1, N, N, 2, false},
             {"residual", residual, M, N, ldr, 2, false},
             {"pre", pre, M, N, ldp, 2, true},
             {"y", y, M, N, ldy, 2, true},
             {"workspace", need ? workspace : nullptr, 1, need, need, 1, true}};
  const int same0[] = {-1, -1, -1, -1, -1, 3, -1}, same1[] = {-1, -1, -1, -1, -1, -1, -1};
  if (zero_status st = check_mats(fn, m, 7, same0, same1)) return st;

  hipStream_t strm = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  GemmArgs g{};
  g.a = x, g.lda = m[0].ld;
  g.b = weight, g.ldb = K;
  const Room room = pack_room(M, K, N, false);
  char* to = static_cast<char*>(workspace) + sums_bytes(M, K, N, false);
  hipError_t e = pack(g.a, g.lda, M, K, room.x, to, strm);
  if (e == hipSuccess) e = pack(g.b, g.ldb, N, K, room.w, to + room.x, strm);
  if (e != hipSuccess) return hip_result(fn, e);
  g.m = (uint32_t)M, g.n = (uint32_t)N, g.k = (uint32_t)K;
  g.dtype = g.out_dtype = s->dtype;
  g.act = s->act;
  g.bias = bias;
  g.res = residual, g.ldr = m[3].ld;
  g.pre = pre, g.ldp = m[4].ld;
  g.out = y, g.ldo = m[5].ld;
  g.ws = static_cast<float*>(workspace);
  return hip_result(fn, gemm(g, strm));
}

zero_status zero_linear_backward(const zero_linear_shape* s, const void* dy, uint64_t lddy,
                                 const void* x, uint64_t ldx, const void* weight, const void* pre,
                                 uint64_t ldp, void* dz, uint64_t lddz, void* dx, uint64_t lddx,
                                 void* dweight, void* dbias, int32_t grad_dtype, int32_t accumulate,
                                 void* workspace, uint64_t workspace_bytes, void* stream) {
  const char* fn = "zero_linear_backward";
  if (zero_status st = check_shape(fn, s)) return st;
  const uint64_t M = s->rows, K = s->in_features, N = s->out_features;
  const bool has_act = s->act != ZERO_ACT_NONE;
  if (!dtype_valid(grad_dtype)) return fail(ZERO_E_INVAL, "%s: unknown grad_dtype %d", fn, grad_dtype);
  if (grad_dtype != s->dtype && grad_dtype != ZERO_F32)
    return fail(ZERO_E_UNSUPPORTED, "%s: grad_dtype must be dtype or fp32", fn);
  if (!has_act) pre = dz = nullptr;
  if (!dz && !dx && !dweight && !dbias && M && N)
    return fail(ZERO_E_INVAL, "%s: no output requested", fn);
  if (M && N) {
    if (!dy) return fail(ZERO_E_INVAL, "%s: dy is NULL", fn);
    if (has_act && (!pre || !dz)) return fail(ZERO_E_INVAL, "%s: pre or dz is NULL", fn);
    if (K && dweight && !x) return fail(ZERO_E_INVAL, "%s: x is NULL", fn);
    if (K && dx && !weight) return fail(ZERO_E_INVAL, "%s: weight is NULL", fn);
  }
  if (zero_status st = check_workspace(fn, s, true, workspace, workspace_bytes)) return st;
  const uint64_t need = zero_linear_workspace_bytes(M, K, N, 1);
  const uint32_t gb = dtype_bytes(grad_dtype);
  Mat m[] = {{"dy", dy, M, N, lddy, 2, false},
             {"x", x, M, K, ldx, 2, false},
             {"weight", weight, N, K, K, 2, false},
             {"pre", pre, M, N, ldp, 2, false},
             {"dz", dz, M, N, lddz, 2, true},
             {"dx", dx, M, K, lddx, 2, true},
             {"dweight", dweight, N, K, K, gb, true},
             {"dbias", dbias, 1, N, N, gb, true},
             {"workspace", need ? workspace : nullptr, 1, need, need, 1, true}};
  const int same0[] = {-1, -1, -1, -1, 0, -1, -1, -1, -1};
  const int same1[] = {-1, -1, -1, -1, 3, -1, -1, -1, -1};
  if (zero_status st = check_mats(fn, m, 9, same0, same1)) return st;

  hipStream_t strm = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  hipError_t e = hipSuccess;
  const bool bf = s->dtype == ZERO_BF16;
  const void* d = dy;
  uint64_t ldd = m[0].ld;
  // the bias gradient's sums are joined before the products use the workspace for theirs
  float* ws = static_cast<float*>(workspace);
  const bool db_wanted = dbias && N && !(M == 0 && accumulate);
  const bool one = dz_chunks(M, N) == 1;
  if ((has_act && M && N) || db_wanted) {
    float* sums = db_wanted && !one ? ws : nullptr;
    void* db = db_wanted && one ? dbias : nullptr;
    const int f32 = grad_dtype == ZERO_F32;
    e = bf ? run_dz<__bf16>(s->act, dy, m[0].ld, pre, m[3].ld, dz, m[4].ld, M, N, sums, db, f32, accumulate, strm)
           : run_dz<_Float16>(s->act, dy, m[0].ld, pre, m[3].ld, dz, m[4].ld, M, N, sums, db, f32, accumulate, strm);
  }
  if (has_act) d = dz, ldd = m[4].ld;
  if (e == hipSuccess && db_wanted && !one) {
    if (grad_dtype == ZERO_F32) e = run_db<float>(ws, M, N, dbias, accumulate, strm);
    else if (bf) e = run_db<__bf16>(ws, M, N, dbias, accumulate, strm);
    else e = run_db<_Float16>(ws, M, N, dbias, accumulate, strm);
  }
  const Room room = pack_room(M, K, N, true);
  char* to = static_cast<char*>(workspace) + sums_bytes(M, K, N, true);
  const bool dx_wanted = dx && M && K, dw_wanted = dweight && N && K && !(M == 0 && accumulate);
  if (e == hipSuccess && (dx_wanted || dw_wanted)) e = pack(d, ldd, M, N, room.dz, to, strm);
  to += room.dz;
  if (e == hipSuccess && dx_wanted) {
    GemmArgs g{};
    g.a = d, g.lda = ldd;
    g.b = weight, g.ldb = K, g.b_kmajor = true;
    e = pack(g.b, g.ldb, N, K, room.w, to, strm);
    if (e != hipSuccess) return hip_result(fn, e);
    g.m = (uint32_t)M, g.n = (uint32_t)K, g.k = (uint32_t)N;
    g.dtype = g.out_dtype = s->dtype;
    g.out = dx, g.ldo = m[5].ld;
    g.ws = ws;
    e = gemm(g, strm);
  }
  if (e == hipSuccess && dw_wanted) {
    GemmArgs g{};
    g.a = d, g.lda = ldd, g.a_kmajor = true;
    g.b = x, g.ldb = m[1].ld, g.b_kmajor = true;
    e = pack(g.b, g.ldb, M, K, room.x, to, strm);
    if (e != hipSuccess) return hip_result(fn, e);
    g.m = (uint32_t)N, g.n = (uint32_t)K, g.k = (uint32_t)M;
    g.dtype = s->dtype, g.out_dtype = grad_dtype;
    g.accumulate = accumulate != 0;
    g.out = dweight, g.ldo = K;
    g.ws = ws;
    e = gemm(g, strm);
  }
  return hip_result(fn, e);
}

}  // extern "C"
