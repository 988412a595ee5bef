// The block boundaries' entry points: argument checks, how the backward's rows fall to blocks, and the join
// of the sums over rows. The row kernels are in zero_norm_kernels.hip. ("ZeRO 优化器的三个阶段深度对比", section
// 三: a gathered layer runs forward, and again for its backward.)
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "zero_arrays.h"
#include "zero_norm.h"

namespace zero {
namespace norm {
namespace {

constexpr uint64_t kMaxRows = 1u << 27;

// A sum over rows as the row kernels left it, and where it goes.
struct Sum {
  const float* part;  // [parts of this output row][cols]
  void* out;
  uint64_t ld_out;
  uint32_t outs, parts;  // output rows, and the blocks that hold parts of each
};

struct JoinArgs {
  Sum sum[kSums];
  uint32_t first[kSums];  // each sum's first blockIdx.y
  uint32_t cols;
  int32_t dtype, grad_f32, accumulate;
};

// 64 columns of one output row: 4 threads a column, every fourth part each, joined in a fixed order.
__global__ __launch_bounds__(256) void k_join(JoinArgs a) {
  __shared__ float lds[4][64];
  uint32_t k = 0;
#pragma unroll
  for (uint32_t i = 1; i < kSums; ++i)
    if (a.sum[i].outs && blockIdx.y >= a.first[i]) k = i;
  const Sum s = a.sum[k];
  const uint32_t r = blockIdx.y - a.first[k], l = threadIdx.x / 64;
  const uint32_t c = blockIdx.x * 64 + threadIdx.x % 64;
  float v = 0.0f;
  if (c < a.cols)
#pragma unroll 8
    for (uint32_t i = l; i < s.parts; i += 4) v += s.part[((uint64_t)r * s.parts + i) * a.cols + c];
  lds[l][threadIdx.x % 64] = v;
  __syncthreads();
  if (l || c >= a.cols) return;
  v = (lds[0][threadIdx.x] + lds[1][threadIdx.x]) + (lds[2][threadIdx.x] + lds[3][threadIdx.x]);
  const uint64_t at = (uint64_t)r * s.ld_out + c;
  if (a.grad_f32) {
    float* o = static_cast<float*>(s.out) + at;
    *o = a.accumulate ? *o + v : v;
  } else if (a.dtype == ZERO_BF16) {
    __bf16* o = static_cast<__bf16*>(s.out) + at;
    *o = (__bf16)(a.accumulate ? (float)*o + v : v);
  } else {
    _Float16* o = static_cast<_Float16*>(s.out) + at;
    *o = (_Float16)(a.accumulate ? (float)*o + v : v);
  }
}

// A row's waves hold 8 columns a lane, or 16. About one block for each compute unit, each for as many rows at a time
// as it has waves for. Blocks of 16 waves hide more of the loads' latency, those of 8 leave each lane 256 registers
// in place of 128, which the variants with more sums over rows need (8192 x 4096 bf16 without biases 92 us, 99 in blocks
// of 8 waves; with two layer norms, their biases and a gate 113, 147 in blocks of 16, when that was chosen; 104 by now). Above 8192 columns the sums are
// formed apart.
Plan plan_of(uint64_t rows, uint64_t features, uint64_t segment, bool many) {
  Plan p{};
  const uint64_t vecs = (features + 7) / 8;
  p.apart = vecs > 1024;
  p.threads = p.apart || !many ? 1024 : 512;
  p.vecs = vecs <= p.threads ? 1 : 2;
  p.waves = 1;
  while ((uint64_t)p.waves * 64 * p.vecs < vecs) p.waves *= 2;
  const uint64_t groups = p.threads / 64 / p.waves;
  const uint64_t want = std::max((rows + 255) / 256, groups);  // rows of a block
  p.per = std::min(segment, rows);
  p.segments = (rows + p.per - 1) / p.per;
  if (p.per >= want) {
    p.segs = 1;
    p.chunks = (p.per + want - 1) / want;
    p.chunk = (p.per + p.chunks - 1) / p.chunks;
    p.chunks = (p.per + p.chunk - 1) / p.chunk;
    p.blocks = p.segments * p.chunks;
  } else {
    p.chunks = 1;
    p.chunk = p.per;
    p.segs = want / p.per;
    p.blocks = (p.segments + p.segs - 1) / p.segs;
  }
  return p;
}

uint64_t part_bytes(const Plan& p, uint64_t features) { return (p.blocks * features * 4 + 15) & ~15ull; }

// What k_columns needs of each row, behind the parts.
uint64_t coef_bytes(uint64_t rows, uint64_t features) { return features > 8192 ? (rows * 8 + 15) & ~15ull : 0; }

uint64_t gates_of(const zero_norm_block* b) {
  return b->rows / b->gate_rows + (b->rows % b->gate_rows != 0);
}

zero_status check_block(const char* fn, const zero_norm_block* b) {
  if (!b) return fail(ZERO_E_INVAL, "%s: b is NULL", fn);
  if (!dtype_valid(b->dtype)) return fail(ZERO_E_INVAL, "%s: unknown dtype %d", fn, b->dtype);
  if (b->dtype == ZERO_F32) return fail(ZERO_E_UNSUPPORTED, "%s: dtype must be bf16 or fp16", fn);
  if (b->stream_dtype != b->dtype && b->stream_dtype != ZERO_F32)
    return fail(ZERO_E_UNSUPPORTED, "%s: stream_dtype is neither dtype nor fp32", fn);
  for (int32_t k : {b->post, b->pre})
    if (k < ZERO_NORM_NONE || k > ZERO_NORM_LAYER) return fail(ZERO_E_INVAL, "%s: unknown norm %d", fn, k);
  if (!b->branch && b->pre == ZERO_NORM_NONE && b->rows && b->features)
    return fail(ZERO_E_INVAL, "%s: no branch and no pre norm: nothing to do", fn);
  if (!b->branch && b->rows && b->features && (b->post != ZERO_NORM_NONE || b->gate))
    return fail(ZERO_E_INVAL, "%s: a post norm or a gate without a branch", fn);
  if ((b->post == ZERO_NORM_NONE && (b->post_weight || b->post_bias)) ||
      (b->pre == ZERO_NORM_NONE && (b->pre_weight || b->pre_bias)))
    return fail(ZERO_E_INVAL, "%s: parameters of a norm that is not there", fn);
  if (b->gate && b->gate_rows == 0) return fail(ZERO_E_INVAL, "%s: gate_rows is 0", fn);
  if (!(b->eps >= 0.0f) || !isfinite(b->eps) || !isfinite(b->residual_scale) || !isfinite(b->branch_scale))
    return fail(ZERO_E_INVAL, "%s: eps or a scale is not finite, or eps negative", fn);
  if (b->features > ZERO_NORM_MAX_FEATURES)
    return fail(ZERO_E_UNSUPPORTED, "%s: features above %d", fn, ZERO_NORM_MAX_FEATURES);
  if (b->rows > kMaxRows) return fail(ZERO_E_OVERFLOW, "%s: rows above 2^27", fn);
  return ZERO_OK;
}

// The block's own arrays; leading dimensions of single rows are replaced by the columns.
int block_arrays(zero_norm_block& b, Arr* arr) {
  const uint64_t g = b.gate ? gates_of(&b) : 0;
  if (b.rows < 2) b.ld_branch = b.features;
  if (g < 2) b.ld_gate = b.features;
  arr[0] = Arr{"branch", b.branch, b.rows, b.features, b.ld_branch, 2, false};
  arr[1] = Arr{"gate", b.gate, g, b.features, b.ld_gate, 2, false};
  arr[2] = Arr{"post_weight", b.post_weight, 1, b.features, b.features, 2, false};
  arr[3] = Arr{"post_bias", b.post_bias, 1, b.features, b.features, 2, false};
  arr[4] = Arr{"pre_weight", b.pre_weight, 1, b.features, b.features, 2, false};
  arr[5] = Arr{"pre_bias", b.pre_bias, 1, b.features, b.features, 2, false};
  return 6;
}

zero_status launched(const char* fn, hipError_t e) {
  if (e != hipSuccess) return fail(ZERO_E_HIP, "%s launch: %s", fn, hipGetErrorString(e));
  return ok();
}

}  // namespace
}  // namespace norm
}  // namespace zero

using namespace zero::norm;
using zero::Arr;
using zero::check_arrays;

extern "C" {

zero_status zero_norm_forward(const zero_norm_block* b, const void* x, uint64_t ldx, void* y, uint64_t ldy, void* h,
                              uint64_t ldh, float* stats, void* stream) {
  const char* fn = "zero_norm_forward";
  zero_status st = check_block(fn, b);
  if (st != ZERO_OK) return st;
  const uint64_t R = b->rows, d = b->features;
  if (R == 0 || d == 0) return zero::ok();
  const bool pre = b->pre != ZERO_NORM_NONE;
  if (!x || (b->branch && !y) || (pre && !h)) return zero::fail(ZERO_E_INVAL, "%s: NULL argument", fn);
  ForwardArgs a{};
  a.b = *b;
  Arr arr[10];
  int n = block_arrays(a.b, arr);
  const uint32_t sb = zero::dtype_bytes(b->stream_dtype);
  a.x = x, a.y = b->branch ? y : nullptr, a.h = pre ? h : nullptr, a.stats = stats;
  a.ldx = R > 1 ? ldx : d, a.ldy = R > 1 ? ldy : d, a.ldh = R > 1 ? ldh : d;
  arr[n] = Arr{"x", a.x, R, d, a.ldx, sb, false};
  arr[n + 1] = Arr{"y", a.y, R, d, a.ldy, sb, true};
  arr[n + 2] = Arr{"h", a.h, R, d, a.ldh, 2, true};
  arr[n + 3] = Arr{"stats", a.stats, 1, 4 * R, 4 * R, 4, true};
  st = check_arrays(fn, arr, n + 4, n + 1, n);
  if (st != ZERO_OK) return st;
  a.stream = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  const bool s32 = b->stream_dtype == ZERO_F32;
  hipError_t e;
  if (b->dtype == ZERO_BF16) e = s32 ? launch_forward<ZERO_BF16, true>(a) : launch_forward<ZERO_BF16, false>(a);
  else e = s32 ? launch_forward<ZERO_F16, true>(a) : launch_forward<ZERO_F16, false>(a);
  return launched(fn, e);
}

uint64_t zero_norm_workspace_bytes(uint64_t rows, uint64_t features, uint64_t gate_rows) {
  if (rows == 0 || features == 0 || rows > kMaxRows || features > ZERO_NORM_MAX_FEATURES) return 0;
  // the largest of what a gate shared by gate_rows rows and no shared gate need, with few sums and with many
  uint64_t most = 0;
  for (const uint64_t segment : {gate_rows ? gate_rows : rows, rows})
    for (const bool many : {false, true}) most = std::max(most, part_bytes(plan_of(rows, features, segment, many), features));
  return kSums * most + coef_bytes(rows, features);
}

zero_status zero_norm_backward(const zero_norm_block* b, const float* stats, const void* y, uint64_t ldy, const void* dy,
                               uint64_t lddy, const void* dh, uint64_t lddh, void* dx, uint64_t lddx, void* dbranch,
                               uint64_t lddbranch, void* dgate, uint64_t lddgate, void* dpost_weight, void* dpost_bias,
                               void* dpre_weight, void* dpre_bias, int32_t grad_dtype, int32_t accumulate,
                               void* workspace, uint64_t workspace_bytes, void* stream) {
  const char* fn = "zero_norm_backward";
  zero_status st = check_block(fn, b);
  if (st != ZERO_OK) return st;
  if (!zero::dtype_valid(grad_dtype)) return zero::fail(ZERO_E_INVAL, "%s: unknown grad_dtype %d", fn, grad_dtype);
  if (grad_dtype != b->dtype && grad_dtype != ZERO_F32)
    return zero::fail(ZERO_E_UNSUPPORTED, "%s: grad_dtype is neither dtype nor fp32", fn);
  const uint64_t R = b->rows, d = b->features;
  if (d == 0) return zero::ok();
  const bool pre = b->pre != ZERO_NORM_NONE;
  if (!dx && !dbranch && !dgate && !dpost_weight && !dpost_bias && !dpre_weight && !dpre_bias)
    return zero::fail(ZERO_E_INVAL, "%s: no output requested", fn);
  // (without rows a branch or gate may be NULL, as arrays of length 0)
  if (R && ((dbranch && !b->branch) || (dgate && !b->gate)))
    return zero::fail(ZERO_E_INVAL, "%s: the gradient of a branch or gate that is not there", fn);
  if ((dpost_weight && !b->post_weight) || (dpost_bias && !b->post_bias) || (dpre_weight && !b->pre_weight) ||
      (dpre_bias && !b->pre_bias))
    return zero::fail(ZERO_E_INVAL, "%s: the gradient of a parameter that is not there", fn);
  if (R && (!stats || (pre && (!y || !dh)))) return zero::fail(ZERO_E_INVAL, "%s: NULL argument", fn);
  BackwardArgs a{};
  a.b = *b;
  Arr arr[20];
  int n = block_arrays(a.b, arr);
  const uint64_t gates = arr[1].rows;
  const uint32_t sb = zero::dtype_bytes(b->stream_dtype), gb = zero::dtype_bytes(grad_dtype);
  a.stats = stats, a.y = pre ? y : nullptr, a.dy = dy, a.dh = pre ? dh : nullptr;
  a.dx = dx, a.dbranch = dbranch, a.dgate = dgate;
  a.ldy = R > 1 ? ldy : d, a.lddy = R > 1 ? lddy : d, a.lddh = R > 1 ? lddh : d, a.lddx = R > 1 ? lddx : d;
  a.lddbranch = R > 1 ? lddbranch : d, a.lddgate = gates > 1 ? lddgate : d;
  void* const sums[kSums] = {dpost_weight, dpost_bias, dpre_weight, dpre_bias, dgate};
  const int in = n;
  arr[n++] = Arr{"dy", a.dy, R, d, a.lddy, sb, false};
  arr[n++] = Arr{"dx", a.dx, R, d, a.lddx, sb, true};
  arr[n++] = Arr{"stats", a.stats, R ? 1u : 0u, 4 * R, 4 * R, 4, false};
  arr[n++] = Arr{"y", a.y, R, d, a.ldy, sb, false};
  arr[n++] = Arr{"dh", a.dh, R, d, a.lddh, 2, false};
  arr[n++] = Arr{"dbranch", a.dbranch, R, d, a.lddbranch, 2, true};
  arr[n++] = Arr{"dgate", a.dgate, gates, d, a.lddgate, gb, true};
  arr[n++] = Arr{"dpost_weight", dpost_weight, 1, d, d, gb, true};
  arr[n++] = Arr{"dpost_bias", dpost_bias, 1, d, d, gb, true};
  arr[n++] = Arr{"dpre_weight", dpre_weight, 1, d, d, gb, true};
  arr[n++] = Arr{"dpre_bias", dpre_bias, 1, d, d, gb, true};
  const bool shared = b->gate && gates < R;
  a.wide = b->post == ZERO_NORM_LAYER || b->pre == ZERO_NORM_LAYER || dpost_bias || dpre_bias || (shared && b->post_bias);
  const Plan p = R ? plan_of(R, d, shared ? b->gate_rows : R, a.wide || (b->gate && !shared)) : Plan{};
  a.gate_mode = !b->gate ? 0 : shared ? 1 : 2;
  const bool any_sum =
      dpost_weight || dpost_bias || dpre_weight || dpre_bias || (dgate && shared && (p.chunks > 1 || p.apart));
  const uint64_t need = R && any_sum ? zero_norm_workspace_bytes(R, d, b->gate ? b->gate_rows : R) : 0;
  if (need) {
    if (!workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 16)
      return zero::fail(ZERO_E_INVAL, "%s: workspace of %llu bytes on 16 expected", fn, (unsigned long long)need);
    arr[n++] = Arr{"workspace", workspace, 1, need, need, 1, true};
  }
  st = check_arrays(fn, arr, n, in + 1, in);
  if (st != ZERO_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  a.stream = s;
  a.grad_f32 = grad_dtype == ZERO_F32;
  a.accumulate = accumulate != 0;
  a.plan = p;

  JoinArgs j{};
  j.cols = (uint32_t)d;
  j.dtype = b->dtype, j.grad_f32 = a.grad_f32, j.accumulate = a.accumulate;
  uint32_t outs = 0;
  const uint64_t each = R ? part_bytes(p, d) : 0;
  for (int k = 0; k < kSums; ++k) {
    j.first[k] = outs;
    if (!sums[k]) continue;
    if (k == kGate && (R == 0 || !shared || p.chunks == 1)) continue;  // written by the rows' kernel
    a.part[k] = reinterpret_cast<float*>(static_cast<char*>(workspace) + k * each);
    const uint32_t rows_out = k == kGate ? (uint32_t)p.segments : 1u;
    j.sum[k] = Sum{a.part[k], sums[k], k == kGate ? a.lddgate : d, rows_out,
                   R == 0 ? 0u : (uint32_t)(k == kGate ? p.chunks : p.blocks)};
    outs += rows_out;
  }
  if (need && p.apart) a.coef = reinterpret_cast<float*>(static_cast<char*>(workspace) + kSums * each);
  (void)hipGetLastError();
  hipError_t e = hipSuccess;
  if (R) {
    const bool s32 = b->stream_dtype == ZERO_F32;
    if (b->dtype == ZERO_BF16) e = s32 ? launch_backward<ZERO_BF16, true>(a) : launch_backward<ZERO_BF16, false>(a);
    else e = s32 ? launch_backward<ZERO_F16, true>(a) : launch_backward<ZERO_F16, false>(a);
  }
  if (e == hipSuccess && outs && !(R == 0 && a.accumulate)) {
    k_join<<<dim3((unsigned)((d + 63) / 64), outs), dim3(256), 0, s>>>(j);
    e = hipGetLastError();
  }
  if (R == 0 && !outs) return zero::ok();
  return launched(fn, e);
}

}  // extern "C"
