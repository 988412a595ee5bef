// Internal interface between the block norms' entry points (zero_norm.hip) and their row kernels
// (zero_norm_kernels.hip, compiled once per 16-bit type and stream type).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero_internal.h"

namespace zero {
namespace norm {

struct ForwardArgs {
  zero_norm_block b;
  const void* x;
  void *y, *h;
  uint64_t ldx, ldy, ldh;
  float* stats;
  hipStream_t stream;
};

// How the backward's rows fall to blocks. A block takes `segs` whole segments (rows of one gate row, or all
// rows without a shared gate), or one of the `chunks` parts of a segment.
struct Plan {
  uint32_t waves;   // a row's
  uint32_t vecs;    // groups of 8 columns of a lane: 1 or 2
  uint32_t threads; // a block's
  bool apart;       // the sums over rows by a kernel of their own
  uint64_t segments, segs, chunks, per, chunk;  // per: rows of a segment; chunk: rows of a part
  uint64_t blocks;
};

enum { kPostW, kPostB, kPreW, kPreB, kGate, kSums };  // the sums over rows

struct BackwardArgs {
  zero_norm_block b;
  const float* stats;
  const void *y, *dy, *dh;
  void *dx, *dbranch, *dgate;
  uint64_t ldy, lddy, lddh, lddx, lddbranch, lddgate;
  int32_t grad_f32, accumulate;
  float* part[kSums];  // [blocks, features] each, NULL: not wanted
  int gate_mode;       // 0: none, 1: shared by rows, 2: one a row
  bool wide;           // sums without the normalised values are formed too (a layer norm, a bias's gradient)
  float* coef;         // plan.apart: [rows, 2], what k_columns needs of each row; NULL: nothing
  Plan plan;
  hipStream_t stream;
};

template <int DT, bool S32>
hipError_t launch_forward(const ForwardArgs& a);
template <int DT, bool S32>
hipError_t launch_backward(const BackwardArgs& a);

}  // namespace norm
}  // namespace zero
