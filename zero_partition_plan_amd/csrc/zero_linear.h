// Internal interface between the linear layer's entry points (zero_linear.hip) and the matrix
// product kernels (zero_gemm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero_internal.h"

namespace zero {

// out[i, j] = epilogue(sum_k A(i, k) * B(j, k)) for i < m, j < n.
// Operand element (row, k) lies at row*ld + k, or at k*ld + row when its *_kmajor is set.
struct GemmArgs {
  const void *a, *b;
  uint64_t lda, ldb;
  bool a_kmajor, b_kmajor;
  uint32_t m, n, k;
  int32_t dtype;       // ZERO_BF16 or ZERO_F16: operands, bias, residual, pre
  int32_t out_dtype;   // dtype or ZERO_F32
  int32_t act;         // zero_act
  int32_t accumulate;  // add the old value of out
  const void* bias;    // [n] or NULL
  const void* res;     // [m, n] or NULL
  void* pre;           // [m, n] or NULL
  void* out;           // [m, n]
  uint64_t ldr, ldp, ldo;
  float* ws;           // gemm_workspace_bytes(m, n, k, a_kmajor || b_kmajor)
};

hipError_t gemm(const GemmArgs& g, hipStream_t stream);
uint64_t gemm_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, bool kmajor);

}  // namespace zero
