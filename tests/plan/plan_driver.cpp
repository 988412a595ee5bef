// Answers a line each. "shapes": every tile shape as the kernels are built and as the plan holds it; otherwise, for "m n k
// direct" on the input, the planned tile, its splits and k a split, whether it can be launched, and the tile
// that then runs. Built by tests/test_linear_plan.py.
#include <stdio.h>

#include "zero_gemm_plan.h"

int main(int argc, char**) {
  if (argc > 1) {
#define ZERO_SHAPE(ID, HELD, BM, BN, WM, WN, G)                                                 \
  printf("%d %d %d %d %d %d %u %u %u %d\n", ID, HELD, BM, BN, G, zero::kShapes[ID].held,           \
         zero::kShapes[ID].bm, zero::kShapes[ID].bn, zero::kShapes[ID].groups, ID == zero::kStandIn);
    ZERO_GEMM_SHAPES
    return 0;
  }
  unsigned long long m, n, k;
  int direct;
  while (scanf("%llu %llu %llu %d", &m, &n, &k, &direct) == 4) {
    const zero::Plan p = zero::plan(m, n, k);
    zero::Plan q = p;
    uint64_t tiles_m, tiles_n;
    const bool fits = zero::place(m, n, direct != 0, q, tiles_m, tiles_n);
    printf("%d %u %u %d %d\n", p.shape, p.splits, p.k_split, fits, q.shape);
  }
  return 0;
}
