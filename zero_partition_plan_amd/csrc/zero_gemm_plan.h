// Which tile takes a product, and how its k is split: host arithmetic on sizes alone, without HIP.
#pragma once

#include <math.h>
#include <stdint.h>

namespace zero {

constexpr uint32_t kGemmStep = 64;  // k per LDS stage; splits of k are whole stages

// Tile shapes: number, whether operands off 4 bytes may take it (the largest would spill with operands held in
// registers), rows, columns, waves along the rows, waves along the columns, groups of such waves that share out the k.
#define ZERO_GEMM_SHAPES                  \
  ZERO_SHAPE(0, false, 256, 256, 2, 4, 1) \
  ZERO_SHAPE(1, true, 128, 128, 2, 2, 1)  \
  ZERO_SHAPE(2, true, 64, 256, 1, 4, 1)   \
  ZERO_SHAPE(3, true, 32, 256, 1, 4, 1)   \
  ZERO_SHAPE(4, true, 64, 64, 2, 2, 1)    \
  ZERO_SHAPE(5, false, 256, 192, 2, 4, 1) \
  ZERO_SHAPE(6, false, 192, 256, 2, 4, 1) \
  ZERO_SHAPE(7, true, 64, 64, 2, 2, 2)    \
  ZERO_SHAPE(8, true, 128, 256, 2, 4, 1)

// What a tile of each shape takes, in us on MI355X: besides its steps (start and epilogue) with the
// card almost empty and full, and a step (64 k) with the card almost empty and with `per_cu` tiles on
// every CU. Fitted to products of 16 to 4096 rows, 768 to 50256 columns and k of 16 to 11008:
// tiles of 128 x 128 and less win where there are few, as the part besides the steps is shorter
// (333 x 2304 over k 768: 6.4 us against 20), tiles of 256 x 256 where there are many, as they read
// least (4096 x 11008 over 4096: 281 us against 311), those of 192 where 256 leave CUs idle (2048 x 5120
// over 5120: 87 us against 102), two groups of waves on a tile where few tiles walk a long k (1001 x 768
// over 2304: 15.0 us against 20.6; four groups a tile gain less than 1% more over all). Measured on operands that
// another kernel has just written: a step of few tiles takes up to twice as long there as on warm ones.
// `groups` share a tile's steps, so a step counts once for all of them.
// The last, 128 x 256, is the fastest at no size (of 3 million tried) and stands in where another cannot be launched.
struct TileShape {
  bool held;
  uint32_t bm, bn, per_cu, groups;
  float rest_alone, rest_full, alone, full;
};
constexpr TileShape kShapes[] = {{false, 256, 256, 1, 1, 8.2f, 13.0f, 1.00f, 1.29f}, {true, 128, 128, 2, 1, 5.1f, 5.1f, 0.40f, 0.88f},
                                 {true, 64, 256, 2, 1, 5.2f, 5.2f, 0.46f, 1.00f},    {true, 32, 256, 2, 1, 3.9f, 3.9f, 0.43f, 0.80f},
                                 {true, 64, 64, 5, 1, 3.5f, 3.4f, 0.28f, 0.88f},     {false, 256, 192, 1, 1, 8.4f, 12.0f, 0.74f, 1.00f},
                                 {false, 192, 256, 1, 1, 7.4f, 10.0f, 0.78f, 1.05f}, {true, 64, 64, 2, 2, 3.7f, 3.8f, 0.40f, 0.98f},
                                 {true, 128, 256, 1, 1, 0.0f, 0.0f, 0.0f, 0.0f}};
constexpr int kStandIn = 8;  // those before it are what the plan chooses among
constexpr uint32_t kCus = 256;
constexpr uint64_t kMaxTiles = 1u << 23;  // of at most 512 threads: a grid dimension holds 2^32

struct Plan {
  int shape;
  uint32_t splits, k_split;
};

// The shape and the split of k with the least predicted time. By sizes alone: the workspace must
// not depend on alignment. Every call asks for it, so it tries a dozen splits of each shape and none
// that would only make more rounds of tiles.
inline Plan plan(uint64_t m, uint64_t n, uint64_t k) {
  static const uint32_t kSplits[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32};
  const uint32_t steps = k ? (uint32_t)((k + kGemmStep - 1) / kGemmStep) : 1u;
  Plan best{0, 1, steps * kGemmStep};
  float best_t = 1e30f;
  for (int i = 0; i < kStandIn; ++i) {
    const TileShape& t = kShapes[i];
    const uint64_t tiles = ((m + t.bm - 1) / t.bm) * ((n + t.bn - 1) / t.bn);
    const float slots = (float)(kCus * t.per_cu);
    for (const uint32_t sp : kSplits) {
      if (sp > 1 && (steps / sp < 2 || (float)tiles * (float)sp > 4.0f * slots)) break;
      const uint32_t turns = (steps + sp * t.groups - 1) / (sp * t.groups);  // steps of a group
      const uint32_t per = turns * t.groups, splits = (steps + per - 1) / per;
      const float loads = (float)tiles * (float)splits / slots, rounds = floorf(loads), part = loads - rounds;
      float time = rounds * (t.rest_full + (float)turns * t.full);
      if (part > 0.0f) time += t.rest_alone + (float)turns * (t.alone + (t.full - t.alone) * part);
      // the join's launch, and the partial sums written and read at some 4 TB/s
      if (splits > 1) time += 3.0f + (float)m * (float)n * (float)splits * 8.0f / 4e6f;
      if (time < best_t) {
        best_t = time;
        best = Plan{i, splits, per * kGemmStep};
      }
    }
  }
  return best;
}

// The tile that a planned product runs with, and how many of it there are. Operands that cannot be
// loaded directly, and small tiles of a result of 2^35 elements and more, take the stand-in: with the plan's
// splits, as the workspace was sized by them. False if not even its tiles fit a grid.
inline bool place(uint64_t m, uint64_t n, bool direct, Plan& p, uint64_t& tiles_m, uint64_t& tiles_n) {
  if (!direct && !kShapes[p.shape].held) p.shape = kStandIn;
  for (;;) {
    tiles_m = (m + kShapes[p.shape].bm - 1) / kShapes[p.shape].bm;
    tiles_n = (n + kShapes[p.shape].bn - 1) / kShapes[p.shape].bn;
    if (tiles_m * tiles_n < kMaxTiles) return true;
    if (p.shape == kStandIn) return false;
    p.shape = kStandIn;
  }
}

}  // namespace zero
