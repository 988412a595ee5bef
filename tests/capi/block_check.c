/* The update of many tensors, the block boundary and the policy loss from plain C on the GPU, through the C ABI only. One
 * tensor with 32-bit moments against zero_host_adam_step, bit for bit, and one with 8-bit moments whose parameters after a
 * first step (moments of value 0) must be the same bits; a boundary without norms but an RMS pre norm against the
 * host's double evaluation, stored values within half a bf16 step of it (and 1e-4 for the fp32 sums); the policy loss of
 * each row's token in one pass and in two calls against the host's, within 1e-4 of numbers of size 10; and what the
 * calls refuse. Exits 0 when all hold. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <hip/hip_runtime_api.h>

#include "zero_shard.h"

#define N 1000u
#define BLOCKS 4u
#define ROWS 30u
#define D 97u
#define VOCAB 333u

#define HIP(x)                                                                  \
  do {                                                                          \
    hipError_t e_ = (x);                                                        \
    if (e_ != hipSuccess) {                                                     \
      fprintf(stderr, "%s:%d: %s\n", __FILE__, __LINE__, hipGetErrorString(e_)); \
      return 2;                                                                 \
    }                                                                           \
  } while (0)
#define ZS(x)                                                                        \
  do {                                                                               \
    zero_status s_ = (x);                                                            \
    if (s_ != ZERO_OK) {                                                             \
      fprintf(stderr, "%s:%d: %s: %s\n", __FILE__, __LINE__, zero_status_str(s_),   \
              zero_last_error());                                                    \
      return 2;                                                                      \
    }                                                                                \
  } while (0)
#define HOLDS(x)                                               \
  do {                                                         \
    if (!(x)) {                                                \
      fprintf(stderr, "%s:%d: not %s\n", __FILE__, __LINE__, #x); \
      return 3;                                                \
    }                                                          \
  } while (0)

static uint64_t state = 0x9e3779b97f4a7c15ull;
static float draw(void) { /* -1 to 1 */
  state = state * 6364136223846793005ull + 1442695040888963407ull;
  return (float)((int32_t)(state >> 33) - (1 << 30)) / (float)(1 << 30);
}

static uint16_t to16(float x) { /* bf16, to nearest even */
  uint32_t u;
  memcpy(&u, &x, 4);
  return (uint16_t)((u + 0x7fffu + (u >> 16 & 1)) >> 16);
}

static float from16(uint16_t h) {
  uint32_t u = (uint32_t)h << 16;
  float x;
  memcpy(&x, &u, 4);
  return x;
}

static void* up(const void* host, size_t bytes) { /* NULL: zeros */
  void* d = NULL;
  void* z = host ? NULL : calloc(1, bytes);
  if (hipMalloc(&d, bytes) != hipSuccess) exit(2);
  if (hipMemcpy(d, host ? host : z, bytes, hipMemcpyHostToDevice) != hipSuccess) exit(2);
  free(z);
  return d;
}

static int update(void) {
  static float p[N], g[N], m[N], v[N], got[N], got8[N];
  for (uint32_t i = 0; i < N; ++i) p[i] = draw(), g[i] = 1e-3f * draw();
  zero_adam_hparams hp[2] = {{1e-3, 0.9, 0.999, 1e-8, 0.1, ZERO_ADAMW, 0, 1}, {1e-3, 0.9, 0.999, 1e-8, 0.1, ZERO_ADAMW, 0, 1}};
  zero_adam_tensor t[3];
  memset(t, 0, sizeof t);
  float* dg = up(g, sizeof g);
  t[0] = (zero_adam_tensor){N, up(p, sizeof p), dg, NULL, up(NULL, sizeof m), up(NULL, sizeof v), NULL, NULL, 0, 32};
  t[1].group = 1, t[1].state_bits = 32; /* an empty entry */
  t[2] = (zero_adam_tensor){N, up(p, sizeof p), dg, NULL, up(NULL, N), up(NULL, N), up(NULL, 4 * BLOCKS), up(NULL, 4 * BLOCKS), 1, 8};
  ZS(zero_adam_tensors_step(t, 3, ZERO_F32, ZERO_BF16, hp, 2, 0.5f, NULL, NULL, NULL));
  HIP(hipMemcpy(got, t[0].param, sizeof got, hipMemcpyDeviceToHost));
  HIP(hipMemcpy(got8, t[2].param, sizeof got8, hipMemcpyDeviceToHost));
  ZS(zero_host_adam_step(g, N, 0.5f, p, m, v, hp, NULL, ZERO_BF16, 1));
  int differ = 0;
  for (uint32_t i = 0; i < N; ++i) differ += memcmp(&got[i], &p[i], 4) != 0 || memcmp(&got8[i], &p[i], 4) != 0;
  float* dv = up(NULL, sizeof m);
  ZS(zero_adam_state_values(t[2].m, t[2].m_scale, N, 1, dv, NULL));
  HIP(hipMemcpy(got, dv, sizeof got, hipMemcpyDeviceToHost));
  float largest = 0.0f;
  for (uint32_t i = 0; i < N; ++i) largest = fabsf(m[i]) > largest ? fabsf(m[i]) : largest;
  for (uint32_t i = 0; i < N; ++i) HOLDS(fabsf(got[i] - m[i]) <= largest * (127.25f / 16129.0f));
  printf("update: %d differ\n", differ);
  t[2].group = 2;
  HOLDS(zero_adam_tensors_step(t, 3, ZERO_F32, ZERO_BF16, hp, 2, 0.5f, NULL, NULL, NULL) == ZERO_E_INVAL);
  t[2] = t[0];
  HOLDS(zero_adam_tensors_step(t, 3, ZERO_F32, ZERO_BF16, hp, 2, 0.5f, NULL, NULL, NULL) == ZERO_E_INVAL);
  return differ != 0;
}

static int boundary(void) {
  static uint16_t o[ROWS * D], h[ROWS * D];
  static float x[ROWS * D], y[ROWS * D];
  for (uint32_t i = 0; i < ROWS * D; ++i) x[i] = draw(), o[i] = to16(draw());
  zero_norm_block b;
  memset(&b, 0, sizeof b);
  b.rows = ROWS, b.features = D, b.gate_rows = 1, b.dtype = ZERO_BF16, b.stream_dtype = ZERO_F32;
  b.post = ZERO_NORM_NONE, b.pre = ZERO_NORM_RMS, b.eps = 1e-5f, b.residual_scale = 0.5f, b.branch_scale = 2.0f;
  b.branch = up(o, sizeof o), b.ld_branch = D;
  float *dx = up(x, sizeof x), *dy = up(NULL, sizeof y), *stats = up(NULL, 16 * ROWS);
  uint16_t* dh = up(NULL, sizeof h);
  ZS(zero_norm_forward(&b, dx, D, dy, D, dh, D, stats, NULL));
  HIP(hipMemcpy(y, dy, sizeof y, hipMemcpyDeviceToHost));
  HIP(hipMemcpy(h, dh, sizeof h, hipMemcpyDeviceToHost));
  int differ = 0;
  for (uint32_t r = 0; r < ROWS; ++r) {
    double sq = 0.0;
    for (uint32_t j = 0; j < D; ++j) sq += (double)y[r * D + j] * y[r * D + j];
    const double rstd = 1.0 / sqrt(sq / D + 1e-5);
    for (uint32_t j = 0; j < D; ++j) {
      const uint32_t i = r * D + j;
      differ += fabs(y[i] - (0.5 * x[i] + 2.0 * from16(o[i]))) > 1e-6;
      differ += fabs(from16(h[i]) - y[i] * rstd) > fabs(y[i] * rstd) / 256 + 1e-4;
    }
  }
  printf("boundary: %d differ\n", differ);
  HOLDS(zero_norm_forward(&b, dx, D, dy, D, dx, D, stats, NULL) == ZERO_E_INVAL);
  HOLDS(zero_norm_backward(&b, stats, dy, D, NULL, D, dh, D, dx, D, NULL, D, dy, D, NULL, NULL, NULL, NULL, ZERO_F32, 0, NULL, 0,
                           NULL) == ZERO_E_INVAL);
  return differ != 0;
}

static int loss(void) {
  static float z[ROWS * VOCAB], old[ROWS], adv[ROWS], got[ROWS], g1[ROWS * VOCAB], g2[ROWS * VOCAB];
  static int32_t label[ROWS];
  for (uint32_t i = 0; i < ROWS * VOCAB; ++i) z[i] = 4.0f * draw();
  for (uint32_t r = 0; r < ROWS; ++r)
    label[r] = r == 3 ? -1 : (int32_t)(r * 11 % VOCAB), old[r] = -6.0f + draw(), adv[r] = draw();
  zero_token_in in = {ROWS, VOCAB, ZERO_F32, 4, 1.0f, 0, up(z, sizeof z), VOCAB, up(label, sizeof label)};
  zero_policy p = {up(old, sizeof old), up(adv, sizeof adv), NULL, NULL, 0.2f, 0.3f, 0.0f, 0};
  float *dl = up(NULL, sizeof got), *stats = up(NULL, 4 * ZERO_TOKEN_STATS * ROWS), *dg = up(NULL, sizeof z);
  ZS(zero_policy_forward(&in, &p, dl, NULL, stats, NULL));
  ZS(zero_token_backward(&in, stats, NULL, 0, 2.0f, dg, VOCAB, NULL));
  HIP(hipMemcpy(g1, dg, sizeof g1, hipMemcpyDeviceToHost));
  ZS(zero_policy_step(&in, &p, NULL, 2.0f, dl, NULL, (void*)in.logits, VOCAB, NULL)); /* over the logits */
  HIP(hipMemcpy(got, dl, sizeof got, hipMemcpyDeviceToHost));
  HIP(hipMemcpy(g2, in.logits, sizeof g2, hipMemcpyDeviceToHost));
  int differ = 0;
  for (uint32_t r = 0; r < ROWS; ++r) {
    const float* zr = z + r * VOCAB;
    double sum = 0.0, want = 0.0, slope = 0.0;
    for (uint32_t v = 0; v < VOCAB; ++v) sum += exp((double)zr[v]);
    if (label[r] >= 0) {
      const double ratio = exp(zr[label[r]] - log(sum) - old[r]), low = 1.0 - (double)0.2f, high = 1.0 + (double)0.3f;
      const double held = ratio < low ? low : ratio > high ? high : ratio;
      want = -fmin(ratio * adv[r], held * adv[r]);
      slope = ratio * adv[r] <= held * adv[r] ? -ratio * adv[r] : 0.0;
    }
    differ += fabs(got[r] - want) > 1e-4 * (1.0 + fabs(want));
    for (uint32_t v = 0; v < VOCAB; ++v) {
      const double g = 2.0 * slope * ((label[r] == (int32_t)v) - exp((double)zr[v]) / sum);
      differ += fabs(g1[r * VOCAB + v] - g) > 1e-4 * (1.0 + fabs(g)) || fabs(g2[r * VOCAB + v] - g) > 1e-4 * (1.0 + fabs(g));
    }
  }
  printf("policy loss: %d differ\n", differ);
  p.clip_low = 2.0f;
  HOLDS(zero_policy_forward(&in, &p, dl, NULL, stats, NULL) == ZERO_E_INVAL);
  in.label_bytes = 3;
  HOLDS(zero_token_logp(&in, dl, NULL, NULL) == ZERO_E_INVAL);
  return differ != 0;
}

int main(void) {
  int bad = update();
  if (!bad) bad = boundary();
  if (!bad) bad = loss();
  return bad;
}
