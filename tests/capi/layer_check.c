/* The layer operators from plain C on the GPU, through the C ABI only. A linear layer (relu, bias, the kept
 * pre-activation; its weight and weight gradient one element into their buffers, the gradients written and then
 * added to) on small whole numbers, so that every sum is exact and must equal the host's, rounded once to
 * bf16 where it is stored so. Then the distillation loss with one entry a row at temperature 1, the cross entropy of a
 * label, as two calls and as one over the logits themselves, against the host's double evaluation: fp32 sums of
 * 513 terms, each off by a few roundings, loss and gradient within 1e-4 of values of size 10 and 1. And what
 * the calls refuse. Exits 0 when all hold. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <hip/hip_runtime_api.h>

#include "zero_shard.h"

#define M 77u
#define K 130u
#define N 96u
#define ROWS 40u
#define VOCAB 513u

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
static uint32_t draw(uint32_t n) {
  state = state * 6364136223846793005ull + 1442695040888963407ull;
  return (uint32_t)(state >> 33) % n;
}

static uint16_t bf16(float x) { /* to nearest even */
  uint32_t u;
  memcpy(&u, &x, 4);
  return (uint16_t)((u + 0x7fffu + (u >> 16 & 1)) >> 16);
}

static int device(void** d, const void* h, size_t bytes) {
  if (hipMalloc(d, bytes) != hipSuccess) return 1;
  if (!h) return 0;
  return hipMemcpy(*d, h, bytes, hipMemcpyHostToDevice) != hipSuccess;
}

static int whole[5]; /* -2 .. 2 drawn into a matrix and its bf16 */
static void fill(float* f, uint16_t* h, uint32_t n) {
  uint32_t i;
  for (i = 0; i < n; ++i) f[i] = (float)whole[draw(5)], h[i] = bf16(f[i]);
}

static float x[M * K], w[N * K], b[N], dy[M * N], z[M * N];
static uint16_t hx[M * K], hw[N * K + 1], hb[N], hdy[M * N], got_y[M * N], got_pre[M * N], got_dz[M * N], got_dx[M * K];
static float got_dw[N * K + 1], got_db[N], logits[ROWS * VOCAB], loss[3][ROWS], grad[2][ROWS * VOCAB];

int main(void) {
  void *dx_, *dw_, *db_, *ddy_, *y, *pre, *dz, *dx, *dw, *db, *ws, *dl, *didx, *dtop, *dloss, *dstats, *dgrad;
  zero_linear_shape s;
  zero_distill_in in;
  uint32_t i, j, k, bad = 0;
  int32_t label[ROWS];
  float top[ROWS];
  uint64_t need = zero_linear_workspace_bytes(M, K, N, 0), back = zero_linear_workspace_bytes(M, K, N, 1);

  for (i = 0; i < 5; ++i) whole[i] = (int)i - 2;
  fill(x, hx, M * K);
  fill(w, hw + 1, N * K);
  fill(b, hb, N);
  fill(dy, hdy, M * N);
  if (back > need) need = back;
  if (device(&dx_, hx, sizeof hx) || device(&dw_, hw, sizeof hw) || device(&db_, hb, sizeof hb) ||
      device(&ddy_, hdy, sizeof hdy) || device(&y, NULL, sizeof got_y) || device(&pre, NULL, sizeof got_pre) ||
      device(&dz, NULL, sizeof got_dz) || device(&dx, NULL, sizeof got_dx) || device(&dw, NULL, sizeof got_dw) ||
      device(&db, NULL, sizeof got_db) || device(&ws, NULL, need + 16)) {
    fprintf(stderr, "no device memory\n");
    return 2;
  }
  s.rows = M, s.in_features = K, s.out_features = N, s.dtype = ZERO_BF16, s.act = ZERO_ACT_RELU;
  ZS(zero_linear_forward(&s, dx_, K, (uint16_t*)dw_ + 1, db_, NULL, 0, pre, N, y, N, ws, need, NULL));
  for (i = 0; i < 2; ++i)
    ZS(zero_linear_backward(&s, ddy_, N, dx_, K, (uint16_t*)dw_ + 1, pre, N, dz, N, dx, K, (float*)dw + 1, db, ZERO_F32,
                            (int32_t)i, ws, need, NULL));
  HIP(hipDeviceSynchronize());
  HIP(hipMemcpy(got_y, y, sizeof got_y, hipMemcpyDeviceToHost));
  HIP(hipMemcpy(got_pre, pre, sizeof got_pre, hipMemcpyDeviceToHost));
  HIP(hipMemcpy(got_dz, dz, sizeof got_dz, hipMemcpyDeviceToHost));
  HIP(hipMemcpy(got_dx, dx, sizeof got_dx, hipMemcpyDeviceToHost));
  HIP(hipMemcpy(got_dw, dw, sizeof got_dw, hipMemcpyDeviceToHost));
  HIP(hipMemcpy(got_db, db, sizeof got_db, hipMemcpyDeviceToHost));
  for (i = 0; i < M; ++i)
    for (j = 0; j < N; ++j) {
      float v = b[j];
      for (k = 0; k < K; ++k) v += x[i * K + k] * w[j * K + k];
      z[i * N + j] = v > 0 ? dy[i * N + j] : 0.0f; /* dz */
      bad += got_pre[i * N + j] != bf16(v) || got_y[i * N + j] != bf16(v > 0 ? v : 0.0f);
      bad += (got_dz[i * N + j] & 0x7fff) != (bf16(z[i * N + j]) & 0x7fff); /* 0 of either sign */
    }
  for (i = 0; i < M; ++i)
    for (k = 0; k < K; ++k) {
      float v = 0.0f;
      for (j = 0; j < N; ++j) v += z[i * N + j] * w[j * K + k];
      bad += (got_dx[i * K + k] & (v == 0 ? 0x7fff : 0xffff)) != bf16(v);
    }
  for (j = 0; j < N; ++j) {
    float sum = 0.0f;
    for (i = 0; i < M; ++i) sum += z[i * N + j];
    bad += got_db[j] != 2 * sum;
    for (k = 0; k < K; ++k) {
      float v = 0.0f;
      for (i = 0; i < M; ++i) v += z[i * N + j] * x[i * K + k];
      bad += got_dw[1 + j * K + k] != 2 * v;
    }
  }
  printf("linear layer: %u differ\n", bad);
  HOLDS(bad == 0);

  for (i = 0; i < ROWS; ++i) {
    label[i] = (int32_t)draw(VOCAB), top[i] = 0.0f;
    for (j = 0; j < VOCAB; ++j) logits[i * VOCAB + j] = (float)draw(4096) / 512.0f - 4.0f;
  }
  if (device(&dl, logits, sizeof logits) || device(&didx, label, sizeof label) || device(&dtop, top, sizeof top) ||
      device(&dloss, NULL, sizeof loss) || device(&dstats, NULL, ROWS * 8) || device(&dgrad, NULL, sizeof grad[0])) {
    fprintf(stderr, "no device memory\n");
    return 2;
  }
  memset(&in, 0, sizeof in);
  in.rows = ROWS, in.vocab = VOCAB, in.topk = 1, in.logit_dtype = in.teacher_dtype = ZERO_F32, in.index_bytes = 4;
  in.temperature = 1.0f, in.logits = dl, in.ld_logits = VOCAB, in.top_index = didx, in.top_logits = dtop, in.ld_top = 1;
  ZS(zero_distill_forward(&in, (float*)dloss, (float*)dstats, NULL));
  ZS(zero_distill_backward(&in, (const float*)dstats, NULL, 1.0f, dgrad, VOCAB, NULL));
  HIP(hipDeviceSynchronize());
  HIP(hipMemcpy(grad[0], dgrad, sizeof grad[0], hipMemcpyDeviceToHost));
  ZS(zero_distill_step(&in, NULL, 1.0f, (float*)dloss + ROWS, dl, VOCAB, NULL)); /* over the logits */
  HIP(hipDeviceSynchronize());
  HIP(hipMemcpy(grad[1], dl, sizeof grad[1], hipMemcpyDeviceToHost));
  HIP(hipMemcpy(loss, dloss, sizeof loss, hipMemcpyDeviceToHost));
  for (i = 0; i < ROWS; ++i) {
    double sum = 0.0;
    for (j = 0; j < VOCAB; ++j) sum += exp(logits[i * VOCAB + j]);
    for (k = 0; k < 2; ++k) {
      bad += !(fabs(loss[k][i] - (log(sum) - logits[i * VOCAB + (uint32_t)label[i]])) <= 1e-4);
      for (j = 0; j < VOCAB; ++j)
        bad += !(fabs(grad[k][i * VOCAB + j] - (exp(logits[i * VOCAB + j]) / sum - (j == (uint32_t)label[i]))) <= 1e-4);
    }
  }
  printf("distillation loss: %u differ\n", bad);
  HOLDS(bad == 0);

  HOLDS(zero_linear_forward(NULL, dx_, K, dw_, NULL, NULL, 0, NULL, 0, y, N, ws, need, NULL) == ZERO_E_INVAL);
  HOLDS(zero_linear_forward(&s, dx_, K - 1, dw_, NULL, NULL, 0, NULL, 0, y, N, ws, need, NULL) == ZERO_E_INVAL);
  HOLDS(zero_linear_backward(&s, ddy_, N, NULL, K, dw_, pre, N, dz, N, dx, K, dw, NULL, ZERO_F32, 0, ws, need, NULL) ==
        ZERO_E_INVAL);
  s.dtype = ZERO_F32;
  HOLDS(zero_linear_forward(&s, dx_, K, dw_, NULL, NULL, 0, NULL, 0, y, N, ws, need, NULL) == ZERO_E_UNSUPPORTED);
  HOLDS(zero_distill_step(&in, NULL, INFINITY, (float*)dloss, dgrad, VOCAB, NULL) == ZERO_E_INVAL);
  in.topk = ZERO_DISTILL_MAX_TOPK + 1;
  HOLDS(zero_distill_forward(&in, (float*)dloss, (float*)dstats, NULL) == ZERO_E_UNSUPPORTED);
  return 0;
}
