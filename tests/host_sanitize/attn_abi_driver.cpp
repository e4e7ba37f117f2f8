// Host-side argument checks of include/qmm_attn.h, run against a build whose
// host code is instrumented with AddressSanitizer and
// UndefinedBehaviorSanitizer (tests/test_attn_host_sanitizers.py builds both).
// Every call either fails a host check or is empty, so nothing is launched and
// no GPU is needed; the pointers are fake. Extreme sizes and strides probe the
// overflow guards of the size arithmetic.
#include <math.h>
#include <initializer_list>
#include <stdint.h>
#include <stdio.h>

#include "qmm_attn.h"

static int failures = 0;

#define EXPECT(expr, want)                                                                                 \
  do {                                                                                                     \
    const long long got_ = (long long)(expr);                                                              \
    if (got_ != (long long)(want)) {                                                                       \
      fprintf(stderr, "FAIL line %d: %s = %lld, expected %lld\n", __LINE__, #expr, got_, (long long)(want)); \
      ++failures;                                                                                          \
    }                                                                                                      \
  } while (0)

static void *ptr(uintptr_t i) { return reinterpret_cast<void *>(i << 20); }
static const int64_t kExtremes[] = {INT64_MIN, INT64_MIN + 1, -1, INT64_MAX - 1, INT64_MAX, int64_t{1} << 62,
                                    int64_t{1} << 61, int64_t{1} << 60, int64_t{1} << 32, int64_t{1} << 31};

static int lora(int64_t n, int64_t k, int64_t ad, int64_t rank, int64_t rows) {
  return qmm_lora(ptr(1), QMM_T_F16, n, k, (const uint16_t *)ptr(2), (const uint16_t *)ptr(3), ad, rank, rows, nullptr,
                  (const int32_t *)ptr(4), nullptr, (float *)ptr(5), nullptr, 0, nullptr);
}
static int rope(qmm_head_part part, int64_t n, int64_t dim, int64_t n_freqs, int64_t n_slots) {
  double freqs[256] = {0.5};
  return qmm_norm_rope(&part, 1, n, dim, 0.f, (const int32_t *)ptr(6), freqs, n_freqs, 0, (const int32_t *)ptr(7), n_slots,
                       nullptr);
}
static qmm_heads heads(int64_t seq, int64_t tok, int64_t head) { return qmm_heads{ptr(8), seq, tok, head}; }
static int prompt(qmm_heads h, int64_t n, int64_t hq, int64_t hkv, int64_t dim, int64_t seqs) {
  return qmm_attn_prompt(QMM_T_F16, &h, &h, &h, &h, n, hq, hkv, dim, (const int32_t *)ptr(9), seqs, 1.f, nullptr);
}
static int shared(qmm_heads h, int64_t n, int64_t prefix, int64_t cap, int64_t hq, int64_t hkv, int64_t dim) {
  return qmm_attn_shared(QMM_T_F16, &h, &h, &h, prefix, &h, &h, cap, (const int32_t *)ptr(9), &h, n, hq, hkv, dim, 1.f,
                         nullptr, 0, nullptr);
}

int main() {
  // lora: each size at each extreme, and products past the limits
  for (int64_t x : kExtremes) {
    EXPECT(lora(x, 64, 2, 8, 16), QMM_ERR_SHAPE);
    EXPECT(lora(3, x, 2, 8, 16), QMM_ERR_SHAPE);
    EXPECT(lora(3, 64, x, 8, 16), QMM_ERR_SHAPE);
    EXPECT(lora(3, 64, 2, x, 16), QMM_ERR_SHAPE);
    EXPECT(lora(3, 64, 2, 8, x), QMM_ERR_SHAPE);
    EXPECT(qmm_lora_workspace_bytes(x, 64, 8), QMM_ERR_SHAPE);
    EXPECT(qmm_lora_workspace_bytes(3, x, 8), QMM_ERR_SHAPE);
    EXPECT(qmm_lora_workspace_bytes(3, 64, x), QMM_ERR_SHAPE);
  }
  const int64_t big_k = (int64_t{1} << 24) - 32, dim31 = (int64_t{1} << 31) - 1;
  EXPECT(lora(3, big_k, dim31, 256, 16), QMM_ERR_SHAPE);
  EXPECT(lora(3, 64, dim31, 256, dim31), QMM_ERR_SHAPE);
  EXPECT(lora((int64_t{1} << 25) - 1, big_k, 1, 1, dim31), QMM_ERR_WORKSPACE);
  EXPECT(qmm_lora_workspace_bytes((int64_t{1} << 25) - 1, big_k, 256) > 0, 1);
  EXPECT(qmm_lora_workspace_bytes(512, big_k, 256) > 0, 1);

  // norm and rotation: strides and sizes
  const qmm_head_part ok{ptr(1), QMM_T_F32, 256, 128, ptr(2), QMM_T_F16, 256, 128, 2, 1, nullptr, 1, 1};
  EXPECT(rope(ok, 0, 128, 64, 9), QMM_OK);
  for (int64_t x : kExtremes) {
    EXPECT(rope(ok, x, 128, 64, 9), QMM_ERR_SHAPE);
    EXPECT(rope(ok, 5, x, 64, 9), QMM_ERR_SHAPE);
    EXPECT(rope(ok, 5, 128, x, 9), QMM_ERR_SHAPE);
    EXPECT(rope(ok, 5, 128, 64, x), QMM_ERR_SHAPE);
    qmm_head_part p = ok;
    p.n_heads = x;
    EXPECT(rope(p, 5, 128, 64, 9), QMM_ERR_SHAPE);
    for (int64_t qmm_head_part::*stride : {&qmm_head_part::x_token_stride, &qmm_head_part::x_head_stride,
                                           &qmm_head_part::y_row_stride, &qmm_head_part::y_head_stride}) {
      p = ok;
      p.*stride = x;
      if (x >= 0 && x <= int64_t{1} << 32) continue;  // a valid stride
      EXPECT(rope(p, 5, 128, 64, 9), x < 0 ? QMM_ERR_STRIDE : QMM_ERR_SHAPE);
    }
  }
  // frequencies that the fixed point does not take
  for (double f : {64.5, -65.0, 1e300, (double)INFINITY, -(double)INFINITY, (double)NAN}) {
    EXPECT(qmm_norm_rope(&ok, 1, 5, 128, 0.f, (const int32_t *)ptr(6), &f, 1, 0, (const int32_t *)ptr(7), 9, nullptr),
           QMM_ERR_SHAPE);
  }

  // attention
  const qmm_heads h = heads(4096, 256, 64);
  EXPECT(prompt(h, 0, 4, 2, 64, 3), QMM_OK);
  EXPECT(shared(h, 0, 10, 10, 4, 2, 64), QMM_OK);
  for (int64_t x : kExtremes) {
    EXPECT(prompt(h, x, 4, 2, 64, 3), QMM_ERR_SHAPE);
    EXPECT(prompt(h, 9, x, 2, 64, 3), QMM_ERR_SHAPE);
    EXPECT(prompt(h, 9, 4, x, 64, 3), QMM_ERR_SHAPE);
    EXPECT(prompt(h, 9, 4, 2, x, 3), QMM_ERR_SHAPE);
    EXPECT(prompt(h, 9, 4, 2, 64, x), QMM_ERR_SHAPE);
    EXPECT(shared(h, x, 10, 10, 4, 2, 64), QMM_ERR_SHAPE);
    EXPECT(shared(h, 9, x, 10, 4, 2, 64), QMM_ERR_SHAPE);
    EXPECT(shared(h, 9, 10, x, 4, 2, 64), QMM_ERR_SHAPE);
    EXPECT(shared(h, 9, 10, 10, x, 2, 64), QMM_ERR_SHAPE);
    EXPECT(shared(h, 9, 10, 10, 4, x, 64), QMM_ERR_SHAPE);
    EXPECT(shared(h, 9, 10, 10, 4, 2, x), QMM_ERR_SHAPE);
    EXPECT(qmm_attn_shared_workspace_bytes(x, 10, 10, 4, 2, 64), QMM_ERR_SHAPE);
    EXPECT(prompt(heads(0, x, 64), 9, 4, 2, 64, 3), QMM_ERR_STRIDE);
    EXPECT(prompt(heads(0, 256, x), 9, 4, 2, 64, 3) < 0, 1);
    EXPECT(shared(heads(x, 256, 64), 9, 10, 10, 4, 2, 64) < 0, 1);
  }
  EXPECT(prompt(heads(0, 256, 64), dim31 - (1 << 20), 1, 1, 64, dim31 - 128), QMM_ERR_SHAPE);
  EXPECT(qmm_attn_shared_workspace_bytes(dim31 - (1 << 20), dim31 - (1 << 20), dim31 - (1 << 20), 1, 1, 64), QMM_ERR_SHAPE);
  EXPECT(qmm_attn_shared_workspace_bytes((int64_t{1} << 20), dim31 - (1 << 20), dim31 - (1 << 20), 8, 8, 128) != 0, 1);

  if (failures) {
    fprintf(stderr, "%d check(s) failed\n", failures);
    return 1;
  }
  printf("abi checks ok\n");
  return 0;
}
