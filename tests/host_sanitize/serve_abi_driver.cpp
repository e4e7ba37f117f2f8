// Host-side argument checks of include/qmm_serve.h, run against a build whose
// host code is instrumented with AddressSanitizer and
// UndefinedBehaviorSanitizer (tests/test_serve_host_sanitizers.py builds both).
// Every call either fails a host check or is empty, so nothing is launched and
// no GPU is needed; the pointers are fake. Extreme sizes and strides probe the
// overflow guards of the size arithmetic.
#include <math.h>
#include <initializer_list>
#include <stdint.h>
#include <stdio.h>

#include "qmm.h"
#include "qmm_serve.h"

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

static qmm_heads heads(int64_t token, int64_t head) { return qmm_heads{ptr(8), 0, token, head}; }
// (without slots, outputs or a workspace, so that a call within the limits stops there)
static int append(qmm_heads h, int64_t n, int64_t hkv, int64_t dim, int64_t n_freqs, int64_t pages, int64_t page) {
  double freqs[64] = {0.5};
  return qmm_kv4_append(QMM_T_F16, &h, &h, n, hkv, dim, 0, nullptr, 1e-6, (const int32_t *)ptr(2), freqs, n_freqs, 0,
                        nullptr, ptr(4), pages, page, nullptr);
}
static int read(qmm_heads h, int64_t n, int64_t hkv, int64_t dim, int64_t pages, int64_t page) {
  return qmm_kv4_read(QMM_T_F16, &h, &h, n, hkv, dim, nullptr, ptr(4), pages, page, nullptr);
}
static int attn(qmm_heads h, int64_t n, int64_t hq, int64_t hkv, int64_t dim, int64_t pages, int64_t page, int64_t stride,
                int64_t width) {
  return qmm_attn_kv4(QMM_T_F16, &h, &h, n, hq, hkv, dim, ptr(4), pages, page, (const int32_t *)ptr(5), stride, width,
                      nullptr, 1.f, nullptr, 0, nullptr);
}
static int moe(int64_t n, int64_t k, int64_t experts, int64_t used, int64_t ff, int64_t s1, int64_t s2, int64_t d1,
               int64_t d2) {
  return qmm_moe(ptr(1), QMM_T_F32, n, k, (const float *)ptr(2), experts, used, 1, ptr(3), ptr(4), QMM_TYPE_Q4_0, ff, s1, s2,
                 ptr(5), QMM_TYPE_Q8_0, d1, d2, (float *)ptr(6), nullptr, nullptr, nullptr, 0, nullptr);
}
static int sample(int64_t n, int64_t vocab, int64_t stride) {
  return qmm_sample(ptr(1), QMM_T_F32, n, vocab, stride, (const float *)ptr(2), nullptr, nullptr, nullptr, nullptr,
                    (int32_t *)ptr(3), nullptr, nullptr, 0, nullptr);
}

int main() {
  const int64_t dim31 = (int64_t{1} << 31) - 1;
  const qmm_heads h = heads(512, 128);

  EXPECT(append(h, 0, 2, 128, 1, 7, 32), QMM_OK);
  EXPECT(append(h, 5, 2, 128, 1, 7, 32), QMM_ERR_NULL);
  EXPECT(append(h, dim31, 2, 128, 1, dim31 / 256, 256), QMM_ERR_NULL);
  EXPECT(read(h, 0, 2, 128, 7, 32), QMM_OK);
  EXPECT(attn(h, 0, 4, 2, 128, 7, 32, 9, 9), QMM_OK);
  EXPECT(attn(h, 3, 4, 2, 128, 7, 32, 9, 9), QMM_ERR_NULL);
  EXPECT(moe(0, 256, 8, 2, 512, 144, 144 * 512, 544, 544 * 256), QMM_OK);
  EXPECT(moe(3, 256, 8, 2, 512, 144, 144 * 512, 544, 544 * 256), QMM_ERR_WORKSPACE);
  EXPECT(sample(0, 100, 100), QMM_OK);
  EXPECT(sample(3, 100, 100), QMM_ERR_WORKSPACE);
  EXPECT(sample((int64_t{1} << 22) - 1, QMM_SAMPLE_MAX_VOCAB, int64_t{1} << 35), QMM_ERR_WORKSPACE);
  for (int64_t x : kExtremes) {
    EXPECT(qmm_kv4_page_bytes(x, 2, 128), QMM_ERR_SHAPE);
    EXPECT(qmm_kv4_page_bytes(32, x, 128), QMM_ERR_SHAPE);
    EXPECT(qmm_kv4_page_bytes(32, 2, x), QMM_ERR_SHAPE);
    EXPECT(append(h, x, 2, 128, 1, 7, 32), QMM_ERR_SHAPE);
    EXPECT(append(h, 5, x, 128, 1, 7, 32), QMM_ERR_SHAPE);
    EXPECT(append(h, 5, 2, x, 1, 7, 32), QMM_ERR_SHAPE);
    EXPECT(append(h, 5, 2, 128, x, 7, 32), QMM_ERR_SHAPE);
    EXPECT(append(h, 5, 2, 128, 1, x, 32), QMM_ERR_SHAPE);
    EXPECT(append(h, 5, 2, 128, 1, 7, x), QMM_ERR_SHAPE);
    EXPECT(read(h, x, 2, 128, 7, 32), QMM_ERR_SHAPE);
    EXPECT(read(h, 5, x, 128, 7, 32), QMM_ERR_SHAPE);
    EXPECT(read(h, 5, 2, 128, x, 32), QMM_ERR_SHAPE);
    EXPECT(attn(h, x, 4, 2, 128, 7, 32, 9, 9), QMM_ERR_SHAPE);
    EXPECT(attn(h, 3, x, 2, 128, 7, 32, 9, 9), QMM_ERR_SHAPE);
    EXPECT(attn(h, 3, 4, x, 128, 7, 32, 9, 9), QMM_ERR_SHAPE);
    EXPECT(attn(h, 3, 4, 2, x, 7, 32, 9, 9), QMM_ERR_SHAPE);
    EXPECT(attn(h, 3, 4, 2, 128, x, 32, 9, 9), QMM_ERR_SHAPE);
    EXPECT(attn(h, 3, 4, 2, 128, 7, x, 9, 9), QMM_ERR_SHAPE);
    EXPECT(attn(h, 3, 4, 2, 128, 7, 32, 9, x), QMM_ERR_SHAPE);
    EXPECT(attn(h, 3, 4, 2, 128, 7, 32, x, 9) < 0, 1);
    EXPECT(moe(x, 256, 8, 2, 512, 144, 144 * 512, 544, 544 * 256), QMM_ERR_SHAPE);
    EXPECT(moe(3, x, 8, 2, 512, 144, 144 * 512, 544, 544 * 256), QMM_ERR_SHAPE);
    EXPECT(moe(3, 256, x, 2, 512, 144, 144 * 512, 544, 544 * 256), QMM_ERR_SHAPE);
    EXPECT(moe(3, 256, 8, x, 512, 144, 144 * 512, 544, 544 * 256), QMM_ERR_SHAPE);
    EXPECT(moe(3, 256, 8, 2, x, 144, 144 * 512, 544, 544 * 256), QMM_ERR_SHAPE);
    EXPECT(moe(3, 256, 8, 2, 512, x, 144 * 512, 544, 544 * 256) < 0, 1);
    EXPECT(moe(3, 256, 8, 2, 512, 144, x, 544, 544 * 256) < 0, 1);
    EXPECT(moe(3, 256, 8, 2, 512, 144, 144 * 512, x, 544 * 256) < 0, 1);
    EXPECT(moe(3, 256, 8, 2, 512, 144, 144 * 512, 544, x) < 0, 1);
    EXPECT(qmm_moe_workspace_bytes(x, 256, 512, 8, 2), QMM_ERR_SHAPE);
    EXPECT(qmm_moe_workspace_bytes(3, 256, 512, 8, x), QMM_ERR_SHAPE);
    EXPECT(sample(x, 100, 100), QMM_ERR_SHAPE);
    EXPECT(sample(3, x, 100), QMM_ERR_SHAPE);
    EXPECT(sample(3, 100, x) < 0, 1);
    EXPECT(qmm_sample_workspace_bytes(x, 100), QMM_ERR_SHAPE);
    EXPECT(append(heads(x, 128), 5, 2, 128, 1, 7, 32) < 0, 1);
    EXPECT(append(heads(512, x), 5, 2, 128, 1, 7, 32) < 0, 1);
    EXPECT(read(heads(x, 128), 5, 2, 128, 7, 32) < 0, 1);
    EXPECT(read(heads(512, x), 5, 2, 128, 7, 32) < 0, 1);
    EXPECT(attn(heads(x, 128), 3, 4, 2, 128, 7, 32, 9, 9) < 0, 1);
    EXPECT(attn(heads(512, x), 3, 4, 2, 128, 7, 32, 9, 9) < 0, 1);
  }
  // the largest of everything
  const int64_t big = (int64_t{1} << 24) - 32;
  EXPECT(qmm_moe_workspace_bytes(QMM_MOE_MAX_TOKENS, big, big, QMM_MOE_MAX_EXPERTS, QMM_MOE_MAX_USED) > 0, 1);
  EXPECT(moe(16, big, 512, 32, big, int64_t{1} << 36, int64_t{1} << 60, int64_t{1} << 36, int64_t{1} << 60), QMM_ERR_SHAPE);
  EXPECT(qmm_attn_kv4_workspace_bytes((int64_t{1} << 24) - 1, 1, 1, 64, dim31 / 256, 256), 0);
  EXPECT(qmm_attn_kv4_workspace_bytes(1, (int64_t{1} << 24) - 1, 1, 64, dim31 / 256, 256) >= 0, 1);
  EXPECT(qmm_attn_kv4_workspace_bytes(1, 1, 1, 128, dim31 / 256, 256) > 0, 1);
  EXPECT(qmm_sample_workspace_bytes((int64_t{1} << 22) - 1, QMM_SAMPLE_MAX_VOCAB) > 0, 1);
  for (double f : {64.5, -65.0, 1e300, (double)INFINITY, (double)NAN})
    EXPECT(qmm_kv4_append(QMM_T_F16, &h, &h, 5, 2, 128, 0, nullptr, 1e-6, (const int32_t *)ptr(2), &f, 1, 0,
                          (const int32_t *)ptr(3), ptr(4), 7, 32, nullptr),
           QMM_ERR_SHAPE);

  if (failures) {
    fprintf(stderr, "%d check(s) failed\n", failures);
    return 1;
  }
  printf("abi checks ok\n");
  return 0;
}
