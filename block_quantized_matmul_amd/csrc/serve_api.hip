// C ABI entry points of the serving-step operators (include/qmm_serve.h):
// argument validation and launch. As in the other entry points, every check
// runs on the host before any HIP call, so invalid arguments are reported
// without a GPU and nothing is enqueued.
#include <math.h>

#include "serve.h"

namespace {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxElems = int64_t{1} << 60;
constexpr int64_t kMaxStride = kMaxElems / 4;
constexpr int64_t kMaxRows = (int64_t{1} << 24) - 1;  // of a launch's workgroups
constexpr int64_t kMaxSampleRows = (int64_t{1} << 22) - 1;  // likewise, of 1024 threads
constexpr double kMaxFreq = 64.;  // radians per position, as in qmm_norm_rope

bool product_within(int64_t a, int64_t b, int64_t limit) { return b == 0 || a <= limit / b; }
bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int status_of(hipError_t e) { return e == hipSuccess ? QMM_OK : QMM_ERR_HIP; }
bool in_dim(int64_t n) { return n >= 0 && n <= kMaxDim; }
bool is_type(int t) { return t == QMM_T_F32 || t == QMM_T_F16 || t == QMM_T_BF16; }

// Offsets of a tensor of heads stay within 2^60 elements; the stride of an axis
// of one element is not used. `multiple`: what strides are multiples of.
int check_heads(const qmm_heads *h, int64_t tokens, int64_t heads, int64_t multiple, uintptr_t alignment) {
  if (h == nullptr || h->data == nullptr) return QMM_ERR_NULL;
  if (tokens > 1 && (h->token_stride < 0 || h->token_stride % multiple != 0)) return QMM_ERR_STRIDE;
  if (heads > 1 && (h->head_stride < 0 || h->head_stride % multiple != 0)) return QMM_ERR_STRIDE;
  if ((tokens > 1 && !product_within(tokens, h->token_stride, kMaxStride)) ||
      (heads > 1 && !product_within(heads, h->head_stride, kMaxStride)))
    return QMM_ERR_SHAPE;
  if (!aligned(h->data, alignment)) return QMM_ERR_ALIGN;
  return QMM_OK;
}
// No two heads of an output share elements.
bool apart(const qmm_heads &h, int64_t rows, int64_t heads, int64_t dim) {
  const int64_t r = h.token_stride, s = h.head_stride;
  if (rows == 0 || heads == 0 || (rows == 1 && heads == 1)) return true;
  if (rows == 1) return s >= dim;
  if (heads == 1) return r >= dim;
  return (s >= dim && r >= (heads - 1) * s + dim) || (r >= dim && s >= (rows - 1) * r + dim);
}

bool page_ok(int64_t page_tokens) {
  return page_tokens >= 16 && page_tokens <= QMM_KV4_MAX_PAGE_TOKENS && (page_tokens & (page_tokens - 1)) == 0;
}
int check_cache(const void *cache, int64_t n_pages, int64_t page_tokens, int64_t n_kv_heads, int64_t head_dim,
                qmm::Kv4Cache &c) {
  const int64_t bytes = qmm_kv4_page_bytes(page_tokens, n_kv_heads, head_dim);
  if (bytes < 0) return static_cast<int>(bytes);
  if (n_pages < 1 || n_pages > kMaxDim / page_tokens || !product_within(n_pages, bytes, kMaxElems)) return QMM_ERR_SHAPE;
  if (cache == nullptr) return QMM_ERR_NULL;
  if (!aligned(cache, 16)) return QMM_ERR_ALIGN;
  c.data = const_cast<uint8_t *>(static_cast<const uint8_t *>(cache));
  c.n_pages = n_pages, c.page_bytes = bytes, c.page_tokens = static_cast<int>(page_tokens);
  c.page_shift = __builtin_ctzll(static_cast<unsigned long long>(page_tokens));
  return QMM_OK;
}

constexpr int64_t kMaxMoeDim = (int64_t{1} << 24) - 32;

// A stack of n_experts matrices of n_rows rows of k weights.
int check_stack(int qtype, int64_t n_rows, int64_t k, int64_t n_experts, int64_t nb1, int64_t nb2) {
  const int64_t dense = qmm_row_bytes(qtype, k);
  if (dense < 0) return static_cast<int>(dense);
  if (nb1 < dense || nb1 % 4 != 0 || nb1 > kMaxElems / kMaxMoeDim || nb2 % 4 != 0 || nb2 < n_rows * nb1) return QMM_ERR_STRIDE;
  if (!product_within(n_experts, nb2, kMaxElems)) return QMM_ERR_SHAPE;
  return QMM_OK;
}

}  // namespace

extern "C" {

int64_t qmm_kv4_page_bytes(int64_t page_tokens, int64_t n_kv_heads, int64_t head_dim) {
  if (!page_ok(page_tokens) || n_kv_heads <= 0 || n_kv_heads > kMaxDim || (head_dim != 64 && head_dim != 128))
    return QMM_ERR_SHAPE;
  return n_kv_heads * (page_tokens / qmm::kKv4Tile) * qmm::kv4_tile_bytes(head_dim);
}

int qmm_kv4_append(int type, const qmm_heads *K, const qmm_heads *V, int64_t n_tokens, int64_t n_kv_heads,
                   int64_t head_dim, int norm, const float *weight, double eps, const int32_t *positions,
                   const double *freqs, int64_t n_freqs, int pairs, const int32_t *slots, void *cache,
                   int64_t n_pages, int64_t page_tokens, void *stream) {
  if (!is_type(type)) return QMM_ERR_TYPE;
  if (pairs != QMM_ROPE_HALVES && pairs != QMM_ROPE_NEIGHBOURS) return QMM_ERR_TYPE;
  qmm::Kv4Cache c{};
  int st = check_cache(cache, n_pages, page_tokens, n_kv_heads, head_dim, c);
  if (st != QMM_OK) return st;
  if (!in_dim(n_tokens) || !product_within(n_tokens, n_kv_heads, int64_t{1} << 40)) return QMM_ERR_SHAPE;
  if (n_freqs < 0 || n_freqs > head_dim / 2 || !(eps >= 0.) || isinf(eps)) return QMM_ERR_SHAPE;
  if (n_freqs > 0 && freqs == nullptr) return QMM_ERR_NULL;
  for (int64_t i = 0; i < n_freqs; ++i)
    if (!(fabs(freqs[i]) <= kMaxFreq)) return QMM_ERR_SHAPE;
  if (n_tokens == 0) return QMM_OK;
  for (const qmm_heads *h : {K, V})
    if ((st = check_heads(h, n_tokens, n_kv_heads, 1, type == QMM_T_F32 ? 4 : 2)) != QMM_OK) return st;
  if (slots == nullptr || (n_freqs > 0 && positions == nullptr)) return QMM_ERR_NULL;
  if (!aligned(slots, 4) || !aligned(positions, 4) || !aligned(weight, 4)) return QMM_ERR_ALIGN;
  return status_of(qmm::launch_kv4_append(type, *K, *V, n_tokens, n_kv_heads, head_dim, norm != 0, weight, eps,
                                          positions, freqs, n_freqs, pairs, slots, c,
                                          static_cast<hipStream_t>(stream)));
}

int qmm_kv4_read(int type, const qmm_heads *K, const qmm_heads *V, int64_t n_rows, int64_t n_kv_heads,
                 int64_t head_dim, const int32_t *slots, const void *cache, int64_t n_pages, int64_t page_tokens,
                 void *stream) {
  if (!is_type(type)) return QMM_ERR_TYPE;
  qmm::Kv4Cache c{};
  int st = check_cache(cache, n_pages, page_tokens, n_kv_heads, head_dim, c);
  if (st != QMM_OK) return st;
  if (!in_dim(n_rows) || !product_within(n_rows, n_kv_heads, int64_t{1} << 40)) return QMM_ERR_SHAPE;
  if (n_rows == 0 || (K == nullptr && V == nullptr)) return QMM_OK;
  for (const qmm_heads *h : {K, V}) {
    if (h == nullptr) continue;
    if ((st = check_heads(h, n_rows, n_kv_heads, 1, type == QMM_T_F32 ? 4 : 2)) != QMM_OK) return st;
    if (!apart(*h, n_rows, n_kv_heads, head_dim)) return QMM_ERR_STRIDE;
  }
  if (slots == nullptr) return QMM_ERR_NULL;
  if (!aligned(slots, 4)) return QMM_ERR_ALIGN;
  const qmm_heads none{};
  return status_of(qmm::launch_kv4_read(type, K ? *K : none, V ? *V : none, n_rows, n_kv_heads, head_dim, slots, c,
                                        static_cast<hipStream_t>(stream)));
}

int64_t qmm_attn_kv4_workspace_bytes(int64_t n_rows, int64_t n_q_heads, int64_t n_kv_heads, int64_t head_dim,
                                     int64_t table_width, int64_t page_tokens) {
  if (!page_ok(page_tokens) || (head_dim != 64 && head_dim != 128)) return QMM_ERR_SHAPE;
  if (n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads > kMaxRows || n_q_heads % n_kv_heads != 0) return QMM_ERR_SHAPE;
  if (n_rows < 0 || n_rows > kMaxRows || !product_within(n_rows, n_q_heads, kMaxRows)) return QMM_ERR_SHAPE;
  if (table_width < 0 || table_width > kMaxDim / page_tokens) return QMM_ERR_SHAPE;
  if (n_rows == 0) return 0;
  const qmm::Kv4Plan p = qmm::kv4_plan(n_rows, n_q_heads, n_kv_heads, head_dim, table_width * page_tokens);
  return qmm::kv4_workspace_bytes(p, n_rows, n_q_heads, head_dim);
}

int qmm_attn_kv4(int type, const qmm_heads *Q, const qmm_heads *O, int64_t n_rows, int64_t n_q_heads,
                 int64_t n_kv_heads, int64_t head_dim, const void *cache, int64_t n_pages, int64_t page_tokens,
                 const int32_t *tables, int64_t table_stride, int64_t table_width, const int32_t *lengths, float scale,
                 void *workspace, int64_t workspace_bytes, void *stream) {
  if (type != QMM_T_F16 && type != QMM_T_BF16) return QMM_ERR_TYPE;
  const int64_t need =
      qmm_attn_kv4_workspace_bytes(n_rows, n_q_heads, n_kv_heads, head_dim, table_width, page_tokens);
  if (need < 0) return static_cast<int>(need);
  if (!(scale > 0.f) || !(scale < 0x1p127f)) return QMM_ERR_SHAPE;  // (the kernel takes scale log2(e))
  qmm::Kv4Cache c{};
  int st = check_cache(cache, n_pages, page_tokens, n_kv_heads, head_dim, c);
  if (st != QMM_OK) return st;
  if (n_rows > 1 && (table_stride < 0 || !product_within(n_rows, table_stride, kMaxStride))) return QMM_ERR_STRIDE;
  if (n_rows == 0) return QMM_OK;
  for (const qmm_heads *h : {Q, O})
    if ((st = check_heads(h, n_rows, n_q_heads, 8, 16)) != QMM_OK) return st;
  if (!apart(*O, n_rows, n_q_heads, head_dim)) return QMM_ERR_STRIDE;
  if (lengths == nullptr || (table_width > 0 && tables == nullptr)) return QMM_ERR_NULL;
  if (!aligned(lengths, 4) || !aligned(tables, 4)) return QMM_ERR_ALIGN;
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need) return QMM_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return QMM_ERR_ALIGN;
  }
  return status_of(qmm::launch_attn_kv4(type, *Q, *O, n_rows, n_q_heads, n_kv_heads, head_dim, c, tables,
                                        n_rows > 1 ? table_stride : 0, table_width, lengths, scale, workspace,
                                        static_cast<hipStream_t>(stream)));
}

int64_t qmm_moe_workspace_bytes(int64_t n_tokens, int64_t k, int64_t n_ff, int64_t n_experts, int64_t n_used) {
  if (n_tokens < 0 || n_tokens > QMM_MOE_MAX_TOKENS || n_experts <= 0 || n_experts > QMM_MOE_MAX_EXPERTS) return QMM_ERR_SHAPE;
  if (n_used <= 0 || n_used > n_experts || n_used > QMM_MOE_MAX_USED) return QMM_ERR_SHAPE;
  if (k <= 0 || k % 32 != 0 || k > kMaxMoeDim || n_ff <= 0 || n_ff % 32 != 0 || n_ff > kMaxMoeDim) return QMM_ERR_SHAPE;
  return n_tokens == 0 ? 0 : qmm::moe_workspace_bytes(n_tokens, k, n_ff, n_experts, n_used);
}

int qmm_moe(const void *X, int x_type, int64_t n_tokens, int64_t k, const float *router, int64_t n_experts,
            int64_t n_used, int renormalise, const void *gate, const void *up, int type_in, int64_t n_ff,
            int64_t row_stride_in, int64_t expert_stride_in, const void *down, int type_out, int64_t row_stride_out,
            int64_t expert_stride_out, float *Y, int32_t *ids, float *weights, void *workspace,
            int64_t workspace_bytes, void *stream) {
  if (x_type != QMM_T_F32 && x_type != QMM_T_F16) return QMM_ERR_TYPE;
  const int64_t need = qmm_moe_workspace_bytes(n_tokens, k, n_ff, n_experts, n_used);
  if (need < 0) return static_cast<int>(need);
  int st = check_stack(type_in, n_ff, k, n_experts, row_stride_in, expert_stride_in);
  if (st == QMM_OK) st = check_stack(type_out, k, n_ff, n_experts, row_stride_out, expert_stride_out);
  if (st != QMM_OK) return st;
  if (n_tokens == 0) return QMM_OK;
  if (X == nullptr || router == nullptr || gate == nullptr || up == nullptr || down == nullptr || Y == nullptr)
    return QMM_ERR_NULL;
  for (const void *p : {X, static_cast<const void *>(router), gate, up, down, static_cast<const void *>(Y),
                        static_cast<const void *>(ids), static_cast<const void *>(weights)})
    if (!aligned(p, 4)) return QMM_ERR_ALIGN;
  if (workspace == nullptr || workspace_bytes < need) return QMM_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return QMM_ERR_ALIGN;
  qmm::MoeLayer m{};
  m.X = X, m.x_f16 = x_type == QMM_T_F16, m.n_tokens = n_tokens, m.k = k, m.n_ff = n_ff;
  m.n_experts = n_experts, m.n_used = n_used, m.router = router, m.gate = gate, m.up = up, m.down = down;
  m.type_in = type_in, m.type_out = type_out, m.nb1_in = row_stride_in, m.nb2_in = expert_stride_in;
  m.nb1_out = row_stride_out, m.nb2_out = expert_stride_out, m.renormalise = renormalise != 0;
  m.Y = Y, m.ids = ids, m.weights = weights;
  return status_of(qmm::launch_moe(m, workspace, static_cast<hipStream_t>(stream)));
}

int64_t qmm_sample_workspace_bytes(int64_t n_rows, int64_t vocab) {
  if (n_rows < 0 || n_rows > kMaxSampleRows || vocab <= 0 || vocab > QMM_SAMPLE_MAX_VOCAB) return QMM_ERR_SHAPE;
  return qmm::sample_workspace_bytes(n_rows, vocab);
}

int qmm_sample(const void *logits, int type, int64_t n_rows, int64_t vocab, int64_t row_stride, const float *u,
               const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
               int32_t *tokens, float *probs, void *workspace, int64_t workspace_bytes, void *stream) {
  if (!is_type(type)) return QMM_ERR_TYPE;
  const int64_t need = qmm_sample_workspace_bytes(n_rows, vocab);
  if (need < 0) return static_cast<int>(need);
  if (n_rows > 1 && row_stride < 0) return QMM_ERR_STRIDE;
  if (n_rows > 1 && !product_within(n_rows, row_stride, kMaxStride)) return QMM_ERR_SHAPE;
  if (n_rows == 0) return QMM_OK;
  if (logits == nullptr || u == nullptr || tokens == nullptr) return QMM_ERR_NULL;
  if (!aligned(logits, type == QMM_T_F32 ? 4 : 2)) return QMM_ERR_ALIGN;
  for (const void *p : {static_cast<const void *>(u), static_cast<const void *>(temperature),
                        static_cast<const void *>(top_k), static_cast<const void *>(top_p),
                        static_cast<const void *>(min_p), static_cast<const void *>(tokens),
                        static_cast<const void *>(probs)})
    if (!aligned(p, 4)) return QMM_ERR_ALIGN;
  if (workspace == nullptr || workspace_bytes < need) return QMM_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return QMM_ERR_ALIGN;
  const qmm::SampleCall c{logits, type, n_rows, vocab, n_rows > 1 ? row_stride : 0, u, temperature, top_k, top_p, min_p,
                          tokens, probs};
  return status_of(qmm::launch_sample(c, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
