// C ABI entry points of the attention-block operators (include/qmm_attn.h):
// argument validation and launch. As in qmm.h's entry points, every check
// runs on the host before any HIP call, so invalid arguments are reported
// without a GPU and nothing is enqueued.
#include <math.h>

#include <utility>

#include "attn.h"

namespace {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxElems = int64_t{1} << 60;
constexpr int64_t kMaxGroups = (int64_t{1} << 24) - 1;  // 256-thread workgroups of one launch (2^32 threads)
constexpr int64_t kMaxCopyStride = int64_t{1} << 25;  // elements: 63 rows of a block within 32-bit byte offsets
constexpr double kMaxFreq = 64.;  // radians per position: what qmm_norm_rope's fixed point stays accurate for
constexpr int64_t kMaxLoraTokens = (int64_t{1} << 25) - 1;
constexpr int64_t kMaxLoraK = (int64_t{1} << 24) - 1;

bool product_within(int64_t a, int64_t b, int64_t limit) { return b == 0 || a <= limit / b; }
bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int status_of(hipError_t e) { return e == hipSuccess ? QMM_OK : QMM_ERR_HIP; }
bool in_dim(int64_t n) { return n >= 0 && n <= kMaxDim; }

// Offsets of `a` rows and `b` columns under strides sa and sb stay within
// 2^60 elements (head_dim included by the margin).
bool span_within(int64_t a, int64_t sa, int64_t b, int64_t sb) {
  return (a <= 1 || product_within(a, sa, kMaxElems / 4)) && (b <= 1 || product_within(b, sb, kMaxElems / 4));
}
// No two heads of an output share elements.
bool apart(int64_t rows, int64_t row_stride, int64_t heads, int64_t head_stride, int64_t dim) {
  if (rows == 0 || heads == 0 || (rows == 1 && heads == 1)) return true;
  if (rows == 1) return head_stride >= dim;
  if (heads == 1) return row_stride >= dim;
  return (head_stride >= dim && row_stride >= (heads - 1) * head_stride + dim) ||
         (row_stride >= dim && head_stride >= (rows - 1) * row_stride + dim);
}

int check_heads(const qmm_heads *h, int64_t seqs, int64_t tokens, int64_t heads) {
  if (h == nullptr || h->data == nullptr) return QMM_ERR_NULL;
  // the stride of an axis of one element is never used
  for (const auto &[n, stride] : {std::pair{seqs, h->seq_stride}, {tokens, h->token_stride}, {heads, h->head_stride}})
    if (n > 1 && (stride < 0 || stride % 8 != 0)) return QMM_ERR_STRIDE;
  if (h->token_stride > kMaxCopyStride && tokens > 1) return QMM_ERR_STRIDE;
  if (!span_within(tokens, h->token_stride, heads, h->head_stride) ||
      (seqs > 1 && !product_within(seqs, h->seq_stride, kMaxElems / 4)))
    return QMM_ERR_SHAPE;
  if (!aligned(h->data, 16)) return QMM_ERR_ALIGN;
  return QMM_OK;
}
int check_attention(int type, int64_t tokens, int64_t n_q_heads, int64_t n_kv_heads, int64_t head_dim, float scale) {
  if (type != QMM_T_F16 && type != QMM_T_BF16) return QMM_ERR_TYPE;
  if (!in_dim(tokens) || n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads > kMaxDim || n_q_heads % n_kv_heads != 0)
    return QMM_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128) return QMM_ERR_SHAPE;
  if (!(scale > 0.f) || !(scale < 0x1p127f)) return QMM_ERR_SHAPE;  // (the kernels take scale log2(e))
  if (tokens > kMaxDim - (1 << 20) || !product_within(tokens, n_q_heads, kMaxDim - (1 << 20))) return QMM_ERR_SHAPE;
  return QMM_OK;
}

// Workgroups of qmm_attn_shared's two launches.
bool shared_fits(int64_t n_seqs, int64_t prefix_len, int64_t own_cap, int64_t n_q_heads, int64_t n_kv_heads) {
  const qmm::SharedPlan p = qmm::shared_plan(n_seqs, prefix_len, own_cap, n_q_heads, n_kv_heads);
  if (!product_within(n_seqs, n_q_heads, kMaxGroups)) return false;
  // row_tiles and own_tiles count rows, so neither product passes 2^31 times
  // the pieces, which number at most prefix_len or own_cap / 256
  return product_within(p.prefix_pieces, p.row_tiles * n_kv_heads, kMaxGroups / 2) &&
         product_within(p.own_pieces, n_seqs * p.own_tiles * n_kv_heads, kMaxGroups / 2);
}

}  // namespace

extern "C" {

int64_t qmm_lora_workspace_bytes(int64_t n_tokens, int64_t k, int64_t rank) {
  if (n_tokens < 0 || n_tokens > kMaxLoraTokens || k <= 0 || k % 32 != 0 || k > kMaxLoraK || rank <= 0 ||
      rank > QMM_LORA_MAX_RANK)
    return QMM_ERR_SHAPE;
  if (n_tokens == 0) return 0;
  return qmm::lora_splits(n_tokens, k, rank) * n_tokens * rank * 4;
}

int qmm_lora(const void *X, int x_type, int64_t n_tokens, int64_t k, const uint16_t *A, const uint16_t *B,
             int64_t n_adapters, int64_t rank, int64_t n_rows, const float *scales, const int32_t *ids,
             const float *base, float *Y, void *workspace, int64_t workspace_bytes, void *stream) {
  if (x_type != QMM_T_F32 && x_type != QMM_T_F16) return QMM_ERR_TYPE;
  const int64_t need = qmm_lora_workspace_bytes(n_tokens, k, rank);
  if (need < 0) return static_cast<int>(need);
  if (!in_dim(n_adapters) || !in_dim(n_rows)) return QMM_ERR_SHAPE;
  if (!product_within(n_tokens, n_rows, kMaxElems) || !product_within(n_adapters * rank, k, kMaxElems) ||
      !product_within(n_adapters * rank, n_rows, kMaxElems))
    return QMM_ERR_SHAPE;
  if (n_tokens == 0 || n_rows == 0) return QMM_OK;
  if (X == nullptr || ids == nullptr || Y == nullptr || (n_adapters > 0 && (A == nullptr || B == nullptr)))
    return QMM_ERR_NULL;
  if (!aligned(X, 16) || !aligned(A, 16) || !aligned(B, 2) || !aligned(scales, 4) || !aligned(ids, 4) ||
      !aligned(base, 4) || !aligned(Y, 4))
    return QMM_ERR_ALIGN;
  if (workspace == nullptr || workspace_bytes < need) return QMM_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return QMM_ERR_ALIGN;
  return status_of(qmm::launch_lora(X, x_type == QMM_T_F16, n_tokens, k, A, B, n_adapters, rank, n_rows, scales, ids,
                                    base, Y, static_cast<float *>(workspace), static_cast<hipStream_t>(stream)));
}

int qmm_norm_rope(const qmm_head_part *parts, int n_parts, int64_t n_tokens, int64_t head_dim, float eps,
                  const int32_t *positions, const double *freqs, int64_t n_freqs, int pairs, const int32_t *slots,
                  int64_t n_slots, void *stream) {
  if (n_parts < 0 || n_parts > QMM_HEAD_PARTS_MAX) return QMM_ERR_SHAPE;
  if (n_parts > 0 && parts == nullptr) return QMM_ERR_NULL;
  if (!in_dim(n_tokens) || !in_dim(n_slots) || head_dim < 2 || head_dim > QMM_NORM_ROPE_MAX_DIM || head_dim % 2 != 0)
    return QMM_ERR_SHAPE;
  if (n_freqs < 0 || n_freqs > head_dim / 2 || !(eps >= 0.f) || isinf(eps)) return QMM_ERR_SHAPE;
  if (pairs != QMM_ROPE_HALVES && pairs != QMM_ROPE_NEIGHBOURS) return QMM_ERR_TYPE;
  if (n_freqs > 0 && freqs == nullptr) return QMM_ERR_NULL;
  for (int64_t i = 0; i < n_freqs; ++i)
    if (!(fabs(freqs[i]) <= kMaxFreq)) return QMM_ERR_SHAPE;
  if (!aligned(positions, 4) || !aligned(slots, 4)) return QMM_ERR_ALIGN;
  int64_t heads = 0;
  for (int p = 0; p < n_parts; ++p) {
    const qmm_head_part &h = parts[p];
    for (int t : {h.x_type, h.y_type})
      if (t != QMM_T_F32 && t != QMM_T_F16 && t != QMM_T_BF16) return QMM_ERR_TYPE;
    if (!in_dim(h.n_heads)) return QMM_ERR_SHAPE;
    const int64_t rows = h.slotted ? n_slots : n_tokens;
    if ((n_tokens > 1 && h.x_token_stride < 0) || (rows > 1 && h.y_row_stride < 0) ||
        (h.n_heads > 1 && (h.x_head_stride < 0 || h.y_head_stride < 0)))
      return QMM_ERR_STRIDE;
    if (!span_within(n_tokens, h.x_token_stride, h.n_heads, h.x_head_stride) ||
        !span_within(rows, h.y_row_stride, h.n_heads, h.y_head_stride))
      return QMM_ERR_SHAPE;
    if (!apart(rows, h.y_row_stride, h.n_heads, h.y_head_stride, head_dim)) return QMM_ERR_STRIDE;
    if (h.n_heads == 0 || n_tokens == 0 || rows == 0) continue;  // nothing to read or store
    if (h.X == nullptr || h.Y == nullptr) return QMM_ERR_NULL;
    if ((h.rotate && (positions == nullptr || n_freqs == 0)) || (h.slotted && slots == nullptr)) return QMM_ERR_NULL;
    if (!aligned(h.X, h.x_type == QMM_T_F32 ? 4 : 2) || !aligned(h.Y, h.y_type == QMM_T_F32 ? 4 : 2) ||
        !aligned(h.weight, 4))
      return QMM_ERR_ALIGN;
    heads += h.n_heads;
  }
  if (heads > (1 << 24)) return QMM_ERR_SHAPE;
  if (n_tokens == 0 || heads == 0) return QMM_OK;
  return status_of(qmm::launch_norm_rope(parts, n_parts, n_tokens, head_dim, eps, positions, freqs, n_freqs, pairs,
                                         slots, n_slots, static_cast<hipStream_t>(stream)));
}

int qmm_attn_prompt(int type, const qmm_heads *Q, const qmm_heads *K, const qmm_heads *V, const qmm_heads *O,
                    int64_t n_tokens, int64_t n_q_heads, int64_t n_kv_heads, int64_t head_dim,
                    const int32_t *seq_starts, int64_t n_seqs, float scale, void *stream) {
  int st = check_attention(type, n_tokens, n_q_heads, n_kv_heads, head_dim, scale);
  if (st != QMM_OK) return st;
  if (n_seqs < 0 || n_seqs > kMaxDim - 128) return QMM_ERR_SHAPE;
  if (n_tokens == 0 || n_seqs == 0) return QMM_OK;
  if (seq_starts == nullptr) return QMM_ERR_NULL;
  const qmm_heads *all[] = {Q, K, V, O};
  for (const qmm_heads *h : all)
    if ((st = check_heads(h, 0, n_tokens, h == K || h == V ? n_kv_heads : n_q_heads)) != QMM_OK) return st;
  if (!apart(n_tokens, O->token_stride, n_q_heads, O->head_stride, head_dim)) return QMM_ERR_STRIDE;
  if (!aligned(seq_starts, 4)) return QMM_ERR_ALIGN;
  if (!product_within(n_tokens * (n_q_heads / n_kv_heads) / 128 + (n_seqs < n_tokens ? n_seqs : n_tokens), n_kv_heads,
                      kMaxGroups))
    return QMM_ERR_SHAPE;
  return status_of(qmm::launch_attn_prompt(type, *Q, *K, *V, *O, n_tokens, n_q_heads, n_kv_heads, head_dim, seq_starts,
                                           n_seqs, scale, static_cast<hipStream_t>(stream)));
}

int64_t qmm_attn_shared_workspace_bytes(int64_t n_seqs, int64_t prefix_len, int64_t own_cap, int64_t n_q_heads,
                                        int64_t n_kv_heads, int64_t head_dim) {
  const int st = check_attention(QMM_T_F16, n_seqs, n_q_heads, n_kv_heads, head_dim, 1.f);
  if (st != QMM_OK) return st;
  if (prefix_len < 0 || own_cap < 0 || prefix_len > kMaxDim - (1 << 20) || own_cap > kMaxDim - (1 << 20))
    return QMM_ERR_SHAPE;
  if (n_seqs == 0) return 0;
  if (!shared_fits(n_seqs, prefix_len, own_cap, n_q_heads, n_kv_heads)) return QMM_ERR_SHAPE;
  // a piece's row is head_dim outputs and a reference; the sums of weights
  // follow, as a further row for every head_dim + 1 pieces
  const int64_t pieces = qmm::shared_plan(n_seqs, prefix_len, own_cap, n_q_heads, n_kv_heads).pieces();
  return (pieces + (pieces + head_dim) / (head_dim + 1)) * n_seqs * n_q_heads * (head_dim + 1) * 4;
}

int qmm_attn_shared(int type, const qmm_heads *Q, const qmm_heads *PK, const qmm_heads *PV, int64_t prefix_len,
                    const qmm_heads *K, const qmm_heads *V, int64_t own_cap, const int32_t *lengths,
                    const qmm_heads *O, int64_t n_seqs, int64_t n_q_heads, int64_t n_kv_heads, int64_t head_dim,
                    float scale, void *workspace, int64_t workspace_bytes, void *stream) {
  int st = check_attention(type, n_seqs, n_q_heads, n_kv_heads, head_dim, scale);
  if (st != QMM_OK) return st;
  const int64_t need =
      qmm_attn_shared_workspace_bytes(n_seqs, prefix_len, own_cap, n_q_heads, n_kv_heads, head_dim);
  if (need < 0) return static_cast<int>(need);
  if (n_seqs == 0) return QMM_OK;
  for (const qmm_heads *h : {Q, O})
    if ((st = check_heads(h, 0, n_seqs, n_q_heads)) != QMM_OK) return st;
  if (prefix_len > 0)
    for (const qmm_heads *h : {PK, PV})
      if ((st = check_heads(h, 0, prefix_len, n_kv_heads)) != QMM_OK) return st;
  if (own_cap > 0) {
    for (const qmm_heads *h : {K, V})
      if ((st = check_heads(h, n_seqs, own_cap, n_kv_heads)) != QMM_OK) return st;
    if (lengths == nullptr) return QMM_ERR_NULL;
    if (!aligned(lengths, 4)) return QMM_ERR_ALIGN;
  }
  if (!apart(n_seqs, O->token_stride, n_q_heads, O->head_stride, head_dim)) return QMM_ERR_STRIDE;
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need) return QMM_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return QMM_ERR_ALIGN;
  }
  const qmm_heads none{};
  return status_of(qmm::launch_attn_shared(type, *Q, prefix_len > 0 ? *PK : none, prefix_len > 0 ? *PV : none,
                                           prefix_len, own_cap > 0 ? *K : none, own_cap > 0 ? *V : none, own_cap,
                                           lengths, *O, n_seqs, n_q_heads, n_kv_heads, head_dim, scale, workspace,
                                           static_cast<hipStream_t>(stream)));
}

}  // extern "C"
