/*
 * qmm_attn.h - C ABI of the operators that stand between the MUL_MATs of a
 * served transformer layer on the AMD MI355X (gfx950), in the same libqmm.so
 * as qmm.h:
 *
 *   qmm_lora         low-rank adapters of many requests beside a shared
 *                    projection (added to a MUL_MAT's Y);
 *   qmm_norm_rope    RMS norm of each query and key head, rotation by
 *                    position, conversion and the store into a cache;
 *   qmm_attn_prompt  causal attention over packed prompts of different
 *                    lengths, with grouped heads;
 *   qmm_attn_shared  attention of a decode batch, one token per sequence,
 *                    over a prefix that all sequences share and each one's
 *                    own cache.
 *
 * Conventions are those of qmm.h: every pointer is device memory owned by
 * the caller unless stated otherwise, nothing is retained or allocated, work
 * is enqueued on `stream` (a hipStream_t of the current device, or NULL) and
 * the call returns without waiting; every check runs on the host before
 * anything is enqueued and returns a QMM_ERR_* status; qmm_status_string()
 * names it. There is no global state: calls on different streams may run
 * concurrently as long as their workspaces and outputs differ. Every call
 * may be captured into a HIP graph (no allocation, copy, memset or
 * synchronisation; host tables are read during the call and travel in the
 * kernel's arguments). Results repeat bit for bit for the same arguments on
 * the same device.
 */
#ifndef QMM_ATTN_H
#define QMM_ATTN_H

#include <stdint.h>

#include "qmm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of these operators (the first two as QMM_X_F32, QMM_X_F16). */
#define QMM_T_F32 0
#define QMM_T_F16 1
#define QMM_T_BF16 2

/* Which elements of a head rotate together (qmm_norm_rope). */
#define QMM_ROPE_HALVES 0     /* element i with element i + n_freqs */
#define QMM_ROPE_NEIGHBOURS 1 /* element 2 i with element 2 i + 1 */

#define QMM_LORA_MAX_RANK 256
#define QMM_HEAD_PARTS_MAX 4
#define QMM_NORM_ROPE_MAX_DIM 512

/*
 * qmm_lora - Y[t][r] = base[t][r] + scales[a] * sum_j B[a][r][j] V[t][j],
 *            V[t][j] = sum_i A[a][j][i] X[t][i],   a = ids[t].
 * The adapters' low-rank products of a batch whose tokens belong to requests
 * with adapters of their own, beside the one projection they share: base is
 * the Y of that MUL_MAT (and may be this call's Y).
 *   X           fp32 or fp16 (x_type QMM_T_F32 / QMM_T_F16) [n_tokens][k],
 *               16-byte aligned
 *   k           positive multiple of 32 (as the MUL_MAT's)
 *   A           fp16 [n_adapters][rank][k], 16-byte aligned
 *   B           fp16 [n_adapters][n_rows][rank], 2-byte aligned
 *   rank        1 .. QMM_LORA_MAX_RANK, one for the whole stack: adapters of
 *               a smaller rank are padded with zero rows of A
 *   scales      fp32 [n_adapters], or NULL for 1
 *   ids         int32 [n_tokens], 4-byte aligned. -1: no adapter, Y = base.
 *               Any other id outside [0, n_adapters) cannot be checked on the
 *               host: that token's row of Y is filled with quiet NaNs and no
 *               adapter is read for it (as qmm_matmul_id does).
 *   base        fp32 [n_tokens][n_rows], 4-byte aligned; NULL for zeros; may
 *               be Y itself, but must not overlap it otherwise
 *   Y           fp32 [n_tokens][n_rows], 4-byte aligned; must not overlap X,
 *               A, B, scales or ids
 *   workspace   at least qmm_lora_workspace_bytes(n_tokens, k, rank) bytes,
 *               16-byte aligned; holds V as partial sums over ranges of k.
 *               Overwritten; two calls in flight must not share one.
 * Numerics: A, B and an fp16 X are multiplied exactly and summed in fp32; an
 * fp32 X is not rounded; V stays in fp32. Non-finite values of one token's
 * X or of an adapter stay in the rows of the tokens that use them.
 * Time: up to 512 tokens are gathered by their adapters, wherever they stand.
 * Beyond, 64 consecutive tokens take theirs one after another, as suits prompts
 * (1000 tokens of 4096 to 4096 rows, rank 16: 19 us in 9 runs, 84 us where 32
 * adapters alternate at random).
 * n_tokens == 0 or n_rows == 0 is a no-op. Sizes: n_tokens < 2^25, k < 2^24,
 * n_rows, n_adapters < 2^31, n_tokens * n_rows, n_adapters * rank * k,
 * n_adapters * n_rows * rank <= 2^60 (QMM_ERR_SHAPE).
 */
int qmm_lora(const void *X, int x_type, int64_t n_tokens, int64_t k, const uint16_t *A, const uint16_t *B,
             int64_t n_adapters, int64_t rank, int64_t n_rows, const float *scales, const int32_t *ids,
             const float *base, float *Y, void *workspace, int64_t workspace_bytes, void *stream);

/* qmm_lora_workspace_bytes - the workspace qmm_lora needs for these sizes, or
 * QMM_ERR_SHAPE. The same on every device. Fewer tokens may need more (2048 of
 * k 4096 more than 2049): a workspace kept for calls of different sizes is as
 * large as qmm_lora_workspace_max_bytes says. */
int64_t qmm_lora_workspace_bytes(int64_t n_tokens, int64_t k, int64_t rank);

/* qmm_lora_workspace_max_bytes - what no call of at most these sizes needs
 * more than; never decreases with any of them. Up to 512 tokens V is kept in at
 * most max_k / 512 (but 16 to 256) partial sums, beyond in as many as make
 * 32768 rows, or in one. */
static inline int64_t qmm_lora_workspace_max_bytes(int64_t max_tokens, int64_t max_k, int64_t max_rank) {
  const int64_t sums = max_k / 512 < 16 ? 16 : max_k / 512 > 256 ? 256 : max_k / 512;
  int64_t rows = (max_tokens < 512 ? max_tokens : 512) * sums;
  if (max_tokens > 512 && rows < 32768) rows = 32768;
  if (rows < max_tokens) rows = max_tokens;
  return rows * max_rank * 4;
}

/* One group of heads of a qmm_norm_rope call (a host struct, read during the
 * call). Strides are in elements; the elements of one head are contiguous. */
typedef struct qmm_head_part {
  const void *X; /* element e of head h of token t at X + t * x_token_stride + h * x_head_stride + e */
  int x_type;    /* QMM_T_* */
  int64_t x_token_stride;
  int64_t x_head_stride;
  void *Y; /* likewise, with the token's slot in place of t if slotted */
  int y_type;
  int64_t y_row_stride;
  int64_t y_head_stride;
  int64_t n_heads;
  int norm;            /* 1: divide by the head's root mean square */
  const float *weight; /* fp32 [head_dim] times the normed head; NULL for 1; only with norm */
  int rotate;          /* 1: rotate by the token's position */
  int slotted;         /* 1: the row of Y is slots[t] */
} qmm_head_part;

/*
 * qmm_norm_rope - for every part, token and head, in this order:
 *   norm:    x = x / sqrt(mean_e x[e]^2 + eps) * weight[e]
 *   rotate:  for i < n_freqs, with angle = positions[t] * freqs[i],
 *            (a, b) = (a cos angle - b sin angle, b cos angle + a sin angle),
 *            where a and b are elements i and i + n_freqs (QMM_ROPE_HALVES)
 *            or 2 i and 2 i + 1 (QMM_ROPE_NEIGHBOURS); elements from
 *            2 n_freqs on stay as they are
 *   store:   rounded once to y_type, at row t or slots[t] of Y.
 * One launch takes the queries, keys and values of a batch from the products
 * that made them into the attention's operands: queries and keys normed and
 * rotated, values only converted, keys and values stored into a cache.
 *   parts, n_parts  host array, 0 .. QMM_HEAD_PARTS_MAX
 *   head_dim        even, 2 .. QMM_NORM_ROPE_MAX_DIM
 *   eps             >= 0, finite
 *   positions       int32 [n_tokens], any value; needed if a part rotates
 *   freqs           HOST array of n_freqs doubles, radians per position,
 *                   magnitudes at most 64; read during the call
 *   n_freqs         0 .. head_dim / 2; at least 1 if a part rotates
 *   slots, n_slots  int32 [n_tokens]; needed if a part is slotted. A token
 *                   whose slot lies outside [0, n_slots) is not stored (so
 *                   -1 leaves it out). Two tokens with one slot: either's
 *                   values remain, element by element.
 * Pointers are aligned to their element type (positions, slots and weight to
 * 4). Strides are >= 0 (those of axes of one element are not used), and two
 * different heads of Y must not share elements:
 * y_row_stride >= (n_heads - 1) * y_head_stride + head_dim, or
 * y_head_stride >= (rows - 1) * y_row_stride + head_dim with rows = n_slots
 * or n_tokens (QMM_ERR_STRIDE). Y may be X itself, with equal types and
 * strides and not slotted; otherwise no Y overlaps any X or another Y.
 * Numerics: fp32, the norm's sum included (a head whose squares leave fp32's
 * range is normed as if by infinity or by sqrt(eps)); an angle is reduced to
 * a turn in 64-bit fixed point (error below 2^-30 of a turn at any position)
 * before sine and cosine. n_tokens == 0 is a no-op. n_tokens, n_slots < 2^31;
 * at most 2^24 heads in all parts; every offset <= 2^60 elements.
 */
int qmm_norm_rope(const qmm_head_part *parts, int n_parts, int64_t n_tokens, int64_t head_dim, float eps,
                  const int32_t *positions, const double *freqs, int64_t n_freqs, int pairs, const int32_t *slots,
                  int64_t n_slots, void *stream);

/* A tensor of heads (a host struct, read during the call): element e of head
 * h of token t (of sequence b) at data + b * seq_stride + t * token_stride +
 * h * head_stride + e. Strides are in elements, >= 0 and multiples of 8,
 * token_stride at most 2^25, and data is 16-byte aligned. seq_stride counts
 * only where stated, and the stride of an axis of one element nowhere. */
typedef struct qmm_heads {
  void *data;
  int64_t seq_stride;
  int64_t token_stride;
  int64_t head_stride;
} qmm_heads;

/*
 * qmm_attn_prompt - causal attention within each of n_seqs sequences packed
 * along the token axis: sequence i holds tokens seq_starts[i] ..
 * seq_starts[i + 1] - 1, and for every token t and query head h
 *   O[t][h] = sum_u w_u V[u][g],  w = softmax_u(scale * Q[t][h] . K[u][g]),
 * over the tokens u <= t of t's sequence, g = h / (n_q_heads / n_kv_heads).
 *   type         QMM_T_F16 or QMM_T_BF16, of Q, K, V and O
 *   Q, O         n_q_heads heads; K, V: n_kv_heads (a divisor of n_q_heads);
 *                all [n_tokens] (seq_stride unused)
 *   head_dim     64 or 128
 *   seq_starts   int32 [n_seqs + 1], non-decreasing within [0, n_tokens].
 *                Device data: a sequence whose two ends are not so is left
 *                out, and where others then overlap, the rows of the tokens
 *                that they share are undefined. Sequences may be empty.
 *   scale        > 0 and < 2^127 (usually 1 / sqrt(head_dim))
 * Tokens outside every sequence keep their rows of O, and their Q, K and V
 * are not read. O must not overlap Q, K or V, nor two of its own heads each
 * other (strides as in qmm_norm_rope).
 * Numerics: scores (infinite beyond fp32's range), the softmax's maximum and
 * sum, and the output's sum in fp32; each weight, relative to a reference
 * within a factor 2^8 of the largest so far, is rounded to `type` for the
 * matrix cores, and the output once at the end. The sum of the values times
 * these weights has to stay within fp32's range: bf16 values below 2^118 over
 * the number of keys do, and all fp16 ones, whose outputs are never beyond the
 * largest finite fp16. A non-finite K or V of a later token does not reach an
 * earlier one; where one is attended to, the outputs it enters are not finite
 * (infinite or NaN). n_tokens == 0 or n_seqs == 0 is a no-op. n_tokens,
 * n_seqs < 2^31 - 128 and n_tokens * n_q_heads < 2^31 - 2^20, and
 * (n_tokens * (n_q_heads / n_kv_heads) / 128 + min(n_seqs, n_tokens)) *
 * n_kv_heads < 2^24, the workgroups of a launch (QMM_ERR_SHAPE).
 */
int qmm_attn_prompt(int type, const qmm_heads *Q, const qmm_heads *K, const qmm_heads *V, const qmm_heads *O,
                    int64_t n_tokens, int64_t n_q_heads, int64_t n_kv_heads, int64_t head_dim,
                    const int32_t *seq_starts, int64_t n_seqs, float scale, void *stream);

/*
 * qmm_attn_shared - attention of one token of each of n_seqs sequences over
 * a prefix of prefix_len tokens whose keys and values all sequences share
 * (read once for all of them), followed by the first lengths[b] tokens of
 * sequence b's own cache:
 *   O[b][h] = sum_u w_u v_u,  w = softmax_u(scale * Q[b][h] . k_u),
 * over both, g = h / (n_q_heads / n_kv_heads) as above.
 *   type         QMM_T_F16 or QMM_T_BF16, of all tensors
 *   Q, O         [n_seqs] in the token axis, n_q_heads heads
 *   PK, PV       [prefix_len], n_kv_heads heads; may be NULL if prefix_len is 0
 *   K, V         sequence b at seq_stride * b, own_cap tokens, n_kv_heads
 *                heads; may be NULL if own_cap is 0
 *   lengths      int32 [n_seqs]; not read if own_cap is 0. A length of 0
 *                with prefix_len 0 gives a row of zeros. Device data: a
 *                length outside [0, own_cap] gives that sequence rows of
 *                quiet NaNs, and its cache is not read. Nothing at or past a
 *                length is read.
 *   head_dim     64 or 128
 *   scale        > 0 and < 2^127
 *   workspace    at least qmm_attn_shared_workspace_bytes(...) bytes, 16-byte
 *                aligned; partial results, overwritten; two calls in flight
 *                must not share one. May be NULL when that size is 0.
 * O must not overlap K, V, PK, PV or the workspace, nor two of its own heads
 * each other; it may be Q itself, with equal strides.
 * Time: the work is divided by own_cap and the number of sequences, since the
 * host does not know the lengths. Of many sequences with one much longer cache
 * than the others', that one decides the time.
 * Numerics as qmm_attn_prompt; partial results are joined in fp32 in a fixed
 * order. n_seqs == 0 is a no-op. prefix_len, own_cap < 2^31 - 2^20. n_seqs *
 * n_q_heads up to 2^22 is taken with any of these; from 2^24 on, and before
 * where a launch would have more than 2^24 workgroups, it is QMM_ERR_SHAPE.
 */
int qmm_attn_shared(int type, const qmm_heads *Q, const qmm_heads *PK, const qmm_heads *PV, int64_t prefix_len,
                    const qmm_heads *K, const qmm_heads *V, int64_t own_cap, const int32_t *lengths,
                    const qmm_heads *O, int64_t n_seqs, int64_t n_q_heads, int64_t n_kv_heads, int64_t head_dim,
                    float scale, void *workspace, int64_t workspace_bytes, void *stream);

/* qmm_attn_shared_workspace_bytes - the workspace qmm_attn_shared needs for
 * these sizes, or QMM_ERR_SHAPE. The same on every device. Fewer sequences or
 * keys may need more (32 sequences on a prefix of 32000 more than 48): a
 * workspace kept for calls of different sizes is as large as
 * qmm_attn_shared_workspace_max_bytes says. */
int64_t qmm_attn_shared_workspace_bytes(int64_t n_seqs, int64_t prefix_len, int64_t own_cap, int64_t n_q_heads,
                                        int64_t n_kv_heads, int64_t head_dim);

/* qmm_attn_shared_workspace_max_bytes - what no call of at most max_seqs
 * sequences needs more than, whatever prefix_len, own_cap and n_kv_heads; never
 * decreases with any of its arguments. Pieces of the prefix make at most 512 x
 * 128 rows of partial results, or one for every row of Q, those of the caches
 * 512 x 32, or one likewise. */
static inline int64_t qmm_attn_shared_workspace_max_bytes(int64_t max_seqs, int64_t n_q_heads, int64_t head_dim) {
  return (512 * (128 + 32) + 3 * max_seqs * n_q_heads) * (head_dim + 2) * 4;
}

#ifdef __cplusplus
}
#endif

#endif /* QMM_ATTN_H */
