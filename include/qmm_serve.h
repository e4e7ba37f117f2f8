/*
 * qmm_serve.h - C ABI of the operators that complete a decode step of a served
 * transformer on the AMD MI355X (gfx950), in the same libqmm.so as qmm.h and
 * qmm_attn.h:
 *
 *   qmm_kv4_append  keys (normed and rotated) and values rounded to 4-bit
 *                   blocks and stored in a paged cache;
 *   qmm_kv4_read    the values that places of such a cache hold;
 *   qmm_attn_kv4    attention of a decode batch over such a cache;
 *   qmm_moe         a whole mixture-of-experts layer for a few tokens, its
 *                   experts in the block types of the MUL_MATs;
 *   qmm_sample      the next token of every row of logits: temperature, top-k,
 *                   top-p, min-p and a given random number.
 *
 * Conventions are those of qmm_attn.h: every pointer is device memory owned by
 * the caller unless stated otherwise, nothing is retained or allocated, work
 * is enqueued on `stream` (a hipStream_t of the current device, or NULL) and
 * the call returns without waiting; every check runs on the host before
 * anything is enqueued and returns a QMM_ERR_* status. There is no global
 * state: calls on different streams may run concurrently as long as their
 * workspaces and outputs differ. Every call may be captured into a HIP graph.
 * Results repeat bit for bit for the same arguments on the same device.
 */
#ifndef QMM_SERVE_H
#define QMM_SERVE_H

#include <stdint.h>

#include "qmm_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The 4-bit paged cache ("kv4"): n_pages pages of qmm_kv4_page_bytes(...) bytes
 * one after another, 16-byte aligned, in one buffer for keys and values. A page
 * has room for page_tokens tokens (16, 32, 64, 128 or 256) of n_kv_heads heads
 * of head_dim (64 or 128) elements; slot s is place s % page_tokens of page
 * s / page_tokens. Values are Q4_0 blocks of 32 elements, w = d (code - 8) with
 * a binary16 d and codes 0 .. 15, laid out for the attention's loads: a page is
 * [n_kv_heads][page_tokens / 16] tiles of 18 * head_dim bytes, each with
 *   8 head_dim bytes  key codes: element e of the tile's token t is nibble e % 8
 *                     of dword (16 (e % 32 / 8) + t) (head_dim / 32) + e / 32
 *   8 head_dim bytes  value codes: [16][head_dim / 2], element e is nibble e % 2
 *                     (low first) of byte e / 2 of token t's row
 *   head_dim bytes    key scales, binary16 [head_dim / 32][16 tokens]
 *   head_dim bytes    value scales, likewise.
 * A page of zeros is valid (it holds zeros).
 */
#define QMM_KV4_MAX_PAGE_TOKENS 256

#define QMM_MOE_MAX_TOKENS 16
#define QMM_MOE_MAX_EXPERTS 512
#define QMM_MOE_MAX_USED 32
#define QMM_SAMPLE_MAX_VOCAB 524287

/* qmm_kv4_page_bytes - bytes of a page, or QMM_ERR_SHAPE. */
int64_t qmm_kv4_page_bytes(int64_t page_tokens, int64_t n_kv_heads, int64_t head_dim);

/*
 * qmm_kv4_append - for every token t with a slot, and every KV head:
 *   key:    x = K[t][h]; norm: x = x / sqrt(mean_e x[e]^2 + eps) * weight[e];
 *           rotated by positions[t] as qmm_norm_rope rotates (n_freqs 0: not);
 *   value:  x = V[t][h];
 *   both:   x rounded to fp32, then for each block of 32 elements
 *             m = its element of largest magnitude (the first of several),
 *             d = binary16(m / -8),  code = floor(x / d + 8.5) within 0 .. 15
 *           (d +0 and the codes 8 where d is zero), stored at slots[t].
 *   type          QMM_T_F32, QMM_T_F16 or QMM_T_BF16, of K and V
 *   K, V          n_kv_heads heads, [n_tokens] in the token axis (seq_stride
 *                 unused); strides are any >= 0, data aligned to the type
 *   norm          1: norm the keys; weight (fp32 [head_dim]) then may be given
 *   positions     int32 [n_tokens], any value; needed if n_freqs > 0
 *   freqs         HOST array of n_freqs doubles, radians per position,
 *                 magnitudes at most 64; read during the call
 *   n_freqs       0 .. head_dim / 2; pairs: QMM_ROPE_HALVES or _NEIGHBOURS
 *   slots         int32 [n_tokens]. A token whose slot lies outside
 *                 [0, n_pages * page_tokens) is not stored (so -1 leaves it out).
 *                 Two tokens with one slot leave a mixture of the two there;
 *                 other places are never touched.
 * Numerics: norm, angles and rotation in 64 bits, so the codes are those of the
 * formula (a code is decided at a border, where an fp32 rotation would choose
 * the other neighbour now and then). A block that holds an infinity, a NaN or
 * an element whose d leaves binary16's range is stored as NaNs (d a quiet NaN,
 * codes 8). K and V do not overlap the cache.
 * n_tokens, n_pages * page_tokens < 2^31; n_tokens * n_kv_heads <= 2^40.
 */
int qmm_kv4_append(int type, const qmm_heads *K, const qmm_heads *V, int64_t n_tokens, int64_t n_kv_heads,
                   int64_t head_dim, int norm, const float *weight, double eps, const int32_t *positions,
                   const double *freqs, int64_t n_freqs, int pairs, const int32_t *slots, void *cache,
                   int64_t n_pages, int64_t page_tokens, void *stream);

/*
 * qmm_kv4_read - K[i], V[i] = the keys and values at slots[i], each rounded
 * once to `type` (QMM_T_F32 is exact). A slot outside the cache reads as NaNs.
 * Either output may be NULL. Outputs have strides >= 0, are aligned to their
 * type, and their heads must not share elements (as in qmm_norm_rope).
 */
int qmm_kv4_read(int type, const qmm_heads *K, const qmm_heads *V, int64_t n_rows, int64_t n_kv_heads,
                 int64_t head_dim, const int32_t *slots, const void *cache, int64_t n_pages, int64_t page_tokens,
                 void *stream);

/*
 * qmm_attn_kv4 - attention of n_rows query tokens, each over the first
 * lengths[i] tokens of the sequence whose pages tables[i] lists:
 *   O[i][h] = sum_u w_u V_u[g],  w = softmax_u(scale * Q[i][h] . K_u[g]),
 * u = 0 .. lengths[i] - 1 at place u % page_tokens of page
 * tables[i * table_stride + u / page_tokens], g = h / (n_q_heads / n_kv_heads).
 * One query token per sequence is a decode step. Several tokens of one sequence
 * (a few drafted ones) are several rows with the same pages and lengths of their
 * own, appended first; table_stride 0 gives all rows one table.
 *   type          QMM_T_F16 or QMM_T_BF16, of Q and O
 *   Q, O          n_q_heads heads, [n_rows] in the token axis (seq_stride unused);
 *                 strides multiples of 8, 16-byte aligned
 *   n_kv_heads    a divisor of n_q_heads; head_dim 64 or 128
 *   tables        int32, table_width entries per row; table_stride >= 0
 *   lengths       int32 [n_rows]. A length of 0 gives a row of zeros
 *   scale         > 0 and < 2^127
 *   workspace     at least qmm_attn_kv4_workspace_bytes(...) bytes, 16-byte
 *                 aligned; overwritten; two calls in flight must not share one.
 *                 May be NULL when that size is 0.
 * Device data: a length outside [0, table_width * page_tokens], or a page
 * outside [0, n_pages) among those that the length reaches, gives that row
 * NaNs, and such a page is not read. Table entries past a length are not used,
 * and places past it do not reach the output whatever they hold.
 * O may be Q itself, with equal strides; otherwise it overlaps nothing.
 * Numerics: codes and Q are multiplied exactly (a Q's element below 2^-25 of the
 * row's largest counts as less than its rounding); scores, maximum and sums in
 * fp32; each weight times its value's scale is taken as two binary16 numbers (error
 * at most 2^-22 of it, or 2^-28 of the row's largest such product), and the output is
 * rounded once. A Q with an infinity or a NaN gives NaNs.
 * n_rows < 2^24, n_rows * n_q_heads < 2^24, table_width * page_tokens < 2^31,
 * n_pages >= 1 (QMM_ERR_SHAPE).
 */
int qmm_attn_kv4(int type, const qmm_heads *Q, const qmm_heads *O, int64_t n_rows, int64_t n_q_heads,
                 int64_t n_kv_heads, int64_t head_dim, const void *cache, int64_t n_pages, int64_t page_tokens,
                 const int32_t *tables, int64_t table_stride, int64_t table_width, const int32_t *lengths, float scale,
                 void *workspace, int64_t workspace_bytes, void *stream);

/* qmm_attn_kv4_workspace_bytes - the workspace qmm_attn_kv4 needs for these
 * sizes, or QMM_ERR_SHAPE. The same on every device. More rows may need less
 * (they are split less): a workspace for calls of several sizes is as large as
 * qmm_attn_kv4_workspace_max_bytes says. */
int64_t qmm_attn_kv4_workspace_bytes(int64_t n_rows, int64_t n_q_heads, int64_t n_kv_heads, int64_t head_dim,
                                     int64_t table_width, int64_t page_tokens);

/* qmm_attn_kv4_workspace_max_bytes - what no call with heads of head_dim needs
 * more than, 9 MB: rows are split where they take fewer than 1024 workgroups, into
 * at most 2048, which have at most 1024 / head_dim heads of head_dim + 4 numbers. */
static inline int64_t qmm_attn_kv4_workspace_max_bytes(int64_t head_dim) {
  return 2048 * (1024 / head_dim) * (head_dim + 4) * 4 + 16 * 1024;
}

/*
 * qmm_moe - a mixture-of-experts layer of up to QMM_MOE_MAX_TOKENS tokens:
 *   r = softmax(router X[t]) over the experts; the n_used experts of largest
 *   logits are chosen (of equal ones the first; a NaN is below all others), with
 *   weights w = r, divided by their sum if renormalise;
 *   Y[t] = sum over them of w down_e (silu(gate_e X[t]) * (up_e X[t])),
 *   silu(z) = z / (1 + e^-z).
 * More tokens are a matter for qmm_matmul_id, whose matrix-core route serves them.
 *   X           fp32 or fp16 (x_type QMM_T_F32 / QMM_T_F16) [n_tokens][k]
 *   router      fp32 [n_experts][k]
 *   n_experts   1 .. QMM_MOE_MAX_EXPERTS; n_used 1 .. QMM_MOE_MAX_USED, and at
 *               most n_experts
 *   gate, up    n_experts matrices of n_ff rows of k weights each, blocks of
 *               type_in as for qmm_matmul: row r of expert e at e *
 *               expert_stride_in + r * row_stride_in. They may be one matrix.
 *   down        n_experts matrices of k rows of n_ff weights, blocks of type_out
 *   strides     bytes, multiples of 4 (rows of an odd number of 18-, 22- or
 *               34-byte blocks are padded by two bytes, which may be read but do
 *               not count); expert strides at least the rows'
 *   k, n_ff     positive multiples of 32 (256 for the side that a Q4_K row has),
 *               below 2^24
 *   Y           fp32 [n_tokens][k], overwritten
 *   ids, weights  int32 and fp32 [n_tokens][n_used], the choice in order of
 *               falling logits; each may be NULL
 *   workspace   at least qmm_moe_workspace_bytes(...) bytes, 16-byte aligned;
 *               overwritten; two calls in flight must not share one
 * All pointers are 4-byte aligned; outputs and workspace overlap nothing else.
 * Numerics: logits are summed in 64 bits. Activations, also those between the two
 * products, are taken as two binary16 numbers each (error at most 2^-22 of the
 * value, or 2^-35), codes are exact, sums and scales fp32. An activation beyond
 * 65504, of X or of w silu(gate) up, makes its token's outputs non-finite, as in
 * qmm_matmul; non-finite values of one token stay in its row.
 */
int qmm_moe(const void *X, int x_type, int64_t n_tokens, int64_t k, const float *router, int64_t n_experts,
            int64_t n_used, int renormalise, const void *gate, const void *up, int type_in, int64_t n_ff,
            int64_t row_stride_in, int64_t expert_stride_in, const void *down, int type_out, int64_t row_stride_out,
            int64_t expert_stride_out, float *Y, int32_t *ids, float *weights, void *workspace,
            int64_t workspace_bytes, void *stream);

/* qmm_moe_workspace_bytes - the workspace qmm_moe needs for these sizes, or
 * QMM_ERR_SHAPE; grows with each of them. The same on every device. */
int64_t qmm_moe_workspace_bytes(int64_t n_tokens, int64_t k, int64_t n_ff, int64_t n_experts, int64_t n_used);

/*
 * qmm_sample - for every row i of logits z, in the order of falling logits (of
 * equal ones the lower index first), with p_j proportional to
 * e^(z_j / temperature):
 *   1. top_k > 0 keeps the first top_k tokens;
 *   2. top_p < 1 keeps the shortest beginning of them whose share of their
 *      probability reaches top_p, one token at least;
 *   3. min_p > 0 keeps those with p_j >= min_p times the first one's;
 *   4. tokens[i] is the first of what is left at which the sum of its
 *      probabilities, as shares of what is left, exceeds u.
 * A temperature that is not above 0 takes the first token.
 *   logits       QMM_T_F32, QMM_T_F16 or QMM_T_BF16, [n_rows] rows of vocab
 *                elements row_stride >= 0 apart, aligned to the type. A NaN counts
 *                as -infinity, which has no probability; where the largest is
 *                infinite, the infinite ones share it equally
 *   vocab        1 .. QMM_SAMPLE_MAX_VOCAB
 *   u            fp32 [n_rows], from [0, 1): below (and NaN) it counts as 0, above
 *                as the largest number below 1
 *   temperature, top_p, min_p  fp32 [n_rows], top_k int32 [n_rows]; each may be
 *                NULL for 1, 1, 0 and 0: none. A NaN for top_p or min_p is none, a
 *                min_p above 1 counts as 1
 *   tokens       int32 [n_rows]; -1 for a row without a probability (every logit
 *                -infinity or NaN)
 *   probs        fp32 [n_rows], the token's share of what step 4 chooses from
 *                (NaN beside -1); may be NULL
 * Numerics: a weight is exact to 2^-44 of the row's largest, and sums of weights
 * are exact; a token whose probability is below 2^-45 of the largest is not chosen.
 *   workspace    at least qmm_sample_workspace_bytes(n_rows, vocab) bytes, 16-byte
 *                aligned; overwritten; two calls in flight must not share one
 * n_rows < 2^22; n_rows == 0 is a no-op.
 */
int qmm_sample(const void *logits, int type, int64_t n_rows, int64_t vocab, int64_t row_stride, const float *u,
               const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
               int32_t *tokens, float *probs, void *workspace, int64_t workspace_bytes, void *stream);

/* qmm_sample_workspace_bytes - the workspace qmm_sample needs, or QMM_ERR_SHAPE;
 * grows with both. The same on every device. */
int64_t qmm_sample_workspace_bytes(int64_t n_rows, int64_t vocab);

#ifdef __cplusplus
}
#endif

#endif /* QMM_SERVE_H */
