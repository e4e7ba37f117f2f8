// Internal launch interface between the C ABI of the serving-step operators
// (serve_api.hip) and their kernels. Arguments have been validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmm_serve.h"

namespace qmm {

// A 4-bit paged cache: the place of a token's tile, and what lies where in it.
struct Kv4Cache {
  uint8_t *data;
  int64_t n_pages, page_bytes;
  int page_tokens, page_shift;  // 2^page_shift tokens
};
constexpr int kKv4Tile = 16;  // tokens per tile
__host__ __device__ constexpr int64_t kv4_tile_bytes(int64_t head_dim) { return 18 * head_dim; }

hipError_t launch_kv4_append(int type, const qmm_heads &K, const qmm_heads &V, int64_t n_tokens, int64_t n_kv_heads,
                             int64_t head_dim, bool norm, const float *weight, double eps, const int32_t *positions,
                             const double *freqs, int64_t n_freqs, int pairs, const int32_t *slots,
                             const Kv4Cache &cache, hipStream_t stream);
hipError_t launch_kv4_read(int type, const qmm_heads &K, const qmm_heads &V, int64_t n_rows, int64_t n_kv_heads,
                           int64_t head_dim, const int32_t *slots, const Kv4Cache &cache, hipStream_t stream);

// qmm_attn_kv4's split into units, which are rows, or ranges of their keys.
struct Kv4Plan {
  int64_t tiles;    // workgroups for the heads of a group
  int64_t columns;  // column tiles of a workgroup, 1 or 2
  int64_t units;    // at most
  int64_t want;     // ranges of equal length that are wanted; 0: units are rows
};
Kv4Plan kv4_plan(int64_t n_rows, int64_t n_q_heads, int64_t n_kv_heads, int64_t head_dim, int64_t cap);
int64_t kv4_workspace_bytes(const Kv4Plan &p, int64_t n_rows, int64_t n_q_heads, int64_t head_dim);
hipError_t launch_attn_kv4(int type, const qmm_heads &Q, const qmm_heads &O, int64_t n_rows, int64_t n_q_heads,
                           int64_t n_kv_heads, int64_t head_dim, const Kv4Cache &cache, const int32_t *tables,
                           int64_t table_stride, int64_t table_width, const int32_t *lengths, float scale,
                           void *workspace, hipStream_t stream);

// qmm_moe. The parts of its workspace (bytes from its start).
struct MoeLayer {
  const void *X;
  bool x_f16;
  int64_t n_tokens, k, n_ff, n_experts, n_used;
  const float *router;
  const void *gate, *up, *down;
  int type_in, type_out;
  int64_t nb1_in, nb2_in, nb1_out, nb2_out;  // row and expert strides
  bool renormalise;
  float *Y;
  int32_t *ids;    // may be null
  float *weights;  // may be null
};
int64_t moe_workspace_bytes(int64_t n_tokens, int64_t k, int64_t n_ff, int64_t n_experts, int64_t n_used);
hipError_t launch_moe(const MoeLayer &m, void *workspace, hipStream_t stream);

// qmm_sample.
struct SampleCall {
  const void *logits;
  int type;
  int64_t n_rows, vocab, row_stride;
  const float *u, *temperature;  // all but u may be null
  const int32_t *top_k;
  const float *top_p, *min_p;
  int32_t *tokens;
  float *probs;  // may be null
};
int64_t sample_workspace_bytes(int64_t n_rows, int64_t vocab);
hipError_t launch_sample(const SampleCall &c, void *workspace, hipStream_t stream);

}  // namespace qmm
