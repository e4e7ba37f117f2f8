// Internal launch interface between the C ABI of the attention-block
// operators (attn_api.hip) and their kernels. Arguments have been validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmm_attn.h"

namespace qmm {

// qmm_lora. V's partial sums: lora_splits ranges of k, each [n_tokens][rank]
// fp32 in the workspace.
int lora_splits(int64_t n_tokens, int64_t k, int64_t rank);
hipError_t launch_lora(const void *X, bool x_f16, int64_t n_tokens, int64_t k, const void *A, const void *B,
                       int64_t n_adapters, int64_t rank, int64_t n_rows, const float *scales, const int32_t *ids,
                       const float *base, float *Y, float *partial, hipStream_t stream);

hipError_t launch_norm_rope(const qmm_head_part *parts, int n_parts, int64_t n_tokens, int64_t head_dim, float eps,
                            const int32_t *positions, const double *freqs, int64_t n_freqs, int pairs,
                            const int32_t *slots, int64_t n_slots, hipStream_t stream);

hipError_t launch_attn_prompt(int type, const qmm_heads &Q, const qmm_heads &K, const qmm_heads &V, const qmm_heads &O,
                              int64_t n_tokens, int64_t n_q_heads, int64_t n_kv_heads, int64_t head_dim,
                              const int32_t *seq_starts, int64_t n_seqs, float scale, hipStream_t stream);

// qmm_attn_shared's split: the keys of the prefix and of the own caches in
// pieces, each of which leaves its rows' partial result in the workspace.
struct SharedPlan {
  bool direct;            // few keys: no pieces, no workspace
  int64_t row_tiles;      // tiles of kSharedRows of the n_seqs * group rows of one KV head
  int64_t prefix_pieces;  // pieces of the prefix, prefix_step keys each
  int64_t prefix_step;
  int64_t own_tiles;  // tiles of kOwnRows of the group rows of one sequence and KV head
  int64_t own_pieces;  // pieces of an own cache, own_step keys each
  int64_t own_step;
  int64_t pieces() const { return prefix_pieces + own_pieces; }
};
constexpr int kSharedRows = 128;
constexpr int kOwnRows = 32;
SharedPlan shared_plan(int64_t n_seqs, int64_t prefix_len, int64_t own_cap, int64_t n_q_heads, int64_t n_kv_heads);
hipError_t launch_attn_shared(int type, const qmm_heads &Q, const qmm_heads &PK, const qmm_heads &PV,
                              int64_t prefix_len, const qmm_heads &K, const qmm_heads &V, int64_t own_cap,
                              const int32_t *lengths, const qmm_heads &O, int64_t n_seqs, int64_t n_q_heads,
                              int64_t n_kv_heads, int64_t head_dim, float scale, void *workspace, hipStream_t stream);

}  // namespace qmm
