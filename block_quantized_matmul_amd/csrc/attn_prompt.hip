// Causal attention over packed prompts (qmm_attn_prompt).
//
//   O[t][h] = sum_{u <= t} softmax_u(scale Q[t][h] . K[u][g]) V[u][g],
//
// u over the tokens of t's own sequence, g = h / group. A KV head's queries
// are flattened: row x of a sequence is token x / group, head g group + x %
// group, so one tile of 128 rows reads its keys once for all the heads that
// share them, whatever the group, and a short prompt fills tiles with heads
// instead of leaving them half empty.
//
// One workgroup of four wavefronts takes a tile of 128 rows of one sequence
// and KV head, each wavefront 32 rows, over blocks of 64 keys up to the
// tile's last token; K and V of the next block are copied into LDS while the
// present one is computed (two buffers, one barrier per block). Only the
// blocks that cross the diagonal are masked. 64 KiB of LDS and at most 256
// registers let two workgroups share a CU, so that one's exponentials run
// beside the other's matrix products.
//
// The grid covers an upper bound of the tiles (the starts are device data) of
// sequences that share no token, as starts in order make them. Where starts
// are not in order, there may be more tiles, and workgroups that have seen so
// take several, one after another (attn_prompt_kernel). Each wavefront finds its
// tile by a search over the starts, 64 sequences at a time, which orders the
// tiles by length. KV heads are the fastest index, so that with 8 of them (or a
// multiple) each XCD's L2 holds the keys of its own heads only.
//
// Measured, 32 heads on 8 KV heads of 128: 8192 tokens bf16 490 to 520 us
// by box (550 GFLOP, 1.1 PFLOP/s where a large library product reaches 1.26;
// matrix cores busy in 65 % of the cycles, vector units in 56 %); 16 prompts of
// up to 950 tokens 82 us (0.54 PFLOP/s: of a tile's 17 us, 4 are its search and
// first loads, 2 the masked block and 2 the store). 16 heads of 64, three
// prompts of up to 2001 tokens, 32 us: half of a block's time is exponentials
// and other vector work, and the last third of the time only the longest
// tiles run. Eight wavefronts that split a tile's keys in two took as long
// there and longer elsewhere (8 x 1024 tokens 123 us instead of 97).
#include "attn.h"
#include "attn_core.h"
#include "launch.h"

namespace qmm {

namespace {

constexpr int kRows = 128;   // query rows per workgroup
constexpr int kThreads = 256;
// Tiles per band (find_tile). Against whole sequences one after the other: two
// prompts of 1024 36 / 30 us, 16 heads of 64 on prompts of up to 2001 35 / 32,
// 16 x 512 65 / 65; bands of one tile lose the keys' neighbours: 30, 32, 73.
constexpr int kBand = 8;

struct PromptArgs {
  const void *q, *k, *v;
  void *o;
  int64_t qt, qh, kt, kh, vt, vh, ot, oh;
  const int32_t *starts;
  int n_seqs, n_tokens, group, n_kv;
  float c;  // scale * log2(e)
};

// f over the lanes up to this one, where f(0, x) = x and x >= 0: in rows of 16
// lanes by shifts of 1, 2, 4 and 8, then the last lanes of rows 0 and 2 into the
// rows behind them, and lane 31 into the upper half (register moves, no trip
// through LDS).
template <class F> __device__ __forceinline__ int scan_lanes(int x, F f) {
  x = f(__builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false), x);
  x = f(__builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false), x);
  x = f(__builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false), x);
  x = f(__builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false), x);
  x = f(__builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false), x);
  x = f(__builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false), x);
  return x;
}
__device__ __forceinline__ int scan_sum(int x) {
  return scan_lanes(x, [](int a, int b) { return a + b; });
}
__device__ __forceinline__ int lane_sum(int x) { return __builtin_amdgcn_readlane(scan_sum(x), 63); }
__device__ __forceinline__ int lane_max(int x) {
  return __builtin_amdgcn_readlane(scan_lanes(x, [](int a, int b) { return max(a, b); }), 63);
}

// The tile with number `number` over all sequences: its sequence's first token
// and length, and its own number in it. False past the last one. Sequences are
// gone through 64 at a time. Among those, tiles go by bands of kBand of their
// numbers, the highest (the longest tiles) first, so that the launch ends with
// short ones; in a band by sequence, so that neighbours share keys, and in a
// sequence downwards. `ahead`: the number of tiles ahead of the first 64
// sequences of which one's ends are not in order; -1 if none was met.
__device__ __forceinline__ bool find_tile(const PromptArgs &a, int64_t number, int lane, int &first, int &len, int &tile,
                                          int64_t &ahead) {
  int64_t left = number;
  ahead = -1;
  for (int s0 = 0; s0 < a.n_seqs; s0 += 64) {
    const int s = s0 + lane;
    int begin = 0, n = 0, tiles = 0;
    bool in_order = true;
    if (s < a.n_seqs) {
      begin = a.starts[s];
      const int end = a.starts[s + 1];
      in_order = begin >= 0 && end >= begin && end <= a.n_tokens;
      if (in_order) n = end - begin;
      tiles = (n * a.group + kRows - 1) / kRows;
    }
    if (__builtin_expect(ahead < 0 && !__all(in_order), 0)) ahead = number - left;
    const int all = lane_sum(tiles);
    if (left >= all) {
      left -= all;
      continue;
    }
    const int index = static_cast<int>(left);
    // tiles in bands >= j: the sum over the sequences of those past j kBand;
    // the largest j for which there are more than `index`
    int low = 0, high = (lane_max(tiles) + kBand - 1) / kBand, above = 0;
    while (high - low > 1) {
      const int j = low + (high - low) / 2;
      const int more = lane_sum(max(tiles - j * kBand, 0));
      if (more > index) {
        low = j;
      } else {
        high = j, above = more;
      }
    }
    const int sum = scan_sum(min(max(tiles - low * kBand, 0), kBand));
    const int at = __builtin_ctzll(__ballot(sum > index - above));
    first = __builtin_amdgcn_readlane(begin, at);
    len = __builtin_amdgcn_readlane(n, at);
    tile = low * kBand + __builtin_amdgcn_readlane(sum, at) - 1 - (index - above);
    return true;
  }
  return false;
}

// One row over its keys 0 .. n_keys - 1, key by key, the lanes sharing the
// head's elements: for the rows of a wavefront whose tile product would let
// a non-finite value of a later token in (no ordinary call's does). Every
// key it reads is one the row attends to. Scores are raw until their difference
// is taken, as in the tiles.
template <class E, int D>
__device__ __forceinline__ void slow_row(const typename E::one *q, const typename E::one *k, int64_t kt,
                                         const typename E::one *v, int64_t vt, int n_keys, float c,
                                         typename E::one *o, int lane) {
  constexpr int kPer = D / 64;
  float x[kPer], acc[kPer], m = -__builtin_inff(), l = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) x[i] = static_cast<float>(q[kPer * lane + i]), acc[i] = 0.f;
  for (int u = 0; u < n_keys; ++u) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) s = __builtin_fmaf(x[i], static_cast<float>(k[u * kt + kPer * lane + i]), s);
#pragma unroll
    for (int d = 32; d > 0; d /= 2) s += __shfl_xor(s, d);
    const float top = fmaxf(m, s);
    const float base = top == -__builtin_inff() ? 0.f : top;
    const float alpha = __builtin_amdgcn_exp2f((m - base) * c), w = __builtin_amdgcn_exp2f((s - base) * c);
    m = top, l = l * alpha + w;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      acc[i] = acc[i] * alpha + w * static_cast<float>(v[u * vt + kPer * lane + i]);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[kPer * lane + i] = static_cast<typename E::one>(E::limit(acc[i] / l));
}

// The tile with number `number` (find_tile). False if there is none.
template <class E, int D>
__device__ __forceinline__ bool prompt_tile(const PromptArgs &a, int64_t number, uint8_t *lds, uint32_t thread,
                                            int64_t &ahead) {
  typedef typename E::one one;
  const int lane = thread & 63;
  const int wave = __builtin_amdgcn_readfirstlane(thread >> 6);
  const int g = blockIdx.x % a.n_kv;
  int first, len, tile;
  if (!find_tile(a, number, lane, first, len, tile, ahead)) return false;

  // this lane's row; rows past the sequence's last repeat it and are not stored
  const int rows = len * a.group;
  const int row = tile * kRows + wave * 32 + (lane & 31);
  const int row_in = row < rows ? row : rows - 1;
  const int token = row_in / a.group;
  typename E::v8 q[D / 16];
  const int head = g * a.group + row_in - token * a.group;
  load_rows<E, D>(static_cast<const one *>(a.q) + (first + token) * a.qt + head * a.qh, lane, q);

  const one *kb = static_cast<const one *>(a.k) + first * a.kt + g * a.kh;
  const one *vb = static_cast<const one *>(a.v) + first * a.vt + g * a.vh;
  const int tile_last = tile * kRows + kRows - 1 < rows ? tile * kRows + kRows - 1 : rows - 1;
  const int n_keys = tile_last / a.group + 1;                // keys the tile's last token sees
  const int wave_first = __builtin_amdgcn_readfirstlane(token);  // the wavefront's first and last token
  const int wave_last = __builtin_amdgcn_readlane(token, 31);

  const Copier<D, TileK<D>, E, kKeys, 4> copy_k(kb, a.kt, wave, lane);
  const Copier<D, TileV<D>, E, kKeys, 4> copy_v(vb, a.vt, wave, lane);
  AttnState<D> st;
  st.clear();
  const int mine = wave_last / kKeys + 1;
  const int full = min((wave_first + 1) / kKeys, mine - 1);
  // The first block that any wavefront of the tile may treat as masked, the
  // same for all of them, since each looks at its share of a block: that of
  // the first token's diagonal, or the one before, if it is a wavefront's last.
  const int first_masked = (tile * kRows / a.group + 1) / kKeys - 1;
  const bool any_bad = attend_blocks<E, D, true>(lds, copy_k, copy_v, n_keys, first_masked, full, mine, token + 1,
                                                 q, st, a.c, wave, lane);
  const float l = row_sum(st);
  // the row again, from the lane: nothing of it is kept in registers meanwhile
  int l2 = lane;
  asm volatile("" : "+v"(l2));
  if (!any_bad) {
    const int row2 = tile * kRows + wave * 32 + (l2 & 31);
    const int t2 = row2 / a.group;
    one *o = static_cast<one *>(a.o) + (first + t2) * a.ot + (g * a.group + row2 - t2 * a.group) * a.oh;
    store_row<E, D>(o, st, 1.f / l, l2, row2 < rows);
  } else {
    for (int r = tile * kRows + wave * 32; r < min(rows, tile * kRows + wave * 32 + 32); ++r) {
      const int t2 = r / a.group;
      const int64_t head = g * a.group + r - t2 * a.group;
      slow_row<E, D>(static_cast<const one *>(a.q) + (first + t2) * a.qt + head * a.qh, kb, a.kt, vb, a.vt, t2 + 1, a.c,
                     static_cast<one *>(a.o) + (first + t2) * a.ot + head * a.oh, l2);
    }
  }
  return true;
}

template <class E, int D>
__global__ __launch_bounds__(kThreads, 2) void attn_prompt_kernel(PromptArgs a) {
  __shared__ __align__(1024) uint8_t lds[attend_lds_bytes<D>()];
  int64_t number = blockIdx.x / a.n_kv, ahead;
  if (!prompt_tile<E, D>(a, number, lds, threadIdx.x, ahead)) return;
  if (__builtin_expect(ahead < 0, 1)) return;
  // Starts that are not in order. Up to where they are, sequences have no more
  // tiles than the grid; the tiles from there on are shared out among the
  // workgroups whose first one was among them, since those before have not seen
  // it. (If there are no such workgroups, every token was a sequence of its own
  // before, and what follows only shares their tokens.) The arguments are read
  // again, so that this costs the first tile no registers.
  do {
    auto *p = (const __attribute__((address_space(4))) PromptArgs *)__builtin_amdgcn_kernarg_segment_ptr();
    uint32_t thread = threadIdx.x;
    asm volatile("" : "+s"(p), "+v"(thread));
    const PromptArgs again{p->q,  p->k,  p->v,  p->o,      p->qt,     p->qh,       p->kt,    p->kh,   p->vt,
                           p->vh, p->ot, p->oh, p->starts, p->n_seqs, p->n_tokens, p->group, p->n_kv, p->c};
    number += gridDim.x / again.n_kv - ahead;
    __syncthreads();  // the next tile's copies go where this one's may still be read
    if (!prompt_tile<E, D>(again, number, lds, thread, ahead)) return;
  } while (true);
}

}  // namespace

hipError_t launch_attn_prompt(int type, const qmm_heads &Q, const qmm_heads &K, const qmm_heads &V, const qmm_heads &O,
                              int64_t n_tokens, int64_t n_q_heads, int64_t n_kv_heads, int64_t head_dim,
                              const int32_t *seq_starts, int64_t n_seqs, float scale, hipStream_t stream) {
  const int64_t group = n_q_heads / n_kv_heads;
  PromptArgs a{Q.data, K.data, V.data, O.data, Q.token_stride, Q.head_stride, K.token_stride, K.head_stride,
               V.token_stride, V.head_stride, O.token_stride, O.head_stride, seq_starts, static_cast<int>(n_seqs),
               static_cast<int>(n_tokens), static_cast<int>(group), static_cast<int>(n_kv_heads),
               scale * 1.4426950408889634f};
  // sum of ceil(rows_i / kRows) <= total / kRows + the sequences that have rows
  const int64_t with_rows = n_seqs < n_tokens ? n_seqs : n_tokens;
  const int64_t tiles = n_tokens * group / kRows + with_rows;
  const dim3 grid(static_cast<unsigned>(tiles * n_kv_heads));
  if (type == QMM_T_F16)
    return head_dim == 128 ? launch(attn_prompt_kernel<ElemF16, 128>, grid, dim3(kThreads), 0, stream, a)
                           : launch(attn_prompt_kernel<ElemF16, 64>, grid, dim3(kThreads), 0, stream, a);
  return head_dim == 128 ? launch(attn_prompt_kernel<ElemBF16, 128>, grid, dim3(kThreads), 0, stream, a)
                         : launch(attn_prompt_kernel<ElemBF16, 64>, grid, dim3(kThreads), 0, stream, a);
}

}  // namespace qmm
