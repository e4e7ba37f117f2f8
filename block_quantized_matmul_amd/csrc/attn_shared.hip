// Attention of a decode batch over a shared prefix and each sequence's own
// cache (qmm_attn_shared).
//
// One softmax over both key ranges; it is computed in pieces of keys. A piece
// leaves, for every row (sequence, query head), its normalised output O_i, its
// reference m_i and its sum of weights l_i relative to that, and the join is
//   O = sum_i f_i O_i / sum_i f_i,  f_i = l_i 2^(c m_i - c m),  m = max_i m_i.
// (One logarithm of c m_i + log2 l_i would lose l_i where scores are large.)
//
// The prefix is read once for all sequences: the rows of all sequences and of
// the heads that share a KV head are flattened (row x: sequence x / group,
// head g group + x % group) into equal tiles of at most 128, four wavefronts
// of 32 rows on blocks of 64 keys, as the prompt kernel runs without its mask.
// A sequence's own cache serves only `group` rows, so there a workgroup's four
// wavefronts share one tile of 32 rows and split the piece's keys, each with
// blocks of 32 keys of its own (copied into its own part of LDS, no barrier),
// and join at the end through LDS.
//
// Both kinds of pieces are workgroups of one launch and alternate in it, since
// the prefix's are bound by the matrix cores and the caches' by memory. A
// second launch joins the pieces.
//
// Measured, 32 heads on 8 KV heads of 128, bf16: 48 sequences on a prefix of
// 32000 and caches of up to 2047 93 us, 6 of them the join (332 MB, 3.6 TB/s);
// 4 sequences on 500 + 130 keys 11 us in one launch (latency).
#include "attn.h"
#include "attn_core.h"
#include "launch.h"

#include <algorithm>

namespace qmm {

namespace {

constexpr int kThreads = 256;
constexpr int kOwnKeys = 32;     // keys per block of one wavefront, own cache
constexpr int kMinPiece = 256;   // keys
constexpr int kWantGroups = 512; // workgroups: two per CU on 256 CUs
constexpr int kWantBoth = 384;   // of each kind of piece, where there are both
// No pieces (attn_direct_kernel) up to so many keys and so many reads of prefix
// keys by all sequences. Measured with 32 heads on 8 KV heads of 128, us
// without and with pieces: 4 sequences on 500 + 192 keys 11.3 / 17.2, on 1000
// + 192 15.1 / 18.2, on 2000 + 192 24.1 / 16.8; 48 on 500 + 256 18.6 / 23.2,
// on 1000 + 256 24.0 / 21.9; 128 on 500 + 256 43.7 / 47.3.
constexpr int64_t kDirectKeys = 1024;
constexpr int64_t kDirectReads = 65536;

struct SharedArgs {
  const void *q, *pk, *pv, *k, *v;
  void *o;
  int64_t qt, qh, pkt, pkh, pvt, pvh, ks, kt, kh, vs, vt, vh, ot, oh;
  const int32_t *lengths;
  float *part_o;  // [pieces][n_seqs * n_q_heads][D]
  float *part_m;  // [pieces][n_seqs * n_q_heads], and the same for l
  float *part_l;
  int n_seqs, n_heads, group, n_kv, prefix_len, own_cap;
  int row_tiles, tile_rows, prefix_pieces, prefix_step, own_tiles, own_pieces, own_step;
  float c;  // scale * log2(e)
};

// A row's partial result; an empty piece (no keys) has m = -infinity, l = 0 and
// zeros for its output.
template <int D>
__device__ __forceinline__ void store_partial(const SharedArgs &a, int piece, int seq, int head,
                                              const AttnState<D> &st, float l, int lane) {
  const int64_t at = (static_cast<int64_t>(piece) * a.n_seqs + seq) * a.n_heads + head;
  const float f = l > 0.f || l != l ? 1.f / l : 0.f;
  float *o = a.part_o + at * D;
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4_t *>(o + 32 * dt + 8 * i + 4 * (lane >> 5)) =
          float4_t{st.o[dt][4 * i] * f, st.o[dt][4 * i + 1] * f, st.o[dt][4 * i + 2] * f, st.o[dt][4 * i + 3] * f};
  if (lane < 32) a.part_m[at] = st.m, a.part_l[at] = l;
}

template <class E, int D>
__device__ __forceinline__ void prefix_piece(const SharedArgs &a, int item, int g, uint8_t *lds, int wave, int lane) {
  typedef typename E::one one;
  const int rt = item % a.row_tiles;
  const int piece = item / a.row_tiles;
  const int rows = a.n_seqs * a.group;
  const int row = rt * a.tile_rows + wave * 32 + (lane & 31);
  const bool busy = wave * 32 < a.tile_rows && rt * a.tile_rows + wave * 32 < rows;  // else it only copies
  const int row_in = row < rows ? row : rows - 1;
  const int seq = row_in / a.group, head = g * a.group + row_in % a.group;
  typename E::v8 q[D / 16];
  load_rows<E, D>(static_cast<const one *>(a.q) + seq * a.qt + head * a.qh, lane, q);

  const int first = piece * a.prefix_step;
  const int n_keys = min(a.prefix_step, a.prefix_len - first);
  const one *kb = static_cast<const one *>(a.pk) + first * a.pkt + g * a.pkh;
  const one *vb = static_cast<const one *>(a.pv) + first * a.pvt + g * a.pvh;
  const Copier<D, TileK<D>, E, kKeys, 4> copy_k(kb, a.pkt, wave, lane);
  const Copier<D, TileV<D>, E, kKeys, 4> copy_v(vb, a.pvt, wave, lane);
  AttnState<D> st;
  st.clear();
  const int blocks = (n_keys + kKeys - 1) / kKeys;
  attend_blocks<E, D, false>(lds, copy_k, copy_v, n_keys, 0, busy ? blocks - 1 : -1, busy ? blocks : 0, n_keys, q, st,
                             a.c, wave, lane);
  const float l = row_sum(st);
  if (busy && row < rows) store_partial<D>(a, piece, seq, head, st, l, lane);
}

// 32 rows over keys 0 .. n_keys - 1, on one of four wavefronts: this one takes
// blocks wave, wave + 4, ... of 32 keys through its own part of LDS, no
// barrier needed. The next block's K is copied while this one's weights are
// computed, its V while its scores are.
template <class E, int D>
__device__ __forceinline__ void own_blocks(const typename E::one *kb, int64_t k_stride, const typename E::one *vb,
                                           int64_t v_stride, int n_keys, typename E::v8 q[D / 16], AttnState<D> &st,
                                           float c, uint8_t *lds, int wave, int lane) {
  constexpr int kTile = kOwnKeys * D * 2, kCopies = kTile / 1024;  // copies: instructions of a K or a V tile
  const uint32_t at = lds_addr(lds) + wave * 2 * kTile;
  const int blocks = (n_keys + kOwnKeys - 1) / kOwnKeys;
  const Copier<D, TileK<D>, E, kOwnKeys, 1> copy_k(kb, k_stride, 0, lane);
  const Copier<D, TileV<D>, E, kOwnKeys, 1> copy_v(vb, v_stride, 0, lane);
  auto load_k = [&](int b) {
    if (b < blocks) copy_k(b * kOwnKeys, n_keys - b * kOwnKeys, at, lane);
  };
  auto load_v = [&](int b) {
    if (b < blocks) copy_v(b * kOwnKeys, n_keys - b * kOwnKeys, at + kTile, lane);
  };
  load_k(wave);
  load_v(wave);
  for (int b = wave; b < blocks; b += 4) {
    wait_loads<kCopies>();  // K has landed, V may be on its way
#pragma unroll
    for (int i = 0; i < D / 16; ++i) asm volatile("" : "+v"(q[i]));
    float16_t s[1];
    typename E::v8 p[2];
    scores<E, D, 1>(at, q, s, lane);
    interleave<D / 16, 4, 1, 0, 0>();
    wait_reads();
    load_k(b + 4);
    const int left = n_keys - b * kOwnKeys;
    if (left < kOwnKeys) mask_scores<1>(s, left, lane);
    follow_max<D, 1>(st, row_max<1>(s), c, s);
    weights<E, D, 1>(s, st, c, p);
    if (b + 4 < blocks)
      wait_loads<kCopies>();  // V has landed, the next K may be on its way
    else
      wait_loads<0>();
    __builtin_amdgcn_sched_barrier(0);
    add_values<E, D, 1>(v_addr<D>(at + kTile, lane), p, st);
    interleave<2 * (D / 32), 3, 2, 0, 0>();
    wait_reads();
    load_v(b + 4);
  }
}

// Joins the states of four wavefronts on the same rows through LDS: the
// largest m, then the sums in wavefront order. Wavefront 3 ends up with the
// whole, and its l is the row's, not a lane's half.
template <int D>
__device__ __forceinline__ void join_wavefronts(AttnState<D> &st, float c, uint8_t *lds, int wave, int lane) {
  float l = row_sum(st);
  __syncthreads();
  float *ml = reinterpret_cast<float *>(lds);        // [4][32][2]
  float *os = reinterpret_cast<float *>(lds) + 256;  // [32][D + 1], added to in turn
  if (lane < 32) {
    ml[(wave * 32 + lane) * 2] = st.m;
    ml[(wave * 32 + lane) * 2 + 1] = l;
  }
  __syncthreads();
  const int col = lane & 31;
  float top = -__builtin_inff();
#pragma unroll
  for (int w = 0; w < 4; ++w) top = fmaxf(top, ml[(w * 32 + col) * 2]);
  l = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) l += ml[(w * 32 + col) * 2 + 1] * rescaling(ml[(w * 32 + col) * 2], top, c);
  const float f = rescaling(st.m, top, c);
  st.m = top, st.l = l;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (wave == w) {
#pragma unroll
      for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          float *x = os + col * (D + 1) + 32 * dt + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
          st.o[dt][r] = st.o[dt][r] * f + (w > 0 ? *x : 0.f);
          if (w < 3) *x = st.o[dt][r];
        }
    }
    if (w < 3) __syncthreads();
  }
}

template <class E, int D>
__device__ __forceinline__ void own_piece(const SharedArgs &a, int item, int g, uint8_t *lds, int wave, int lane) {
  typedef typename E::one one;
  const int rt = item % a.own_tiles;
  const int seq = item / a.own_tiles % a.n_seqs;
  const int piece = item / a.own_tiles / a.n_seqs;
  const int row = rt * kOwnRows + (lane & 31);  // of the group
  const int head = g * a.group + min(row, a.group - 1);
  const int len = __builtin_amdgcn_readfirstlane(a.lengths[seq]);
  const int first = piece * a.own_step;
  // a length outside [0, own_cap] is answered by the join
  const int n_keys = len < 0 || len > a.own_cap ? 0 : min(max(len - first, 0), a.own_step);
  AttnState<D> st;
  st.clear();
  if (n_keys > 0) {
    typename E::v8 q[D / 16];
    load_rows<E, D>(static_cast<const one *>(a.q) + seq * a.qt + head * a.qh, lane, q);
    own_blocks<E, D>(static_cast<const one *>(a.k) + seq * a.ks + first * a.kt + g * a.kh, a.kt,
                     static_cast<const one *>(a.v) + seq * a.vs + first * a.vt + g * a.vh, a.vt, n_keys, q, st, a.c,
                     lds, wave, lane);
  }
  join_wavefronts<D>(st, a.c, lds, wave, lane);
  if (wave == 3 && row < a.group) store_partial<D>(a, a.prefix_pieces + piece, seq, head, st, st.l, lane);
}

// Few keys: one workgroup per (sequence, KV head, 32 rows of the group) goes
// over the prefix and the cache and writes the result, without partial
// results to join. It reads the prefix once per sequence (from L2), so this is
// for short prefixes and small batches.
template <class E, int D> __global__ __launch_bounds__(kThreads, 2) void attn_direct_kernel(SharedArgs a) {
  typedef typename E::one one;
  __shared__ __align__(1024) uint8_t lds[4 * 2 * kOwnKeys * D * 2];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = blockIdx.x % a.n_kv, rt = blockIdx.x / a.n_kv % a.own_tiles, seq = blockIdx.x / a.n_kv / a.own_tiles;
  const int row = rt * kOwnRows + (lane & 31);
  const int head = g * a.group + min(row, a.group - 1);
  const int len = a.own_cap > 0 ? __builtin_amdgcn_readfirstlane(a.lengths[seq]) : 0;
  const bool bad = len < 0 || len > a.own_cap;
  AttnState<D> st;
  st.clear();
  typename E::v8 q[D / 16];
  load_rows<E, D>(static_cast<const one *>(a.q) + seq * a.qt + head * a.qh, lane, q);
  if (a.prefix_len > 0)
    own_blocks<E, D>(static_cast<const one *>(a.pk) + g * a.pkh, a.pkt, static_cast<const one *>(a.pv) + g * a.pvh,
                     a.pvt, a.prefix_len, q, st, a.c, lds, wave, lane);
  if (len > 0 && !bad)
    own_blocks<E, D>(static_cast<const one *>(a.k) + seq * a.ks + g * a.kh, a.kt,
                     static_cast<const one *>(a.v) + seq * a.vs + g * a.vh, a.vt, len, q, st, a.c, lds, wave, lane);
  join_wavefronts<D>(st, a.c, lds, wave, lane);
  if (wave != 3) return;
  // without a key a row of zeros; with keys, but no weight (every score -infinity), 0 / 0
  const float f = bad ? __builtin_bit_cast(float, 0x7FC00000u) : a.prefix_len == 0 && len == 0 ? 0.f : 1.f / st.l;
  store_row<E, D>(static_cast<one *>(a.o) + seq * a.ot + head * a.oh, st, f, lane, row < a.group);
}

template <class E, int D>
__global__ __launch_bounds__(kThreads, 2) void attn_shared_kernel(SharedArgs a) {
  __shared__ __align__(1024) uint8_t lds[attend_lds_bytes<D>()];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // KV heads are the fastest index (their keys stay in one XCD's L2); the two
  // kinds of pieces alternate, in proportion
  const int g = blockIdx.x % a.n_kv;
  const int64_t unit = blockIdx.x / a.n_kv;
  const int prefix_units = a.prefix_pieces * a.row_tiles, units = prefix_units + a.own_pieces * a.n_seqs * a.own_tiles;
  const int before = static_cast<int>(unit * prefix_units / units);
  if (static_cast<int>((unit + 1) * prefix_units / units) > before)
    prefix_piece<E, D>(a, before, g, lds, wave, lane);
  else
    own_piece<E, D>(a, static_cast<int>(unit) - before, g, lds, wave, lane);
}

// One workgroup per (sequence, query head): the weighted sum of its pieces.
// Thread (part, four elements): every kParts-th piece, eight on their way at
// once, then the parts through LDS; all in a fixed order.
template <class E, int D> __global__ __launch_bounds__(kThreads) void attn_join_kernel(SharedArgs a) {
  constexpr int kFours = D / 4, kParts = kThreads / kFours;
  __shared__ float4_t sums[kParts][kFours];
  __shared__ float weights[kParts];
  const int seq = blockIdx.x / a.n_heads, head = blockIdx.x % a.n_heads;
  const int64_t rows = static_cast<int64_t>(a.n_seqs) * a.n_heads;
  const int pieces = a.prefix_pieces + a.own_pieces;
  const int part = threadIdx.x / kFours, e = threadIdx.x % kFours;
  const int len = a.own_cap > 0 ? a.lengths[seq] : 0;
  const int lane = threadIdx.x & 63;
  float top = -__builtin_inff();
  for (int i = lane; i < pieces; i += 64) top = fmaxf(top, a.part_m[i * rows + blockIdx.x]);
#pragma unroll
  for (int d = 32; d > 0; d /= 2) top = fmaxf(top, __shfl_xor(top, d));
  float sum = 0.f;
  float4_t o{};
  for (int i0 = part; i0 < pieces; i0 += 8 * kParts) {
    float m[8], l[8];
    float4_t x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t at = (i0 + k * kParts < pieces ? i0 + k * kParts : part) * rows + blockIdx.x;
      m[k] = a.part_m[at], l[k] = a.part_l[at];
      x[k] = *reinterpret_cast<const float4_t *>(a.part_o + at * D + 4 * e);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (i0 + k * kParts >= pieces) continue;
      const float f = l[k] * rescaling(m[k], top, a.c);
      sum += f;
      o += f * x[k];
    }
  }
  sums[part][e] = o;
  if (e == 0) weights[part] = sum;
  __syncthreads();
  if (part != 0) return;
#pragma unroll
  for (int k = 1; k < kParts; ++k) o += sums[k][e], sum += weights[k];
  const float f = a.prefix_len == 0 && len == 0 ? 0.f : 1.f / sum;  // with keys, but no weight, 0 / 0
  const bool bad = len < 0 || len > a.own_cap;
  typename E::v4 out;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    out[k] = static_cast<typename E::one>(bad ? __builtin_bit_cast(float, 0x7FC00000u) : E::limit(o[k] * f));
  *reinterpret_cast<typename E::v4 *>(static_cast<typename E::one *>(a.o) + seq * a.ot + head * a.oh + 4 * e) = out;
}

template <class E, int D> hipError_t run(const SharedArgs &a, int64_t items, bool direct, hipStream_t stream) {
  if (direct)
    return launch(attn_direct_kernel<E, D>, dim3(static_cast<unsigned>(items)), dim3(kThreads), 0, stream, a);
  if (items > 0) {
    const hipError_t e =
        launch(attn_shared_kernel<E, D>, dim3(static_cast<unsigned>(items)), dim3(kThreads), 0, stream, a);
    if (e != hipSuccess) return e;
  }
  const dim3 rows(static_cast<unsigned>(a.n_seqs * a.n_heads));
  return launch(attn_join_kernel<E, D>, rows, dim3(kThreads), 0, stream, a);
}

}  // namespace

// Pieces: enough workgroups to fill the GPU, but at least kMinPiece keys in
// each, since every piece costs its rows' partial result. Lengths are device
// data, so the pieces of the caches follow from their number, not from how long
// each is: from kWantGroups (or kWantBoth) caches and KV heads on, a cache is one
// workgroup's, and a long one among short ones is that workgroup's chain while
// the GPU is otherwise idle (32 heads on 8 of 128: 64 caches of 500 25 us, with
// one of 32000 among them 312). (The header's
// qmm_attn_shared_workspace_max_bytes follows from kWantGroups and the tiles'
// rows.)
SharedPlan shared_plan(int64_t n_seqs, int64_t prefix_len, int64_t own_cap, int64_t n_q_heads, int64_t n_kv_heads) {
  const int64_t group = n_q_heads / n_kv_heads;
  SharedPlan p{};
  p.row_tiles = (n_seqs * group + kSharedRows - 1) / kSharedRows;
  p.own_tiles = (group + kOwnRows - 1) / kOwnRows;
  // (without a prefix, where the caches fill the GPU there would be one piece of
  // each, which only adds the join; us without and with it: 64 caches of 2000
  // 96 / 101, of 8000 356 / 362, of 32000 1392 / 1400, of 500 25 / 30)
  p.direct = (prefix_len + own_cap <= kDirectKeys && prefix_len * n_seqs <= kDirectReads) ||
             (prefix_len == 0 && n_seqs * n_kv_heads * p.own_tiles >= kWantGroups);
  if (p.direct) return p;
  const int64_t groups = prefix_len > 0 && own_cap > 0 ? kWantBoth : kWantGroups;
  auto cut = [groups](int64_t keys, int64_t items, int64_t block, int64_t &pieces, int64_t &step) {
    if (keys == 0) return;
    const int64_t want = std::max<int64_t>(1, std::min((groups + items - 1) / items, keys / kMinPiece));
    step = ((keys + want - 1) / want + block - 1) / block * block;
    pieces = (keys + step - 1) / step;
  };
  cut(prefix_len, p.row_tiles * n_kv_heads, kKeys, p.prefix_pieces, p.prefix_step);
  cut(own_cap, n_seqs * n_kv_heads * p.own_tiles, kOwnKeys, p.own_pieces, p.own_step);
  return p;
}

hipError_t launch_attn_shared(int type, const qmm_heads &Q, const qmm_heads &PK, const qmm_heads &PV,
                              int64_t prefix_len, const qmm_heads &K, const qmm_heads &V, int64_t own_cap,
                              const int32_t *lengths, const qmm_heads &O, int64_t n_seqs, int64_t n_q_heads,
                              int64_t n_kv_heads, int64_t head_dim, float scale, void *workspace, hipStream_t stream) {
  const SharedPlan p = shared_plan(n_seqs, prefix_len, own_cap, n_q_heads, n_kv_heads);
  SharedArgs a{};
  a.q = Q.data, a.pk = PK.data, a.pv = PV.data, a.k = K.data, a.v = V.data, a.o = O.data;
  a.qt = Q.token_stride, a.qh = Q.head_stride;
  a.pkt = PK.token_stride, a.pkh = PK.head_stride, a.pvt = PV.token_stride, a.pvh = PV.head_stride;
  a.ks = K.seq_stride, a.kt = K.token_stride, a.kh = K.head_stride;
  a.vs = V.seq_stride, a.vt = V.token_stride, a.vh = V.head_stride;
  a.ot = O.token_stride, a.oh = O.head_stride;
  a.lengths = lengths;
  a.part_o = static_cast<float *>(workspace);
  a.part_m = a.part_o + p.pieces() * n_seqs * n_q_heads * head_dim;
  a.part_l = a.part_m + p.pieces() * n_seqs * n_q_heads;
  a.n_seqs = static_cast<int>(n_seqs), a.n_heads = static_cast<int>(n_q_heads);
  a.group = static_cast<int>(n_q_heads / n_kv_heads), a.n_kv = static_cast<int>(n_kv_heads);
  a.prefix_len = static_cast<int>(prefix_len), a.own_cap = static_cast<int>(own_cap);
  // equal tiles, of whole wavefronts' rows
  const int64_t row_waves = (n_seqs * a.group + 31) / 32;
  a.row_tiles = static_cast<int>(p.row_tiles);
  a.tile_rows = static_cast<int>((row_waves + p.row_tiles - 1) / p.row_tiles) * 32;
  a.prefix_pieces = static_cast<int>(p.prefix_pieces);
  a.prefix_step = static_cast<int>(p.prefix_step), a.own_tiles = static_cast<int>(p.own_tiles);
  a.own_pieces = static_cast<int>(p.own_pieces), a.own_step = static_cast<int>(p.own_step);
  a.c = scale * 1.4426950408889634f;
  const int64_t items = (p.direct ? n_seqs * p.own_tiles
                                  : p.prefix_pieces * p.row_tiles + p.own_pieces * n_seqs * p.own_tiles) * n_kv_heads;
  auto by_dim = [&](auto elem) {
    typedef decltype(elem) E;
    return head_dim == 128 ? run<E, 128>(a, items, p.direct, stream) : run<E, 64>(a, items, p.direct, stream);
  };
  return type == QMM_T_F16 ? by_dim(ElemF16{}) : by_dim(ElemBF16{});
}

}  // namespace qmm
