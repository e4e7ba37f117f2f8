// A whole mixture-of-experts layer for a few tokens (qmm_moe).
//
//   r = softmax(R x), the `used` largest;  y = sum_e r_e D_e h_e,
//   h_e = silu(G_e x) * (U_e x)
//
// Bound by memory for few tokens: the chosen experts' blocks are read once. Three to
// five launches: the router's logits and the activations' operands; the choice, where
// gate's and up's workgroups are too many to make it themselves; gate and up with the
// activation; down with the sum over experts; and for more than one token the sum over
// workgroups that share rows of down.
//
// The columns of an expert's products are the tokens that chose it, at most 8: an
// expert of more has two sets, and its blocks are read twice. (With all tokens as
// columns of every expert, 16 tokens on 8 experts took 357 us instead of 254.) The
// routing weight is multiplied into h, so down's sums over experts are additions to
// the tokens' rows, in order, by each wavefront for its part of the (expert, n_ff)
// axis; there is no output per expert.
//
// Operands. v_mfma_f32_16x16x32_f16 sums a block of 32 weights of 16 rows with 16
// columns. An activation x takes two columns, hi = fp16(x) and lo = fp16(2^11 (x -
// hi)), so that it is not rounded (to 2^-22, or absolutely to 2^-35); they are
// prepared once, in operand order, by the launch before. A 4-bit code n becomes a
// half by a shift and a mask, 16 + n (n in the upper bits of the mantissa; in the
// lower ones it would be 1024 + n or a subnormal, and the sums a hundred times
// less exact); -(16 + 8) times the activations' sum, one more product that the
// rows' groups share, starts a Q4_0 row's sum. A block's scale multiplies the
// block's 16 x 16 sums in fp32.
//
// Weights are copied to LDS as they lie in memory, 16 bytes per lane, a quad of
// blocks (256 weights) of a wavefront's 16 or 32 rows at a time, one quad ahead, and
// read from there as operands. A quad's operands of a token are 1 KiB, as much as
// the weights of 7 rows, so the wavefronts of a workgroup that have different rows of
// the same stages copy them together; those that share rows add their sums at the end.
//
// Measured (one MI355X): 1 token, 2 of 8 experts of 14336 x 4096 Q4_0: 4.9 + 37 + 23
// us, 198 MB at 3.8 TB/s in the products (copies alone, in pieces of 144 bytes a row,
// take 31 + 20; of 288 bytes 28 + 17, but leave room for half as many wavefronts). 5
// tokens, 6 of 64 experts of 1408 x 2048, Q4_0 and Q8_0: 4.2 + 5.2 + 28 + 21 + 4.6 us.
// 16 tokens, 2 of 8 experts of 14336 x 4096 Q4_K: 9 + 5 + 160 + 95 + 5 us, 793 MB at 3.1
// TB/s; vector instructions fill 90 % of the cycles, matrix cores 60 %. (Scales of a
// Q4_K quad computed once and handed to the lanes that need them saved no time.)
#include "attn_core.h"
#include "gemv_common.h"
#include "launch.h"
#include "serve.h"

#include <algorithm>

namespace qmm {

namespace {

constexpr int kInnerWaves = 4;  // wavefronts of a workgroup
constexpr int kSetTokens = 8;  // of a set: its columns are a tile of the matrix cores
constexpr int kRouteThreads = 1024;
constexpr int kLogitThreads = 256;
constexpr int kLogitTokens = 4;  // tokens of a logit workgroup
constexpr float kLoScale = 2048.f;
constexpr int kLdsBytes = 160 * 1024;  // of a CU

// ------------------------------------------------------------- operands

// Where element i of a block stands among the operands: place j of lane group g.
struct Spot {
  int g, j;
};
__device__ __forceinline__ Spot spot_of(int qtype, int i) {
  if (qtype == QMM_TYPE_Q4_K) return {i / 8, (i & 4) | (i & 1) << 1 | (i >> 1 & 1)};
  if (qtype == QMM_TYPE_Q4_0 || qtype == QMM_TYPE_Q4_1) return {i % 16 / 4, (i & 1) << 2 | (i >> 1 & 1) | (i / 16) << 1};
  if (qtype == QMM_TYPE_Q8_0) return {i / 8, i & 7};
  return {i % 16 / 4, (i & 3) | (i / 16) << 2};
}
// The two halves of an activation.
__device__ __forceinline__ void split(float x, _Float16 &hi, _Float16 &lo) {
  hi = static_cast<_Float16>(x);
  // (an infinite hi makes the sum it enters infinite or NaN by itself)
  const float rest = (x - static_cast<float>(hi)) * kLoScale;
  lo = static_cast<_Float16>(__builtin_fabsf(rest) < __builtin_inff() ? rest : 0.f);
}
// Operand halves: [block][g][column][j], columns 2 t and 2 t + 1 of token t; 1 KiB per quad and token.
__device__ __forceinline__ int64_t operand_at(int64_t block, int columns, int column, int g) {
  return ((block * 4 + g) * columns + column) * 8;
}
constexpr int kQuadOps = 1024;  // bytes, of a token

template <int QT> struct Quad {
  static constexpr int chunks = Block<QT>::bytes / 2;  // 16-byte pieces of a row's 8 blocks
  static constexpr int row = chunks * 16;
};

// One block's codes as an operand, with its scale (and its term of the columns' sums).
struct BlockOp {
  half8_t codes;
  float d, m;
};
// Four-bit codes n as the halves 16 + n (n in the mantissa's upper bits): those
// whose nibbles lie `up` bits below the place, or above it if negative.
template <int UP> __device__ __forceinline__ uint32_t codes_at(uint32_t v) {
  return ((UP > 0 ? v << (UP & 31) : v >> (-UP & 31)) & 0x03C003C0u) | 0x4C004C00u;
}
// A dword's nibbles in the order 0, 4, 1, 5, 2, 6, 3, 7.
__device__ __forceinline__ half8_t nibbles(uint32_t v) {
  return __builtin_bit_cast(half8_t, u32x4_t{codes_at<6>(v), codes_at<2>(v), codes_at<-2>(v), codes_at<-6>(v)});
}
// The two blocks of pair u of the row at rb (LDS), for lane group g.
template <int QT> __device__ __forceinline__ void pair_ops(const uint8_t *rb, int u, int g, BlockOp op[2]) {
  auto ld = [&](int off) { return *reinterpret_cast<const uint32_t *>(rb + off); };
  if constexpr (QT == QMM_TYPE_Q4_K) {
    const uint32_t h0 = ld(0), s0 = ld(4), s1 = ld(8), s2 = ld(12);
    const float d = half_bits_to_float(h0 & 0xFFFFu), dmin = half_bits_to_float(h0 >> 16);
    const uint32_t a0 = ld(16 + 32 * u + 8 * g), a1 = ld(20 + 32 * u + 8 * g);
    op[0].codes = __builtin_bit_cast(half8_t, u32x4_t{codes_at<6>(a0), codes_at<-2>(a0), codes_at<6>(a1), codes_at<-2>(a1)});
    op[1].codes = __builtin_bit_cast(half8_t, u32x4_t{codes_at<2>(a0), codes_at<-6>(a0), codes_at<2>(a1), codes_at<-6>(a1)});
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t sc, mn;
      q4k_scale_min(s0, s1, s2, 2 * u + h, sc, mn);
      op[h].d = d * static_cast<float>(sc);
      op[h].m = __builtin_fmaf(-dmin, static_cast<float>(mn), -16.f * op[h].d);
    }
  } else {
    const uint8_t *p = rb + u * (2 * Block<QT>::bytes);
    auto lp = [&](int off) { return *reinterpret_cast<const uint32_t *>(p + off); };
    if constexpr (QT == QMM_TYPE_Q4_0) {
      const uint32_t a0 = lp(4 * g), a1 = lp(4 * g + 4), b = lp(20 + 4 * g), d0 = lp(0), d1 = lp(16);
      op[0].codes = nibbles(shift16(a0, a1)), op[1].codes = nibbles(b);
      op[0].d = half_bits_to_float(d0 & 0xFFFFu), op[1].d = half_bits_to_float(d1 >> 16);
    } else if constexpr (QT == QMM_TYPE_Q4_1) {
      const uint32_t a = lp(4 + 4 * g), b = lp(24 + 4 * g), dm0 = lp(0), dm1 = lp(20);
      op[0].codes = nibbles(a), op[1].codes = nibbles(b);
      op[0].d = half_bits_to_float(dm0 & 0xFFFFu), op[1].d = half_bits_to_float(dm1 & 0xFFFFu);
      op[0].m = __builtin_fmaf(-16.f, op[0].d, half_bits_to_float(dm0 >> 16));
      op[1].m = __builtin_fmaf(-16.f, op[1].d, half_bits_to_float(dm1 >> 16));
    } else if constexpr (QT == QMM_TYPE_Q5_0) {
      const uint32_t w0 = lp(0), w1 = lp(4), a0 = lp(4 + 4 * g), a1 = lp(8 + 4 * g);
      const uint32_t w5 = lp(20), h1 = lp(24), b = lp(28 + 4 * g);
      op[0].codes = gemv_codes5<QT>(shift16(a0, a1), shift16(w0, w1), 4 * g);
      op[1].codes = gemv_codes5<QT>(b, h1, 4 * g);
      op[0].d = half_bits_to_float(w0 & 0xFFFFu), op[1].d = half_bits_to_float(w5 >> 16);
    } else if constexpr (QT == QMM_TYPE_Q5_1) {
      const uint32_t dm0 = lp(0), h0 = lp(4), a = lp(8 + 4 * g), dm1 = lp(24), h1 = lp(28), b = lp(32 + 4 * g);
      op[0].codes = gemv_codes5<QT>(a, h0, 4 * g), op[1].codes = gemv_codes5<QT>(b, h1, 4 * g);
      op[0].d = half_bits_to_float(dm0 & 0xFFFFu), op[0].m = half_bits_to_float(dm0 >> 16);
      op[1].d = half_bits_to_float(dm1 & 0xFFFFu), op[1].m = half_bits_to_float(dm1 >> 16);
    } else {
      const uint32_t a0 = lp(8 * g), a1 = lp(8 * g + 4), a2 = lp(8 * g + 8);
      const uint32_t b0 = lp(36 + 8 * g), b1 = lp(40 + 8 * g), d0 = lp(0), d1 = lp(32);
      op[0].codes = gemv_codes<QT>(shift16(a0, a1), shift16(a1, a2)), op[1].codes = gemv_codes<QT>(b0, b1);
      op[0].d = half_bits_to_float(d0 & 0xFFFFu), op[1].d = half_bits_to_float(d1 >> 16);
    }
  }
}
// The constant operand whose product with the activations is what a Q4_0 row's sum
// starts with, -(16 + 8) times their sum, or what a minimum multiplies, their sum.
template <int QT> __device__ __forceinline__ half8_t sum_operand() {
  const _Float16 c = static_cast<_Float16>(QT == QMM_TYPE_Q4_0 ? -24.f : 1.f);
  return half8_t{c, c, c, c, c, c, c, c};
}
template <int QT> constexpr bool has_min() { return QTraits<QT>::has_min || QTraits<QT>::kquant; }

// --------------------------------------------------------------- streaming

// A wavefront's rows: G groups of 16, from which a lane copies piece lane + 64 j
// of every quad. Rows past the last repeat it.
//
// The blocks behind the last whole quad, the tail, are copied as the last 16-byte
// pieces of the row, which begin before the tail where its length is no multiple
// of 16, so that nothing behind the row is read. (Rows shorter than that go dword
// by dword, take_short.)
template <int QT, int G> struct Rows {
  static constexpr int kPieces = 16 * G * Quad<QT>::chunks;
  static constexpr int kCopies = (kPieces + 63) / 64;
  static constexpr int kStage = kPieces * 16;   // bytes of LDS
  static constexpr int kStages = 2;             // quads in use or on their way
  int64_t off[kCopies];  // from the expert's matrix (group 0's), of this lane's pieces in quad 0
  bool on_last;          // whether this lane has a piece in the last copy
  int tail_at, tail_pieces, tail_skip;  // of a row: its tail's first piece's byte, pieces, and bytes before the tail

  // With two groups they are the same rows of two matrices, `apart` bytes from each other.
  __device__ __forceinline__ Rows(int64_t nb1, int row0, int n_rows, int blocks, int64_t apart, int lane) {
#pragma unroll
    for (int j = 0; j < kCopies; ++j) {
      const int c = min(64 * j + lane, kPieces - 1), r = c / Quad<QT>::chunks;
      const int64_t row = min(row0 + r % 16, n_rows - 1);
      off[j] = row * nb1 + 16 * (c % Quad<QT>::chunks) + (r / 16 ? apart : 0);
    }
    on_last = 64 * (kCopies - 1) + lane < kPieces;
    const int bytes = (blocks % 8 * Block<QT>::bytes + 3) / 4 * 4;
    tail_pieces = (bytes + 15) / 16;
    tail_skip = 16 * tail_pieces - bytes;
    tail_at = blocks / 8 * Quad<QT>::row - tail_skip;
  }
  __device__ __forceinline__ void copy(const uint8_t *w, int q, bool tail, uint32_t lds, int lane) const {
    const uint8_t *p = w + (tail ? tail_at : static_cast<int64_t>(q) * Quad<QT>::row);
#pragma unroll
    for (int j = 0; j < kCopies; ++j) {
      if (j < kCopies - 1 || kPieces % 64 == 0 || on_last) {
        const uint8_t *from = p + off[j];
        if (tail) from -= 16 * max((64 * j + lane) % Quad<QT>::chunks - (tail_pieces - 1), 0);
        asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "s"(lds + 1024 * j)
                     : "memory", "m0");
      }
    }
  }
};

// The operands of some of the tokens: pieces of 16 bytes, of every lane group of
// every block two of each token, in memory among those of all tokens (`stride`
// columns), or by themselves.
struct Ops {
  const _Float16 *p;
  uint32_t columns, stride;
  uint64_t tokens;   // in order, 4 bits each
  uint32_t inverse;  // 2^16 / columns, rounded up: exact quotients of pieces of a quad, of which there are at most 1024
  __device__ __forceinline__ Ops(const _Float16 *ops, int count, uint64_t which, int of_tokens)
      : p(ops), columns(2 * count), stride(2 * of_tokens), tokens(which), inverse((65536 + 2 * count - 1) / (2 * count)) {}
  __device__ __forceinline__ Ops(const _Float16 *ops, int count)
      : p(ops), columns(2 * count), stride(2 * count), tokens(0), inverse(0) {}
  // Where piece i of quad q is.
  __device__ __forceinline__ const uint8_t *piece(int q, uint32_t i) const {
    const uint8_t *quad = reinterpret_cast<const uint8_t *>(p) + static_cast<int64_t>(q) * (32 * 16) * stride;
    if (stride == columns) return quad + 16 * i;
    const uint32_t group = i * inverse >> 16, column = i - group * columns;
    return quad + 16 * (group * stride + 2 * (static_cast<uint32_t>(tokens >> (2 * (column & ~1u))) & 15u) + (column & 1u));
  }
};

// A quad in LDS times its activations (there too), into the rows' sums. `valid`: blocks that exist.
template <int QT, int G>
__device__ __forceinline__ void take_quad(const uint8_t *stage, const uint8_t *ops, int columns, int valid,
                                          float4_t acc[G], int lane) {
  const int g = lane >> 4;
  const uint8_t *rb = stage + (lane & 15) * Quad<QT>::row;
  const uint8_t *xp = ops + 16 * (g * columns + min(lane & 15, columns - 1));  // the others repeat the last, for nothing
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (2 * u >= valid) break;
    BlockOp op[G][2];
#pragma unroll
    for (int k = 0; k < G; ++k) pair_ops<QT>(rb + k * 16 * Quad<QT>::row, u, g, op[k]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (2 * u + h >= valid) break;
      const half8_t x = *reinterpret_cast<const half8_t *>(xp + (2 * u + h) * 64 * columns);
      float4_t start{}, sums{};
      if constexpr (QT == QMM_TYPE_Q4_0) start = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, sum_operand<QT>(), start, 0, 0, 0);
      if constexpr (has_min<QT>()) sums = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, sum_operand<QT>(), sums, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const float4_t part = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, op[k][h].codes, start, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[k][e] = __builtin_fmaf(op[k][h].d, part[e], acc[k][e]);
          if constexpr (has_min<QT>()) acc[k][e] = __builtin_fmaf(op[k][h].m, sums[e], acc[k][e]);
        }
      }
    }
  }
}

// Rows of fewer than 8 blocks, copied dword by dword so that nothing behind a
// row's last dword is read, and their activations. The wavefront has `ops` for itself.
template <int QT, int G>
__device__ __forceinline__ void take_short(const uint8_t *w, int64_t nb1, int row0, int n_rows, int64_t apart, int blocks,
                                           const Ops &x, uint8_t *stage, uint8_t *ops, float4_t acc[G], int lane) {
  const int dwords = (blocks * Block<QT>::bytes + 3) / 4;
  wait_reads();  // of what lay in this place before
  for (int i = lane; i < 16 * G * dwords; i += 64) {
    const int r = i / dwords, at = i % dwords;
    const int64_t row = min(row0 + r % 16, n_rows - 1);
    const uint8_t *from = w + row * nb1 + (r >= 16 ? apart : 0) + 4 * at;
    *reinterpret_cast<uint32_t *>(stage + r * Quad<QT>::row + 4 * at) = *reinterpret_cast<const uint32_t *>(from);
  }
  for (int i = lane; i < blocks * 4 * static_cast<int>(x.columns); i += 64)
    *reinterpret_cast<half8_t *>(ops + 16 * i) = *reinterpret_cast<const half8_t *>(x.piece(0, i));
  wait_reads();
  take_quad<QT, G>(stage, ops, x.columns, blocks, acc, lane);
}

struct Stage {
  const uint8_t *w;
  int q, index;  // quad, and index of the expert
  Ops ops;
};

// All wavefronts are here; what each has waited for itself is there for all.
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// A workgroup's place in LDS: the wavefronts' rings of weights, then stage by stage
// the activations of each part of the stages. (A pair of blocks is read whole, also
// where a tail ends with its first, which may be a few bytes behind the last ring.)
template <class R, int WAVES> struct Lds {
  uint8_t *base;
  int parts, tokens;
  static constexpr int kRings = WAVES * R::kStages * R::kStage;
  __device__ __forceinline__ uint8_t *weights(int wave, int slot) const { return base + (wave * R::kStages + slot) * R::kStage; }
  __device__ __forceinline__ uint8_t *ops(int part, int slot) const {
    return base + kRings + (slot * parts + part) * tokens * kQuadOps;
  }
};

// n stages (at most `most`, the same for the workgroup) through LDS, from `first`
// on: a stage is a quad of an expert's matrix, and advance(s) goes to the next. The wavefronts of a part, `peer` of
// `peers`, have different rows of the same stages and copy its activations together.
// Behind an expert's last stage comes flush(its index).
template <int QT, int G, class R, class L, class Advance, class Flush>
__device__ __forceinline__ void stream(const R &rows, const Stage &first, const Advance &advance, const Flush &flush, int n,
                                       int most, int blocks, const L &lds, int part, int peer, int peers, bool live,
                                       float4_t acc[G], int wave, int lane) {
  const int whole = blocks / 8;
  auto copy = [&](const Stage &s, int slot) {
    rows.copy(s.w, s.q, s.q == whole, lds_addr(lds.weights(wave, slot)), lane);
    const int pieces = min(8, blocks - 8 * s.q) * 4 * s.ops.columns;  // (of a tail there are fewer)
    for (int k = 64 * peer; k < pieces; k += 64 * peers)
      asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(
                       s.ops.piece(s.q, min(k + lane, pieces - 1))),
                   "s"(lds_addr(lds.ops(part, slot)) + 16 * k)
                   : "memory", "m0");
  };
  Stage next = first;
  if (n > 0) copy(next, 0);
  for (int i = 0; i < most; ++i) {
    wait_loads<0>();
    meet();
    const Stage s = next;
    if (i + 1 < n) {
      advance(next);
      copy(next, (i + 1) & 1);
    }
    if (i < n && live) {
      const uint8_t *ops = lds.ops(part, i & 1);
      const bool tail = s.q == whole;
      take_quad<QT, G>(lds.weights(wave, i & 1) + (tail ? rows.tail_skip : 0), ops, s.ops.columns, tail ? blocks % 8 : 8,
                           acc, lane);
      if (i + 1 == n || s.q == (blocks + 7) / 8 - 1) flush(s.index);
    }
    wait_reads();
  }
}

// Adds the sums of the `parts` wavefronts that share rows, in order; the first of
// them has the result. (Wavefront: part + parts * unit.)
template <int G> __device__ __forceinline__ void add_parts(float4_t acc[G], uint8_t *lds, int parts, int wave, int lane) {
  if (parts == 1) return;
  __syncthreads();
  float4_t *at = reinterpret_cast<float4_t *>(lds) + lane;
#pragma unroll
  for (int k = 0; k < G; ++k) at[(wave * G + k) * 64] = acc[k];
  __syncthreads();
  if (wave % parts != 0) return;
  for (int s = 1; s < parts; ++s)
#pragma unroll
    for (int k = 0; k < G; ++k) acc[k] += at[((wave + s) * G + k) * 64];
}

// ----------------------------------------------------------------- kernels

struct Table {  // what the choice leaves for the products
  int n_active;
  int pad[3];
};
struct Active {  // a set: an expert that was chosen,
  int expert, count;  // by so many tokens (of more than 8, some: it has two sets),
  uint64_t tokens;    // these, in order, 4 bits each
};
struct MoeArgs {
  const void *x;
  const float *router;
  const uint8_t *gate, *down;
  int64_t up_apart;  // up - gate, in bytes
  int64_t nb1_in, nb2_in, nb1_out, nb2_out;
  float *y;
  int32_t *ids;
  float *weights;
  // workspace
  double *logits;     // [n_tokens][n_experts]
  Table *table;
  Active *active;     // [most active], in order
  float *share;       // [most active][kSetTokens] routing weights of its tokens
  _Float16 *x_ops, *h_ops;  // operands of x, and of h set by set, of its tokens alone
  int64_t h_step;     // halves of one set's h
  int n_tokens, set_tokens, most, route_here, k, n_ff, n_experts, n_used, renormalise, x_f16, type_in, type_out;
  int logit_groups;   // workgroups of the first launch that compute logits; the others prepare operands
  int parts_in, parts_out;  // wavefronts of a workgroup that share rows
  int sums_out;             // where the tokens' sums lie in LDS
  int groups_out;           // workgroups that share rows (their sums go to `partial`)
  float *partial;           // [groups_out][n_tokens][k]
};

__device__ __forceinline__ float load_x(const MoeArgs &a, int64_t at) {
  return a.x_f16 ? static_cast<float>(static_cast<const _Float16 *>(a.x)[at]) : static_cast<const float *>(a.x)[at];
}

// Logits in 64 bits (a choice is decided at a border), and x as operands.
__global__ __launch_bounds__(kLogitThreads) void moe_prepare_kernel(MoeArgs a) {
  __shared__ double sums[kLogitThreads / 64][kLogitTokens];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (static_cast<int>(blockIdx.x) < a.logit_groups) {
    const int e = blockIdx.x % a.n_experts, t0 = blockIdx.x / a.n_experts * kLogitTokens;
    const float *r = a.router + static_cast<int64_t>(e) * a.k;
    double s[kLogitTokens] = {};
#pragma unroll 4
    for (int i = 4 * threadIdx.x; i < a.k; i += 4 * kLogitThreads) {
      const float4_a4 w = *reinterpret_cast<const float4_a4 *>(r + i);
#pragma unroll
      for (int t = 0; t < kLogitTokens; ++t) {
        const int64_t at = static_cast<int64_t>(min(t0 + t, a.n_tokens - 1)) * a.k + i;
        float x[4];
        if (a.x_f16) {
          const half4_a4 h = *reinterpret_cast<const half4_a4 *>(static_cast<const _Float16 *>(a.x) + at);
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = static_cast<float>(h[j]);
        } else {
          const float4_a4 f = *reinterpret_cast<const float4_a4 *>(static_cast<const float *>(a.x) + at);
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = f[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) s[t] = __builtin_fma(static_cast<double>(w[j]), static_cast<double>(x[j]), s[t]);
      }
    }
#pragma unroll
    for (int t = 0; t < kLogitTokens; ++t) {
#pragma unroll
      for (int d = 32; d > 0; d /= 2) s[t] += __shfl_xor(s[t], d);
      if (lane == 0) sums[wave][t] = s[t];
    }
    __syncthreads();
    const int t = threadIdx.x;
    if (t < kLogitTokens && t0 + t < a.n_tokens) {
      double total = 0.;
#pragma unroll
      for (int w = 0; w < kLogitThreads / 64; ++w) total += sums[w][t];
      a.logits[static_cast<int64_t>(t0 + t) * a.n_experts + e] = total;
    }
    return;
  }
  // a thread: one element of a block, all tokens' in turn
  const int64_t i = static_cast<int64_t>(blockIdx.x - a.logit_groups) * kLogitThreads + threadIdx.x;
  if (i >= static_cast<int64_t>(a.k) * a.n_tokens) return;
  const int t = static_cast<int>(i / a.k), e = static_cast<int>(i % a.k);
  const Spot s = spot_of(a.type_in, e % 32);
  _Float16 hi, lo;
  split(load_x(a, i), hi, lo);
  a.x_ops[operand_at(e / 32, 2 * a.n_tokens, 2 * t, s.g) + s.j] = hi;
  a.x_ops[operand_at(e / 32, 2 * a.n_tokens, 2 * t + 1, s.g) + s.j] = lo;
}

// The choice, by a workgroup: an expert's rank among a token's is the number of
// larger logits, of equal ones before it (a NaN is below all others), and those
// of rank below n_used are chosen. The sets and their tokens' weights are left in LDS,
// and where `write`, in the workspace and the outputs.
struct Routed {
  const Active *sets;
  const float *share;  // [sets][kSetTokens]
  int n;
};
constexpr int64_t route_lds(int64_t n, int64_t experts, int64_t used, int64_t most) {
  return n * experts * 8 + most * (static_cast<int64_t>(sizeof(Active)) + kSetTokens * 4) + n * used * 8 + (2 * experts + 1) * 4;
}
// An integer of a logit's order; a NaN's is below all others.
__device__ __forceinline__ int64_t order_of(double x) {
  const int64_t bits = __builtin_bit_cast(int64_t, x + 0.);  // (-0 is 0)
  return x != x ? INT64_MIN : bits < 0 ? bits ^ INT64_MAX : bits;
}
template <int THREADS> __device__ __forceinline__ Routed route(const MoeArgs &a, uint8_t *smem, bool write) {
  const int n = a.n_tokens, experts = a.n_experts, items = n * experts;
  int64_t *l = reinterpret_cast<int64_t *>(smem);                    // [n][experts] order_of
  Active *sets = reinterpret_cast<Active *>(l + items);              // [most]
  float *share = reinterpret_cast<float *>(sets + a.most);           // [most][kSetTokens]
  float *w = share + a.most * kSetTokens;                            // [n][n_used]
  int *id = reinterpret_cast<int *>(w + n * a.n_used);               // [n][n_used]
  int *place = id + n * a.n_used;                                    // [experts + 1], the last: sets in all
  uint32_t *by = reinterpret_cast<uint32_t *>(place + experts + 1);  // [experts] a bit for each token
  for (int i = threadIdx.x; i < items; i += THREADS) l[i] = order_of(a.logits[i]);
  for (int i = threadIdx.x; i < experts; i += THREADS) by[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < items; i += THREADS) {
    const int t = i / experts, e = i % experts;
    const int64_t mine = l[i], *row = l + t * experts;
    int rank = 0;
    for (int k = 0; k < experts; ++k) rank += row[k] > mine || (row[k] == mine && k < e);
    if (rank < a.n_used) {
      id[t * a.n_used + rank] = e;
      atomicOr(&by[e], 1u << t);
    }
  }
  __syncthreads();
  // weights: a wavefront per token
  const int lane = threadIdx.x & 63;
  for (int t = threadIdx.x >> 6; t < n; t += THREADS / 64) {
    const double *row = a.logits + static_cast<int64_t>(t) * experts;
    const double top = row[id[t * a.n_used]];
    float sum = 0.f;
    if (a.renormalise) {
      for (int k = lane; k < a.n_used; k += 64) sum += expf(static_cast<float>(row[id[t * a.n_used + k]] - top));
    } else {
      for (int k = lane; k < experts; k += 64) sum += expf(static_cast<float>(row[k] - top));
    }
#pragma unroll
    for (int d = 32; d > 0; d /= 2) sum += __shfl_xor(sum, d);
    for (int k = lane; k < a.n_used; k += 64) {
      const int e = id[t * a.n_used + k];
      const float v = expf(static_cast<float>(row[e] - top)) / sum;
      w[t * a.n_used + k] = v;
      if (write && a.ids) a.ids[t * a.n_used + k] = e;
      if (write && a.weights) a.weights[t * a.n_used + k] = v;
    }
  }
  // the sets in order, by the first wavefront
  if (threadIdx.x < 64) {
    int before = 0;
    for (int e0 = 0; e0 < experts; e0 += 64) {
      const int e = e0 + lane;
      uint32_t tokens = e < experts ? by[e] : 0;
      const int count = __popc(tokens);
      const uint64_t some = __ballot(count > 0), many = __ballot(count > kSetTokens), in_front = (uint64_t{1} << lane) - 1;
      int at = before + __popcll(some & in_front) + __popcll(many & in_front);
      if (count > 0) place[e] = at;
      while (tokens) {
        Active set{e, 0, 0};
        for (; tokens && set.count < kSetTokens; tokens &= tokens - 1)
          set.tokens |= static_cast<uint64_t>(__builtin_ctz(tokens)) << (4 * set.count++);
        if (write) a.active[at] = set;
        sets[at++] = set;
      }
      before += __popcll(some) + __popcll(many);
    }
    if (lane == 0) {
      place[experts] = before;
      if (write) a.table->n_active = before;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n * a.n_used; i += THREADS) {
    const int t = i / a.n_used, e = id[i];
    const int at = place[e] * kSetTokens + __popc(by[e] & ((1u << t) - 1));  // (its second set comes right behind)
    share[at] = w[i];
    if (write) a.share[at] = w[i];
  }
  __syncthreads();
  return {sets, share, place[experts]};
}
__global__ __launch_bounds__(kRouteThreads) void moe_route_kernel(MoeArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  route<kRouteThreads>(a, smem, true);
}

// Columns 4 g + e: hi and lo of tokens 2 g and 2 g + 1.
__device__ __forceinline__ float token_value(const float4_t &acc, int which) {
  return __builtin_fmaf(acc[2 * which + 1], 1.f / kLoScale, acc[2 * which]);
}

// gate, up and their product: blockIdx.y is the set, a unit 16 rows of both.
template <int QT> using InnerRows = Rows<QT, 2>;
template <int QT> __global__ __launch_bounds__(64 * kInnerWaves, 4) void moe_inner_kernel(MoeArgs a) {
  typedef InnerRows<QT> R;
  typedef Lds<R, kInnerWaves> L;
  extern __shared__ __align__(1024) uint8_t smem[];
  Active mine;
  float shares[2];  // of the set's tokens 2 g and 2 g + 1
  {
    const int at = blockIdx.y * kSetTokens + 2 * ((threadIdx.x & 63) >> 4);
    if (a.route_here) {
      const Routed routed = route<64 * kInnerWaves>(a, smem, blockIdx.x == 0 && blockIdx.y == 0);
      if (static_cast<int>(blockIdx.y) >= routed.n) return;
      const Active &set = routed.sets[blockIdx.y];
      mine.expert = __builtin_amdgcn_readfirstlane(set.expert), mine.count = __builtin_amdgcn_readfirstlane(set.count);
      mine.tokens = static_cast<uint64_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(set.tokens >> 32))) << 32 |
                    static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(set.tokens)));
#pragma unroll
      for (int k = 0; k < 2; ++k) shares[k] = routed.share[at + k];
      __syncthreads();  // the rings take its place
    } else {
      if (static_cast<int>(blockIdx.y) >= a.table->n_active) return;
      mine = a.active[blockIdx.y];
#pragma unroll
      for (int k = 0; k < 2; ++k) shares[k] = a.share[at + k];
    }
  }
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int parts = a.parts_in, part = wave % parts, peer = wave / parts, peers = kInnerWaves / parts;
  const int row0 = 16 * (blockIdx.x * peers + peer);
  const bool live = row0 < a.n_ff;  // (else it copies for the others)
  const int blocks = a.k / 32;
  const uint8_t *w = a.gate + static_cast<int64_t>(mine.expert) * a.nb2_in;
  const Ops x(a.x_ops, mine.count, mine.tokens, a.n_tokens);
  const L lds{smem, parts, a.set_tokens};
  float4_t acc[2] = {};
  if (blocks >= 8) {
    const int stages = (blocks + 7) / 8;
    const int lo = stages * part / parts, hi = stages * (part + 1) / parts;
    const R rows(a.nb1_in, row0, a.n_ff, blocks, a.up_apart, lane);
    stream<QT, 2>(rows, Stage{w, lo, 0, x}, [](Stage &s) { ++s.q; }, [](int) {}, hi - lo,
                      (stages + parts - 1) / parts, blocks, lds, part, peer, peers, live, acc, wave, lane);
  } else if (live && part == 0) {
    take_short<QT, 2>(w, a.nb1_in, row0, a.n_ff, a.up_apart, blocks, x, lds.weights(wave, 0),
                          smem + L::kRings + wave * a.set_tokens * kQuadOps, acc, lane);
  }
  add_parts<2>(acc, smem, parts, wave, lane);
  if (part != 0 || !live) return;
  const int row = row0 + (lane & 15), g = lane >> 4;
  if (row >= a.n_ff) return;
  const Spot s = spot_of(a.type_out, row % 32);
  _Float16 *h = a.h_ops + blockIdx.y * a.h_step;
  const int columns = 2 * mine.count;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int token = 2 * g + k;  // among the set's
    if (token >= mine.count) continue;
    const float share = shares[k];
    const float gate = token_value(acc[0], k), up = token_value(acc[1], k);
    const float v = share == 0.f ? 0.f : gate / (1.f + expf(-gate)) * up * share;
    _Float16 hi, lo;
    qmm::split(v, hi, lo);
    h[operand_at(row / 32, columns, 2 * token, s.g) + s.j] = hi;
    h[operand_at(row / 32, columns, 2 * token + 1, s.g) + s.j] = lo;
  }
}

// down: 16 rows over all active experts' quads, split evenly between the parts of
// the workgroups that share rows. Columns are an expert's tokens, so its sums are
// added to the tokens' own (in LDS, each wavefront's) behind its last quad.
template <int QT> using OuterRows = Rows<QT, 1>;
template <int QT, int WAVES> __global__ __launch_bounds__(64 * WAVES, 4) void moe_outer_kernel(MoeArgs a) {
  typedef OuterRows<QT> R;
  typedef Lds<R, WAVES> L;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int parts = a.parts_out, part = wave % parts, peer = wave / parts, peers = WAVES / parts;
  const int group = blockIdx.x % a.groups_out;
  const int row0 = 16 * (blockIdx.x / a.groups_out * peers + peer);
  const bool live = row0 < a.k;
  const int n_active = __builtin_amdgcn_readfirstlane(a.table->n_active);
  const int blocks = a.n_ff / 32;
  const L lds{smem, parts, a.set_tokens};
  float *sums = reinterpret_cast<float *>(smem + a.sums_out) + wave * a.n_tokens * 16;  // [n_tokens][16 rows]
  for (int i = lane; i < 16 * a.n_tokens; i += 64) sums[i] = 0.f;
  float4_t acc[1] = {};
  auto flush = [&](int index) {
    const Active &e = a.active[index];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = 2 * g + k;
      if (i < e.count) sums[static_cast<int>(e.tokens >> (4 * i) & 15) * 16 + (lane & 15)] += token_value(acc[0], k);
    }
    acc[0] = float4_t{};
  };
  auto matrix = [&](int index) { return a.down + static_cast<int64_t>(a.active[index].expert) * a.nb2_out; };
  auto operands = [&](int index) { return Ops(a.h_ops + index * a.h_step, a.active[index].count); };
  const int all_parts = parts * a.groups_out, my_part = group * parts + part;
  if (blocks >= 8) {
    const int stages = (blocks + 7) / 8;
    const int64_t all = static_cast<int64_t>(n_active) * stages;
    const int lo = __builtin_amdgcn_readfirstlane(static_cast<int>(all * my_part / all_parts));
    const int hi = __builtin_amdgcn_readfirstlane(static_cast<int>(all * (my_part + 1) / all_parts));
    const R rows(a.nb1_out, row0, a.k, blocks, 0, lane);
    const int e0 = min(__builtin_amdgcn_readfirstlane(lo / stages), n_active - 1);
    auto advance = [&](Stage &s) {
      if (++s.q < stages) return;
      s.q = 0, ++s.index;
      s.w = matrix(s.index), s.ops = operands(s.index);
    };
    stream<QT, 1>(rows, Stage{matrix(e0), lo - e0 * stages, e0, operands(e0)}, advance, flush, hi - lo,
                  static_cast<int>((all + all_parts - 1) / all_parts), blocks, lds, part, peer, peers, live, acc, wave, lane);
  } else if (live) {
    for (int e = my_part; e < n_active; e += all_parts) {
      take_short<QT, 1>(matrix(e), a.nb1_out, row0, a.k, 0, blocks, operands(e), lds.weights(wave, 0),
                            smem + L::kRings + wave * a.set_tokens * kQuadOps, acc, lane);
      flush(e);
    }
  }
  __syncthreads();
  if (part != 0) return;
  float *y = a.groups_out > 1 ? a.partial + static_cast<int64_t>(group) * a.n_tokens * a.k : a.y;
  for (int i = lane; i < 16 * a.n_tokens; i += 64) {
    const int row = row0 + i % 16;
    if (row >= a.k) continue;
    float sum = sums[i];
    for (int s = 1; s < parts; ++s) sum += sums[s * a.n_tokens * 16 + i];
    y[static_cast<int64_t>(i / 16) * a.k + row] = sum;
  }
}

// y: the sums of the workgroups that share rows, in order.
__global__ __launch_bounds__(256) void moe_add_kernel(const float *partial, int groups, int64_t n, float *y) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  float sum = 0.f;
  for (int g = 0; g < groups; g += 4) {  // (a power of two, 4 at least)
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = partial[(g + k) * n + i];
    sum += (v[0] + v[1]) + (v[2] + v[3]);
  }
  y[i] = sum;
}

int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }
// Sets, at most.
int64_t most_active(int64_t n_tokens, int64_t n_experts, int64_t n_used) {
  return std::min(n_experts, n_tokens * n_used) + std::min(n_experts, n_tokens * n_used / (kSetTokens + 1));
}
int64_t set_tokens(int64_t n_tokens) { return std::min<int64_t>(n_tokens, kSetTokens); }

// How a product's rows and stages are divided. `peers` wavefronts with different
// rows share a stage's activations, as many as leave each about so many tokens' to
// copy (and so that LDS holds three workgroups' or four: with twice as many tokens each
// down's 16 tokens took 120 us instead of 94). The other wavefronts of a workgroup
// take other parts of the stages, and so do other workgroups, where rows are few.
int pieces_for(int64_t n_tokens) { return n_tokens <= 4 ? 1 : 2; }
struct Plan {
  int waves, peers, parts, groups;
};
// down: one token's rows by 16 wavefronts each (8 for Q8_0, whose rings are larger);
// of more tokens' by as many workgroups as make about 4 a CU, since only wavefronts
// with different rows can share the tokens.
Plan outer_plan(int64_t n_tokens, int64_t k, int qtype) {
  Plan p{n_tokens > 1 ? 4 : qtype == QMM_TYPE_Q8_0 ? 8 : 16, 1, 1, 1};
  const int64_t units = (k + 15) / 16;
  while (p.peers * pieces_for(n_tokens) < set_tokens(n_tokens)) p.peers *= 2;
  p.parts = p.waves / p.peers;
  if (n_tokens > 1) p.groups = 4;
  while (n_tokens > 1 && p.groups < 16 && (units + p.peers - 1) / p.peers * p.groups * 2 <= 1024) p.groups *= 2;
  return p;
}

// At most, in elements, and growing with both sizes: a plan of more than 4 groups has at most 1024 workgroups.
int64_t most_partial(int64_t n_tokens, int64_t k) {
  if (n_tokens == 1) return 0;
  const int64_t peers = outer_plan(n_tokens, k, 0).peers;
  return n_tokens * std::max(4 * k, std::min(16 * k, 1024 * 16 * peers));
}

// The rings and the activations, or what take_short or the partial sums use instead.
template <class R, int WAVES> int lds_bytes(const Plan &p, int64_t n_tokens, bool short_rows) {
  return Lds<R, WAVES>::kRings + static_cast<int>(set_tokens(n_tokens)) * kQuadOps * (short_rows ? WAVES : R::kStages * p.parts);
}

// gate and up, of `most` sets: workgroups of few rows, but in one round if that is
// possible, of as many as a CU's registers (four) and LDS hold: two of Q8_0, whose rings
// are larger. (1 token, 8 of 256 experts of 2048 x 4096 Q4_0: 51 us in one round, 63 in
// a third more workgroups than run at once; 2 of 8 of 14336 x 4096 Q8_0 90 and 95.)
template <int QT> struct InnerPlan : Plan {
  int64_t blocks;  // workgroups of a set
  bool one_round;
  InnerPlan(const MoeArgs &a, int64_t most) : Plan{kInnerWaves, 1, 1, 1} {
    const int64_t units = (a.n_ff + 15) / 16;
    while (peers * pieces_for(a.n_tokens) < set_tokens(a.n_tokens)) peers *= 2;
    for (;; peers *= 2) {
      parts = waves / peers, blocks = (units + peers - 1) / peers;
      one_round = blocks * most <= 256 * std::min(4, kLdsBytes / lds(a));
      if (one_round || peers == waves) return;
    }
  }
  int lds(const MoeArgs &a) const { return lds_bytes<InnerRows<QT>, kInnerWaves>(*this, a.n_tokens, a.k < 256); }
};

// Where a thread has a logit at most, and the workgroups run all at once, each makes
// the choice for itself (1 token of 8 experts: 37 us instead of 35 + 5 and a launch; 16
// tokens, in many rounds: 180 instead of 160 + 5).
template <int QT> hipError_t run_inner(MoeArgs &a, hipStream_t stream) {
  const InnerPlan<QT> p(a, a.most);
  const int64_t route = route_lds(a.n_tokens, a.n_experts, a.n_used, a.most);
  a.parts_in = p.parts;
  a.route_here = a.n_tokens * a.n_experts <= 64 * kInnerWaves && p.one_round;
  if (!a.route_here) {
    const hipError_t e = launch(moe_route_kernel, dim3(1), dim3(kRouteThreads), static_cast<size_t>(route), stream, a);
    if (e != hipSuccess) return e;
  }
  const dim3 grid(static_cast<unsigned>(p.blocks), static_cast<unsigned>(a.most));
  return launch(moe_inner_kernel<QT>, grid, dim3(64 * kInnerWaves),
                static_cast<size_t>(std::max<int64_t>(p.lds(a), a.route_here ? route : 0)), stream, a);
}
template <int QT, int WAVES> hipError_t run_outer(MoeArgs a, hipStream_t stream) {
  const Plan p = outer_plan(a.n_tokens, a.k, QT);
  const dim3 grid(static_cast<unsigned>(((a.k + 15) / 16 + p.peers - 1) / p.peers * p.groups));
  a.sums_out = lds_bytes<OuterRows<QT>, WAVES>(p, a.n_tokens, a.n_ff < 256);
  const hipError_t e = launch(moe_outer_kernel<QT, WAVES>, grid, dim3(64 * WAVES),
                              static_cast<size_t>(a.sums_out + WAVES * a.n_tokens * 64), stream, a);
  if (e != hipSuccess || p.groups == 1) return e;
  const int64_t n = static_cast<int64_t>(a.n_tokens) * a.k;
  return launch(moe_add_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, stream, a.partial, p.groups, n, a.y);
}

}  // namespace

int64_t moe_workspace_bytes(int64_t n_tokens, int64_t k, int64_t n_ff, int64_t n_experts, int64_t n_used) {
  const int64_t most = most_active(n_tokens, n_experts, n_used);
  return round16(n_tokens * n_experts * 8) + 16 + most * static_cast<int64_t>(sizeof(Active)) + most * kSetTokens * 4 + n_tokens * k * 4 +
         most * set_tokens(n_tokens) * n_ff * 4 + most_partial(n_tokens, k) * 4;
}

hipError_t launch_moe(const MoeLayer &m, void *workspace, hipStream_t stream) {
  const int64_t most = most_active(m.n_tokens, m.n_experts, m.n_used);
  MoeArgs a{};
  a.x = m.X, a.x_f16 = m.x_f16, a.router = m.router;
  a.gate = static_cast<const uint8_t *>(m.gate), a.down = static_cast<const uint8_t *>(m.down);
  a.up_apart = static_cast<const uint8_t *>(m.up) - a.gate;
  a.nb1_in = m.nb1_in, a.nb2_in = m.nb2_in, a.nb1_out = m.nb1_out, a.nb2_out = m.nb2_out;
  a.y = m.Y, a.ids = m.ids, a.weights = m.weights;
  uint8_t *p = static_cast<uint8_t *>(workspace);
  a.logits = reinterpret_cast<double *>(p), p += round16(m.n_tokens * m.n_experts * 8);
  a.table = reinterpret_cast<Table *>(p), p += 16;
  a.active = reinterpret_cast<Active *>(p), p += most * sizeof(Active);
  a.share = reinterpret_cast<float *>(p), p += most * kSetTokens * 4;
  a.x_ops = reinterpret_cast<_Float16 *>(p), p += m.n_tokens * m.k * 4;
  a.h_ops = reinterpret_cast<_Float16 *>(p);
  a.h_step = set_tokens(m.n_tokens) * m.n_ff * 2, p += most * a.h_step * 2;
  a.set_tokens = static_cast<int>(set_tokens(m.n_tokens));
  a.partial = reinterpret_cast<float *>(p);
  const Plan out = outer_plan(m.n_tokens, m.k, m.type_out);
  a.parts_out = out.parts, a.groups_out = out.groups;
  a.n_tokens = static_cast<int>(m.n_tokens), a.k = static_cast<int>(m.k), a.n_ff = static_cast<int>(m.n_ff);
  a.n_experts = static_cast<int>(m.n_experts), a.n_used = static_cast<int>(m.n_used), a.renormalise = m.renormalise;
  a.type_in = m.type_in, a.type_out = m.type_out;
  a.logit_groups = static_cast<int>(m.n_experts * ((m.n_tokens + kLogitTokens - 1) / kLogitTokens));
  const unsigned first = static_cast<unsigned>(a.logit_groups + (m.k * m.n_tokens + kLogitThreads - 1) / kLogitThreads);
  hipError_t e = launch(moe_prepare_kernel, dim3(first), dim3(kLogitThreads), 0, stream, a);
  if (e != hipSuccess) return e;
  a.most = static_cast<int>(most);
  e = by_qtype_k(m.type_in, [&](auto q) {
    constexpr int QT = decltype(q)::value;
    return run_inner<QT>(a, stream);
  });
  if (e != hipSuccess) return e;
  return by_qtype_k(m.type_out, [&](auto q) {
    constexpr int QT = decltype(q)::value;
    return m.n_tokens == 1 ? run_outer<QT, QT == QMM_TYPE_Q8_0 ? 8 : 16>(a, stream) : run_outer<QT, 4>(a, stream);
  });
}

}  // namespace qmm
