// The step both attention kernels are made of: one wavefront's 32 query rows
// against 32 or 64 keys and values that lie in LDS.
//
// For one query row, with scores s_u = scale q . k_u in base-2 units, the
// running state over the keys seen so far is m = max s_u, l = sum 2^(s_u - m)
// and o = sum 2^(s_u - m) v_u; a block of keys updates it in one pass:
//   m' = max(m, max_block s),  (l, o) = 2^(m - m') (l, o) + block's sums.
// s_u = c x_u with the raw score x_u = q . k_u, and c = scale log2(e) is applied
// where a difference is taken (Reference, below).
//
// Both products run on v_mfma_f32_32x32x16 with the query row along the
// columns: S^T = K Q^T and O^T = V^T P^T. A lane then owns one query row
// (column lane % 32), half of its scores (the C layout gives lane half h =
// lane / 32 the keys 8 i + 4 h + 0..3 of each 32) and half of its outputs, so
// the row's maximum needs one exchange with lane ^ 32, the rescaling factor
// no exchange at all, and the exponentials already lie where the second
// product reads its B operand: operand element j of step s holds key
// 16 s + 8 (j / 4) + 4 h + j % 4 when V^T is read in the same key order. K
// comes from LDS as 16-byte pieces of its rows, V^T through the transposing
// LDS read (ds_read_b64_tr_b16: 16 lanes take a 4 x 16 block by columns).
//
// K and V tiles are copied from global memory straight into LDS, 16 bytes per
// lane, with the 16-byte chunks of a row permuted (by the choice of the
// global address) so that both kinds of read spread over all banks.
#pragma once

#include "common.h"

namespace qmm {

typedef float float16_t __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef short short4_t __attribute__((ext_vector_type(4)));

// Element types of the attention operands.
struct ElemF16 {
  typedef _Float16 one;
  typedef half8_t v8;
  typedef half4_t v4;
  static constexpr uint32_t exp_mask = 0x7C00u;  // exponent bits all ones: infinity or NaN
  __device__ static __forceinline__ float16_t mfma(v8 a, v8 b, float16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  // An output is a mean of values with rounded weights over the sum of the
  // unrounded ones, and may thus pass the largest value by a half step, hence
  // the type's range: x within it, but for infinities and NaN.
  static constexpr float largest = 65504.f;
  __device__ static __forceinline__ float limit(float x) {
    return __builtin_fabsf(x) < __builtin_inff() ? __builtin_amdgcn_fmed3f(x, -largest, largest) : x;
  }
};
struct ElemBF16 {
  typedef __bf16 one;
  typedef bf16x8_t v8;
  typedef bf16x4_t v4;
  static constexpr uint32_t exp_mask = 0x7F80u;
  __device__ static __forceinline__ float16_t mfma(v8 a, v8 b, float16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  // fp32 has no room for sums of values that large either.
  static constexpr float largest = __builtin_inff();
  __device__ static __forceinline__ float limit(float x) { return x; }
};

__device__ __forceinline__ uint32_t lds_addr(const void *p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) void *)p));
}
// 16 bytes per lane from base + off into LDS at byte address lds + 16 lane
// (base and lds the same in all lanes). M0 is written by a scalar move, and
// an LDS-DMA load must not follow it directly.
__device__ __forceinline__ void dma_to_lds(uint32_t off, const void *base, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds)
               : "memory", "m0");
}
template <int N> __device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// This wavefront's LDS reads are done, so what they read may be overwritten.
__device__ __forceinline__ void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// A tile of rows of D elements in LDS: chunk c (16 bytes) of row r at slot
// perm(r, c) of the row. K reads take one chunk of 32 consecutive rows: the
// permutation puts any 16 consecutive rows (8 pairs for D = 64, whose rows
// fill half the banks) on distinct slots. V reads take 4 chunks of 8
// consecutive rows: 4 rows fill the banks once.
template <int D> struct TileK {
  __device__ static __forceinline__ int perm(int r, int c) { return D == 128 ? c ^ (r & 15) : c ^ ((r >> 1) & 7); }
};
template <int D> struct TileV {
  __device__ static __forceinline__ int perm(int r, int c) {
    return D == 128 ? c ^ (((r & 3) << 2) | ((r >> 2) & 3)) : c ^ (((r >> 1) & 1) << 2 | ((r >> 2) & 3));
  }
};

// Copies blocks of ROWS rows of a K or V into LDS, for one of PARTS wavefronts
// that copy a block together. A copy instruction moves kPer rows; the chunk a
// lane takes does not depend on which of the wavefront's rows it is for, so
// one 32-bit offset per lane serves all of them and the rest of the address
// is scalar (63 rows of 2^25 elements still fit).
template <int D, class Tile, class E, int ROWS, int PARTS> struct Copier {
  static constexpr int kChunks = D / 8;           // 16-byte chunks per row
  static constexpr int kPer = 64 / kChunks;       // rows per instruction
  static constexpr int kCount = ROWS / kPer / PARTS;
  static_assert(kPer * PARTS % 16 == 0 || kCount == 1 || PARTS == 1, "the permutation repeats every 16 rows");
  const uint8_t *base;  // row 0
  int64_t row_bytes;
  uint32_t off;  // this lane's, in its wavefront's first row group
  int part;

  __device__ __forceinline__ Copier(const typename E::one *p, int64_t token_stride, int wave, int lane)
      : base(reinterpret_cast<const uint8_t *>(p)), row_bytes(token_stride * 2), part(wave) {
    const int r = part * kPer + lane / kChunks;
    off = static_cast<uint32_t>(r) * static_cast<uint32_t>(row_bytes) + 16 * Tile::perm(r, lane % kChunks);
  }
  // Rows row0 .. row0 + count - 1 (1 <= count <= ROWS). Rows past the last
  // valid one repeat it, so nothing behind it is read and whatever the
  // masked places hold, they hold values that the row attends to anyway.
  __device__ __forceinline__ void operator()(int64_t row0, int count, uint32_t lds, int lane) const {
    const uint8_t *b = base + row0 * row_bytes;
    if (count >= ROWS && PARTS > 1) {
#pragma unroll
      for (int j = 0; j < kCount; ++j) {
        const uint8_t *bj = b + j * (kPer * PARTS) * row_bytes;
        dma_to_lds(off, bj, lds + (part + j * PARTS) * 1024);
      }
    } else {
      int l = lane;
      asm volatile("" : "+v"(l));  // computed here, not kept in registers through the loops around
#pragma unroll
      for (int j = 0; j < kCount; ++j) {
        const int r = (part + j * PARTS) * kPer + l / kChunks;
        const uint32_t o = static_cast<uint32_t>(r < count ? r : count - 1) * static_cast<uint32_t>(row_bytes) +
                           16 * Tile::perm(r, l % kChunks);
        dma_to_lds(o, b, lds + (part + j * PARTS) * 1024);
      }
    }
  }
};

// What a row's weights are relative to: the weight of raw score x is
// 2^(c x - c m) for the row's reference m, itself a raw score. It is computed as
// 2^fma(x - sub, c, -mu) with one of
//   mu = c m rounded, sub = 0: one instruction. The rounding of c m only moves
//     the reference, by at most 2^-4 where |c m| < kLarge;
//   mu = 0, sub = m: where c m is larger, its rounding could be off by so much
//     that the weights leave their type's range, or all vanish.
// An infinite m has neither (mu = sub = 0): -infinity stands for no key, whose
// weights are zeros, and infinity for rows that come out as infinity or NaN.
constexpr float kLarge = 0x1p20f;
struct Reference {
  float mu, sub;
  __device__ __forceinline__ Reference(float m, float c) {
    const float scaled = m * c;
    const bool large = !(__builtin_fabsf(scaled) < kLarge);
    mu = large ? 0.f : scaled;
    sub = large && __builtin_fabsf(m) < __builtin_inff() ? m : 0.f;
  }
};
// The factor that takes sums relative to m over to those relative to `to`.
__device__ __forceinline__ float rescaling(float m, float to, float c) {
  const Reference a(m, c), b(to, c);
  return m == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(__builtin_fmaf(a.sub - b.sub, c, a.mu - b.mu));
}

// The state of a wavefront's 32 rows (a lane's column lane % 32).
template <int D> struct AttnState {
  float16_t o[D / 32];
  float m, l;  // m: the reference, a raw score; l: this lane's half of the sum
  float mu;    // Reference(m, c).mu
  bool large;  // some row of the wavefront has had a Reference with a sub
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = float16_t{};
    m = -__builtin_inff();
    l = mu = 0.f;
    large = false;
  }
};

// x of lane ^ 32 and x itself, in either order.
__device__ __forceinline__ float2_t both_halves(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return float2_t{__builtin_bit_cast(float, static_cast<uint32_t>(r[0])),
                  __builtin_bit_cast(float, static_cast<uint32_t>(r[1]))};
}

// The wavefront's rows as the B operand of S^T: element j of step ks is
// element 16 ks + 8 h + j of the lane's row.
template <class E, int D>
__device__ __forceinline__ void load_rows(const typename E::one *row, int lane, typename E::v8 q[D / 16]) {
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks)
    q[ks] = *reinterpret_cast<const typename E::v8 *>(row + 16 * ks + 8 * (lane >> 5));
}

// True, in every lane, if this wavefront's share (one of `parts`) of the
// `bytes` of LDS at byte address a holds an infinity or a NaN.
template <class E, int BYTES, int PARTS>
__device__ __forceinline__ bool any_nonfinite(uint32_t a, int part, int lane) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 most = {0, 0};  // the largest magnitude, as bits
#pragma unroll
  for (int i = 0; i < BYTES / PARTS / 1024; ++i) {
    const u32x4_t u = *reinterpret_cast<const __attribute__((address_space(3))) u32x4_t *>(
        a + (i * PARTS + part) * 1024 + 16 * lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, u[j] & 0x7FFF7FFFu));
  }
  return __any(most.x >= E::exp_mask || most.y >= E::exp_mask);
}
// Weights are kept relative to a reference that follows the maximum only
// when it is exceeded by more than kSlack (in base-2 units): any reference
// gives the same quotient, and weights up to 2^kSlack neither overflow fp16
// nor cost precision, while rescaling the outputs (64 multiplies at D = 128)
// for every new maximum would cost as much as a quarter of a block's products.
constexpr float kSlack = 8.f;

__device__ __forceinline__ void lds_read(half8_t &v, uint32_t a) {
  v = *reinterpret_cast<const __attribute__((address_space(3))) half8_t *>(a);
}
__device__ __forceinline__ void lds_read(bf16x8_t &v, uint32_t a) {
  v = *reinterpret_cast<const __attribute__((address_space(3))) bf16x8_t *>(a);
}

__device__ __forceinline__ short4_t lds_read_transposed(uint32_t a) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<__attribute__((address_space(3))) short4_t *>(a));
}

// V^T's operand for keys 16 k .. + 15 and outputs 32 dt .. + 31; va is the
// lane's address for k = dt = 0. Exclusive ors again: 64 for dt, 32 for the
// second four keys of a lane (8 rows on).
template <class E, int D> __device__ __forceinline__ typename E::v8 read_v(uint32_t va, int k, int dt) {
  constexpr int kRow = 2 * D;
  struct { short4_t a, b; } both;
  both.a = lds_read_transposed((va ^ (64 * dt)) + k * 16 * kRow);
  both.b = lds_read_transposed((va ^ (64 * dt) ^ 32) + k * 16 * kRow + 8 * kRow);
  return __builtin_bit_cast(typename E::v8, both);
}

// Raw scores of 32 * NT keys, whose K tile lies at LDS byte address kt.
template <class E, int D, int NT>
__device__ __forceinline__ void scores(uint32_t kt, const typename E::v8 q[D / 16], float16_t s[NT], int lane) {
  constexpr int kRow = 2 * D;  // bytes of a row
  const int h = lane >> 5, col = lane & 31;
  // row 32 t + col, chunk 2 ks + h: permuting is an exclusive or, so a
  // step's address is the first one's with 32 ks flipped in
  const uint32_t ka = kt + col * kRow + 16 * TileK<D>::perm(col, h);
  typename E::v8 kf[D / 16 * NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) s[t] = float16_t{};
#pragma unroll
  for (int i = 0; i < D / 16 * NT; ++i) lds_read(kf[i], (ka ^ (32 * (i / NT))) + (i % NT) * 32 * kRow);
#pragma unroll
  for (int i = 0; i < D / 16 * NT; ++i) s[i % NT] = E::mfma(kf[i], q[i / NT], s[i % NT]);
}

// The largest raw score of each lane's row.
template <int NT> __device__ __forceinline__ float row_max(const float16_t s[NT]) {
  float mx[2] = {s[0][0], s[0][1]};
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 16; r += 2) {
      mx[(r >> 1) & 1] = fmaxf(fmaxf(mx[(r >> 1) & 1], s[t][r]), s[t][r + 1]);
    }
  const float2_t two = both_halves(fmaxf(mx[0], mx[1]));
  return fmaxf(two.x, two.y);
}

// Keys at and past `lim` of the block take no part.
template <int NT> __device__ __forceinline__ void mask_scores(float16_t s[NT], int lim, int lane) {
  const int l = lim - 4 * (lane >> 5);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r)
      if (32 * t + 8 * (r >> 2) + (r & 3) >= l) s[t][r] = -__builtin_inff();
}

// Moves the reference up to the block's largest raw score mx where some row's
// exceeds it by more than kSlack, which is also so for a row's first keys; then
// makes the scores s ready for weights().
template <int D, int NT>
__device__ __forceinline__ void follow_max(AttnState<D> &st, float mx, float c, float16_t s[NT]) {
  if (__any((mx - st.m) * c > kSlack)) {
    const float m = fmaxf(st.m, mx);
    const float alpha = rescaling(st.m, m, c);
    const Reference ref(m, c);
    st.m = m, st.mu = ref.mu;
    st.large = st.large || __any(ref.sub != 0.f);
    st.l *= alpha;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) st.o[i][r] *= alpha;
  }
  if (st.large) {
    const float sub = Reference(st.m, c).sub;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) s[t][r] -= sub;
  }
}

// Weights of the scores, rounded for the second product, and their sum, which
// goes to l unrounded. The matrix cores take fp32 operands at a small fraction
// of the rate (154 against 1191 TFLOP/s, large library products), so weights are
// rounded to the values' type: with the output's own rounding the error is then
// 1.2 to 1.4 times that of the output's rounding alone (8192 bf16 tokens: 2.0e-3
// against 1.5e-3 of the outputs' size).
template <class E, int D, int NT>
__device__ __forceinline__ void weights(const float16_t s[NT], AttnState<D> &st, float c, typename E::v8 p[2 * NT]) {
  float sum[2] = {0.f, 0.f};
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][r], c, -st.mu));
      sum[r & 1] += w;
      p[2 * t + (r >> 3)][r & 7] = static_cast<typename E::one>(w);
    }
  st.l += sum[0] + sum[1];
}

// The lane's address of V^T's first operand in the tile at vt: lane column
// d = 32 dt + lane % 32; the 16 lanes of a read take rows key .. key + 3,
// columns 32 dt + 16 ((lane / 16) % 2) .. + 15.
template <int D> __device__ __forceinline__ uint32_t v_addr(uint32_t vt, int lane) {
  const int row = 4 * (lane >> 5) + ((lane & 15) >> 2), col = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  return vt + row * (2 * D) + 16 * TileV<D>::perm(row, col >> 3) + 2 * (col & 7);
}
template <class E, int D, int NT>
__device__ __forceinline__ void add_values(uint32_t va, const typename E::v8 p[2 * NT], AttnState<D> &st) {
  constexpr int kSteps = 2 * NT * (D / 32);
  typename E::v8 vf[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) vf[i] = read_v<E, D>(va, i / (D / 32), i % (D / 32));
#pragma unroll
  for (int i = 0; i < kSteps; ++i) st.o[i % (D / 32)] = E::mfma(vf[i], p[i / (D / 32)], st.o[i % (D / 32)]);
}
// Scheduling of the instructions since the last barrier: `n` products, each
// after the first `ahead` operands' reads (`reads` per operand), and beside
// each product `valu` vector and `trans` transcendental instructions.
template <int N, int AHEAD, int READS, int VALU, int TRANS> __device__ __forceinline__ void interleave() {
  __builtin_amdgcn_sched_group_barrier(0x100, AHEAD * READS, 0);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if (i < N - AHEAD) __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
    if (VALU > 0) __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
    if (TRANS > 0) __builtin_amdgcn_sched_group_barrier(0x400, TRANS, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
}

// A workgroup of four wavefronts, 32 rows each, over keys 0 .. n_keys - 1 in
// blocks of 64, with two buffers of a K and a V tile each in LDS.
//
// The two products of a block depend on each other through its weights, and
// a wavefront alone issues a vector instruction only every 7 cycles or so,
// so within a wavefront the products of one block run beside the vector
// arithmetic of another: the scores of block b + 1 beside the weights of
// block b, and the values of block b beside the maximum of block b + 1's
// scores. The scores therefore run one block ahead: K is copied two blocks
// ahead, V one.
//
// A wavefront's rows need its first `mine` blocks (>= 1; without CAUSAL also
// 0, for a wavefront that only copies); the first `full` (< mine) of them are
// taken whole by all its rows, of the others a lane's row takes keys below lim.
//
// A masked key's weight is zero, but zero times a non-finite value is a NaN.
// With CAUSAL, the values of the blocks from first_masked on (at most any
// wavefront's `full`, and the same for all) are therefore looked over, and
// true is returned where the wavefront's masked blocks held an infinity or a
// NaN: its rows have to be computed another way then. Without CAUSAL all rows share one end, behind
// which copied rows only repeat the last.
constexpr int kKeys = 64;
template <int D> constexpr int attend_lds_bytes() { return 4 * kKeys * D * 2 + 32; }
template <class E, int D, bool CAUSAL, class CopyK, class CopyV>
__device__ __forceinline__ bool attend_blocks(uint8_t *lds, const CopyK &copy_k, const CopyV &copy_v, int n_keys,
                                              int first_masked, int full, int mine, int lim,
                                              typename E::v8 q[D / 16], AttnState<D> &st, float c, int wave, int lane) {
  constexpr int kTile = kKeys * D * 2;
  typedef typename E::v8 v8;
  const int blocks = (n_keys + kKeys - 1) / kKeys;
  const uint32_t k0 = lds_addr(lds), v0 = k0 + 2 * kTile;
  int *nonfinite = reinterpret_cast<int *>(lds + 4 * kTile);  // [2][4], by buffer and wavefront
  auto kt = [&](int b) { return k0 + (b & 1) * kTile; };
  auto vt = [&](int b) { return v0 + (b & 1) * kTile; };
  auto load_k = [&](int b) {
    if (b < blocks) copy_k(static_cast<int64_t>(b) * kKeys, n_keys - b * kKeys, kt(b), lane);
  };
  auto load_v = [&](int b) {
    if (b < blocks) copy_v(static_cast<int64_t>(b) * kKeys, n_keys - b * kKeys, vt(b), lane);
  };
  // Before block b: V of b and K of b + 1 have landed for all wavefronts, and
  // the buffers of V of b - 1 and K of b are free to be filled again.
  auto next = [&](int b) {
    wait_loads<0>();
    if (CAUSAL && b >= first_masked) {  // each wavefront looks at the rows it copied
      const bool bad = any_nonfinite<E, kTile, 4>(vt(b), wave, lane);
      if (lane == 0) nonfinite[(b & 1) * 4 + wave] = bad;
    }
    __syncthreads();
    load_k(b + 2);
    load_v(b + 1);
  };

  float16_t s[2], ahead[2];
  v8 p[4];
  int any_bad = 0;
  load_k(0);
  load_v(0);
  wait_loads<0>();
  // the compiler waits for its own loads of q here, while nothing else is on its way
#pragma unroll
  for (int i = 0; i < D / 16; ++i) asm volatile("" : "+v"(q[i]));
  __syncthreads();
  load_k(1);
  float mx = 0.f;
  if (CAUSAL || mine > 0) {
    scores<E, D, 2>(kt(0), q, s, lane);
    interleave<D / 8, 4, 1, 0, 0>();
    mx = row_max<2>(s);
  }
  auto step = [&](int b, float16_t(&now)[2], float16_t(&then)[2]) {
    next(b);
    follow_max<D, 2>(st, mx, c, now);
    __builtin_amdgcn_sched_barrier(0);
    scores<E, D, 2>(kt(b + 1), q, then, lane);
    weights<E, D, 2>(now, st, c, p);
    interleave<D / 8, 4, 1, 5, 2>();
    add_values<E, D, 2>(v_addr<D>(vt(b), lane), p, st);
    mx = row_max<2>(then);
    interleave<D / 8, 3, 2, 2, 0>();
  };
  int b = 0;
  for (; b + 1 < full; b += 2) {  // two at a time: the scores' registers swap
    step(b, s, ahead);
    step(b + 1, ahead, s);
  }
  if (b < full) {
    step(b, s, ahead);
    s[0] = ahead[0], s[1] = ahead[1];
    ++b;
  }
  for (; b < mine; ++b) {
    next(b);
    mask_scores<2>(s, lim - b * kKeys, lane);
    follow_max<D, 2>(st, row_max<2>(s), c, s);
    weights<E, D, 2>(s, st, c, p);
    __builtin_amdgcn_sched_barrier(0);
    if (CAUSAL) {
      const int *bad = nonfinite + (b & 1) * 4;
      any_bad |= __builtin_amdgcn_readfirstlane(bad[0] | bad[1] | bad[2] | bad[3]);
    }
    __builtin_amdgcn_sched_barrier(0);
    add_values<E, D, 2>(v_addr<D>(vt(b), lane), p, st);
    interleave<D / 8, 3, 2, 0, 0>();
    if (b + 1 < mine) {
      scores<E, D, 2>(kt(b + 1), q, s, lane);
      interleave<D / 8, 4, 1, 0, 0>();
    }
  }
  for (; b < blocks; ++b) next(b);  // the other wavefronts' blocks
  return any_bad != 0;
}

// The whole sum of weights of a lane's row.
template <int D> __device__ __forceinline__ float row_sum(const AttnState<D> &st) {
  const float2_t two = both_halves(st.l);
  return two.x + two.y;
}

// Writes a row's D outputs, times f, from the two lanes that hold it. A lane
// has 4 of every 8 elements; lanes l and l + 32 trade, so that l stores the 8
// elements of one chunk and l + 32 those of the next (16 bytes per store).
// Both lanes of a row call it, with the same `live`.
template <class E, int D>
__device__ __forceinline__ void store_row(typename E::one *row, AttnState<D> &st, float f, int lane, bool live) {
  if (E::largest < __builtin_inff()) {
    float top = 0.f;
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, __builtin_fabsf(st.o[dt][r]));
    if (__builtin_expect(__any(top * f > E::largest), 0)) {
#pragma unroll
      for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int r = 0; r < 16; ++r) st.o[dt][r] = E::limit(st.o[dt][r] * f);
      f = 1.f;
    }
  }
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      u32x2_t two[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        typename E::v4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = static_cast<typename E::one>(st.o[dt][4 * (i + k) + j] * f);
        two[k] = __builtin_bit_cast(u32x2_t, v);
      }
      const auto x = __builtin_amdgcn_permlane32_swap(two[0].x, two[1].x, false, false);
      const auto y = __builtin_amdgcn_permlane32_swap(two[0].y, two[1].y, false, false);
      if (live) *reinterpret_cast<u32x4_t *>(row + 32 * dt + 8 * (i + (lane >> 5))) = u32x4_t{x[0], y[0], x[1], y[1]};
    }
}

}  // namespace qmm
