// The step both attention kernels are made of: one wavefront's 32 query rows
// against 32 or 64 keys and values that lie in LDS.
//
// For one query row, with scores s_u = scale q . k_u in base-2 units, the
// running state over the keys seen so far is m = max s_u, l = sum 2^(s_u - m)
// and o = sum 2^(s_u - m) v_u; a block of keys updates it in one pass:
//   m' = max(m, max_block s),  (l, o) = 2^(m - m') (l, o) + block's sums.
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
};
struct ElemBF16 {
  typedef __bf16 one;
  typedef bf16x8_t v8;
  typedef bf16x4_t v4;
  static constexpr uint32_t exp_mask = 0x7F80u;
  __device__ static __forceinline__ float16_t mfma(v8 a, v8 b, float16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
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
    off = static_cast<uint32_t>(r * row_bytes) + 16 * Tile::perm(r, lane % kChunks);
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
#pragma unroll
      for (int j = 0; j < kCount; ++j) {
        const int r = (part + j * PARTS) * kPer + lane / kChunks;
        const uint32_t o =
            static_cast<uint32_t>((r < count ? r : count - 1) * row_bytes) + 16 * Tile::perm(r, lane % kChunks);
        dma_to_lds(o, b, lds + (part + j * PARTS) * 1024);
      }
    }
  }
};

// The state of a wavefront's 32 rows (a lane's column lane % 32).
template <int D> struct AttnState {
  float16_t o[D / 32];
  float m, l;  // l: this lane's half of the sum
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = float16_t{};
    m = -__builtin_inff();
    l = 0.f;
  }
};

__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32); }

// The wavefront's rows as the B operand of S^T: element j of step ks is
// element 16 ks + 8 h + j of the lane's row.
template <class E, int D>
__device__ __forceinline__ void load_rows(const typename E::one *row, int lane, typename E::v8 q[D / 16]) {
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks)
    q[ks] = *reinterpret_cast<const typename E::v8 *>(row + 16 * ks + 8 * (lane >> 5));
}

// True if any of the operand's 8 elements is an infinity or a NaN.
template <class E> __device__ __forceinline__ bool any_nonfinite(typename E::v8 v) {
  const u32x4_t u = __builtin_bit_cast(u32x4_t, v);
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    bad |= (u[i] & E::exp_mask) == E::exp_mask;
    bad |= ((u[i] >> 16) & E::exp_mask) == E::exp_mask;
  }
  return bad;
}
template <class E> __device__ __forceinline__ typename E::v8 finite_or_zero(typename E::v8 v) {
  u32x4_t u = __builtin_bit_cast(u32x4_t, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((u[i] & E::exp_mask) == E::exp_mask) u[i] &= 0xFFFF0000u;
    if (((u[i] >> 16) & E::exp_mask) == E::exp_mask) u[i] &= 0x0000FFFFu;
  }
  return __builtin_bit_cast(typename E::v8, u);
}

// Weights are kept relative to a reference m that follows the maximum only
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

// 32 * NT keys of the LDS tiles at byte addresses kt and vt. With MASK, a
// lane's row takes the block's first `lim` keys only (lim may be <= 0 or past
// the block); without it, all. `c` is scale * log2(e) > 0.
//
// A masked key's weight is zero, but zero times a non-finite value is a NaN:
// with MASK, non-finite values enter the product as zeros, and where there
// are any (no ordinary call) their contributions to the rows that do take
// the key are added one key at a time.
template <class E, int D, int NT, bool MASK>
__device__ __forceinline__ void attend(uint32_t kt, uint32_t vt, const typename E::v8 q[D / 16], AttnState<D> &st,
                                       float c, int lim, int lane) {
  typedef typename E::v8 v8;
  constexpr int kRow = 2 * D;  // bytes of a row
  const int h = lane >> 5, col = lane & 31;
  // K: row 32 t + col, chunk 2 ks + h: permuting is an exclusive or, so a
  // step's address is the first one's with 32 ks flipped in
  const uint32_t ka = kt + col * kRow + 16 * TileK<D>::perm(col, h);
  v8 kf[D / 16 * NT];
  float16_t s[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) s[t] = float16_t{};
#pragma unroll
  for (int i = 0; i < D / 16 * NT; ++i) lds_read(kf[i], (ka ^ (32 * (i / NT))) + (i % NT) * 32 * kRow);
#pragma unroll
  for (int i = 0; i < D / 16 * NT; ++i) s[i % NT] = E::mfma(kf[i], q[i / NT], s[i % NT]);
  // reads run kAhead operands ahead of the products
  constexpr int kAhead = 4;
  __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
  for (int i = 0; i < D / 16 * NT - kAhead; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
  __builtin_amdgcn_sched_barrier(0);

  if constexpr (MASK) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (32 * t + 8 * (r >> 2) + 4 * h + (r & 3) >= lim) s[t][r] = -__builtin_inff();
  }
  float mx = s[0][0];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[t][r]);
  mx = fmaxf(mx, other_half(mx)) * c;
  if (__any(mx > st.m + kSlack)) {  // also the first keys of a row: m is -infinity
    const float m = fmaxf(st.m, mx);
    const float alpha = m == -__builtin_inff() ? 1.f : __builtin_amdgcn_exp2f(st.m - m);
    st.m = m;
    st.l *= alpha;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) st.o[i][r] *= alpha;
  }
  const float mu = st.m == -__builtin_inff() ? 0.f : st.m;  // no key yet: weights of zero, not NaN
  v8 p[2 * NT];
  float sum[2] = {0.f, 0.f};
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][r], c, -mu));
      sum[r & 1] += w;
      p[2 * t + (r >> 3)][r & 7] = static_cast<typename E::one>(w);
    }
  st.l += sum[0] + sum[1];

  // V^T: lane column d = 32 dt + col; the 16 lanes of a read take rows key ..
  // key + 3, columns 32 dt + 16 ((lane / 16) % 2) .. + 15. Again exclusive
  // ors: 64 for dt, 32 for the second four keys (8 rows on)
  const int i16 = lane & 15;
  const int vrow = 4 * h + (i16 >> 2), vcol = 16 * ((lane >> 4) & 1) + 4 * (i16 & 3);
  const uint32_t va = vt + vrow * kRow + 16 * TileV<D>::perm(vrow, vcol >> 3) + 2 * (vcol & 7);
  auto read_v = [&](int k, int dt) {
    const uint32_t a = (va ^ (64 * dt)) + k * 16 * kRow;
    struct { short4_t a, b; } both;
    both.a = lds_read_transposed(a);
    both.b = lds_read_transposed((va ^ (64 * dt) ^ 32) + k * 16 * kRow + 8 * kRow);
    return __builtin_bit_cast(v8, both);
  };
  constexpr int kSteps = 2 * NT * (D / 32);
  v8 vf[kSteps];
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) vf[i] = read_v(i / (D / 32), i % (D / 32));
  if constexpr (!MASK) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) st.o[i % (D / 32)] = E::mfma(vf[i], p[i / (D / 32)], st.o[i % (D / 32)]);
    constexpr int kAheadV = 3;
    __builtin_amdgcn_sched_group_barrier(0x100, 2 * kAheadV, 0);
#pragma unroll
    for (int i = 0; i < kSteps - kAheadV; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, kAheadV, 0);
    __builtin_amdgcn_sched_barrier(0);
  } else {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      bad |= any_nonfinite<E>(vf[i]);
      st.o[i % (D / 32)] = E::mfma(finite_or_zero<E>(vf[i]), p[i / (D / 32)], st.o[i % (D / 32)]);
    }
    if (__any(bad)) {
#pragma unroll 1
      for (int u = 0; u < 32 * NT; ++u) {
        // key u's weight: operand step u / 16, element 4 (u % 16 / 8) + u % 4, of the lanes of half (u / 4) % 2
        const int word = 4 * (u >> 4) + 2 * ((u >> 3) & 1) + ((u >> 1) & 1);
        uint32_t two = 0;
#pragma unroll
        for (int k = 0; k < 2 * NT; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (4 * k + i == word) two = __builtin_bit_cast(u32x4_t, p[k])[i];
        two = __shfl(two, col + 32 * ((u >> 2) & 1)) >> (16 * (u & 1));
        const float w = static_cast<float>(__builtin_bit_cast(typename E::one, static_cast<uint16_t>(two)));
        if (u >= lim) continue;
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int e = 32 * dt + 8 * (r >> 2) + 4 * h + (r & 3);
            const float v = static_cast<float>(*reinterpret_cast<const __attribute__((address_space(3))) typename E::one *>(
                vt + u * kRow + 16 * TileV<D>::perm(u, e >> 3) + 2 * (e & 7)));
            if (!__builtin_isfinite(v)) st.o[dt][r] += w * v;
          }
      }
    }
  }
}

// The whole sum of weights of a lane's row.
template <int D> __device__ __forceinline__ float row_sum(const AttnState<D> &st) { return st.l + other_half(st.l); }

// Writes a lane's half of its row's D outputs, times f, to `row` (8 bytes
// per store).
template <class E, int D>
__device__ __forceinline__ void store_row(typename E::one *row, const AttnState<D> &st, float f, int lane) {
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      typename E::v4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = static_cast<typename E::one>(st.o[dt][4 * i + j] * f);
      *reinterpret_cast<typename E::v4 *>(row + 32 * dt + 8 * i + 4 * (lane >> 5)) = v;
    }
}

}  // namespace qmm
