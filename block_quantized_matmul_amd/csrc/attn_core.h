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
// 16 bytes per lane from p into LDS at byte address lds + 16 lane (lds the
// same in all lanes). M0 is written by a scalar move, and an LDS-DMA load
// must not follow it directly.
__device__ __forceinline__ void dma_to_lds(const void *p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(lds) : "memory", "m0");
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

// Copies `count` (1 .. rows) rows of a K or V tile of `rows` rows into LDS,
// row r from base + row0 + min(r, count - 1): rows past the last valid one
// repeat it, so nothing behind it is read and whatever the masked places
// hold, they hold values that the row attends to anyway. `part` of `parts`
// wavefronts; the copies are awaited with wait_loads.
template <int D, class Tile, class E>
__device__ __forceinline__ void copy_tile(const E *base, int64_t token_stride, int64_t row0, int count, int rows,
                                          uint32_t lds, int part, int parts, int lane) {
  constexpr int kChunks = D / 8;            // 16-byte chunks per row
  constexpr int kRowsPer = 64 / kChunks;    // rows one instruction copies
  for (int g = part; g < rows / kRowsPer; g += parts) {
    const int r = g * kRowsPer + lane / kChunks;
    const int c = Tile::perm(r, lane % kChunks);
    const E *p = base + (row0 + (r < count ? r : count - 1)) * token_stride + c * 8;
    dma_to_lds(p, __builtin_amdgcn_readfirstlane(lds + g * 1024));
  }
}

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

// 32 * NT keys of LDS tiles kt and vt. With MASK, a lane's row takes the
// block's first `lim` keys only (lim may be <= 0 or past the block); without
// it, all. `c` is scale * log2(e) > 0.
//
// A masked key's weight is zero, but zero times a non-finite value is a NaN:
// with MASK, non-finite values enter the product as zeros, and where there
// are any (no ordinary call) their contributions to the rows that do take
// the key are added one key at a time.
template <class E, int D, int NT, bool MASK>
__device__ __forceinline__ void attend(const uint8_t *kt, const uint8_t *vt, const typename E::v8 q[D / 16],
                                       AttnState<D> &st, float c, int lim, int lane) {
  const int h = lane >> 5, col = lane & 31;
  float16_t s[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) s[t] = float16_t{};
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = 32 * t + col;
      const auto a = *reinterpret_cast<const typename E::v8 *>(kt + r * (2 * D) + 16 * TileK<D>::perm(r, 2 * ks + h));
      s[t] = E::mfma(a, q[ks], s[t]);
    }
  }
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
  const float m = fmaxf(st.m, mx);
  const float mu = m == -__builtin_inff() ? 0.f : m;  // no key yet: weights of zero, not NaN
  const float alpha = __builtin_amdgcn_exp2f(st.m - mu);
  st.m = m;
  if (__any(alpha != 1.f)) {
    st.l *= alpha;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) st.o[i][r] *= alpha;
  }
  typename E::v8 p[2 * NT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][r], c, -mu));
      st.l += w;
      p[2 * t + (r >> 3)][r & 7] = static_cast<typename E::one>(w);
    }
  // V^T: lane column d = 32 dt + col; the 16 lanes of a read take rows
  // key .. key + 3, columns 32 dt + 16 ((lane / 16) % 2) .. + 15
  const int i16 = lane & 15;
  const int vcol = 16 * ((lane >> 4) & 1) + 4 * (i16 & 3);
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 2 * NT; ++k) {
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt) {
      short4_t half[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 16 * k + 8 * i + 4 * h + (i16 >> 2);
        const int e = 32 * dt + vcol;
        const uint8_t *a = vt + r * (2 * D) + 16 * TileV<D>::perm(r, e >> 3) + 2 * (e & 7);
        half[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) short4_t *)(reinterpret_cast<short4_t *>(const_cast<uint8_t *>(a))));
      }
      struct { short4_t a, b; } both = {half[0], half[1]};
      auto v = __builtin_bit_cast(typename E::v8, both);
      if constexpr (MASK) {
        bad |= any_nonfinite<E>(v);
        v = finite_or_zero<E>(v);
      }
      st.o[dt] = E::mfma(v, p[k], st.o[dt]);
    }
  }
  if constexpr (MASK) {
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
            const float v = static_cast<float>(*reinterpret_cast<const typename E::one *>(
                vt + u * (2 * D) + 16 * TileV<D>::perm(u, e >> 3) + 2 * (e & 7)));
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
