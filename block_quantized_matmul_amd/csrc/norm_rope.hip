// Norm, rotation, conversion and store of a batch's heads (qmm_norm_rope).
//
// Bound by memory: every element is read once and written once, and the few
// arithmetic steps between run on the loaded registers. A head is handled by
// `lanes` neighbouring lanes of a wavefront, each lane holding the elements
// that rotate together: two runs of V elements, first elements i.. and
// n_freqs + i.. (QMM_ROPE_HALVES) or 8 neighbouring ones
// (QMM_ROPE_NEIGHBOURS), so the rotation needs no exchange and the norm's sum
// one butterfly over the head's lanes. V is 4 (16-byte loads and stores of
// fp32, 8-byte ones of 16-bit types), or 1 for head sizes and alignments
// that do not allow it.
//
// An angle p f (position times radians per position) matters modulo a turn
// only: f / 2 pi is rounded to 64-bit fixed point on the host, and the
// product with the integer position, modulo 2^64, is the fraction of a turn
// (error below |p| (2^-64 + |f| 2^-67)). Its top bits choose the quadrant, the
// rest is an angle in [-pi/4, pi/4] for the Taylor polynomials of sine and
// cosine. A wavefront computes its lanes' sines once per token and then goes
// over the heads of the token.
//
// Measured: 16384 tokens of 32 query, 8 key and 8 value heads of 128, fp32 to
// fp16, 135 us (604 MB, 4.5 TB/s; a large copy reaches 4.9). One token 5 us,
// which the host's 11 us for a call hide.
#include "attn.h"
#include "common.h"
#include "launch.h"

#include <algorithm>

namespace qmm {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxFreqs = QMM_NORM_ROPE_MAX_DIM / 2;
constexpr int kFewFreqs = 64;  // the table travels in the kernel's arguments, so its size costs launch time

struct Part {
  const void *x;
  void *y;
  const float *w;
  int64_t xt, xh, yt, yh;
  int heads, passes;  // passes: wavefront passes over the heads
  int x_type, y_type;
  int norm, rotate, slotted;
};
template <int F> struct RopeArgs {
  Part part[QMM_HEAD_PARTS_MAX];
  const int32_t *positions, *slots;
  int64_t n_tokens;
  int n_parts, dim, n_freqs, neighbours, n_slots;
  int lanes;   // lanes per head, a power of two
  int chunks;  // wavefronts per token
  int chunk;   // passes per wavefront
  float eps, inv_dim;
  uint64_t turn[F];  // f / 2 pi in units of 2^-64
};

typedef uint16_t u16x4_a8 __attribute__((ext_vector_type(4), aligned(8)));

__device__ __forceinline__ float from_bits16(uint32_t u, bool bf16) {
  return bf16 ? __builtin_bit_cast(float, u << 16) : half_bits_to_float(u);
}
__device__ __forceinline__ uint16_t to_bits16(float x, bool bf16) {
  return bf16 ? __builtin_bit_cast(uint16_t, static_cast<__bf16>(x))
              : __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
}
template <int V> __device__ __forceinline__ void load_run(const void *x, int64_t at, int type, float *out) {
  if (type == QMM_T_F32) {
    if constexpr (V == 4) {
      const float4_t f = *reinterpret_cast<const float4_t *>(static_cast<const float *>(x) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) out[i] = f[i];
    } else {
      out[0] = static_cast<const float *>(x)[at];
    }
  } else {
    const bool bf = type == QMM_T_BF16;
    if constexpr (V == 4) {
      const u16x4_a8 u = *reinterpret_cast<const u16x4_a8 *>(static_cast<const uint16_t *>(x) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) out[i] = from_bits16(u[i], bf);
    } else {
      out[0] = from_bits16(static_cast<const uint16_t *>(x)[at], bf);
    }
  }
}
template <int V> __device__ __forceinline__ void store_run(void *y, int64_t at, int type, const float *v) {
  if (type == QMM_T_F32) {
    if constexpr (V == 4)
      *reinterpret_cast<float4_t *>(static_cast<float *>(y) + at) = float4_t{v[0], v[1], v[2], v[3]};
    else
      static_cast<float *>(y)[at] = v[0];
  } else {
    const bool bf = type == QMM_T_BF16;
    if constexpr (V == 4)
      *reinterpret_cast<u16x4_a8 *>(static_cast<uint16_t *>(y) + at) =
          u16x4_a8{to_bits16(v[0], bf), to_bits16(v[1], bf), to_bits16(v[2], bf), to_bits16(v[3], bf)};
    else
      static_cast<uint16_t *>(y)[at] = to_bits16(v[0], bf);
  }
}

// Sine and cosine of 2 pi t / 2^64. On [-pi/4, pi/4] the Taylor polynomials'
// first omitted terms are at most 1.8e-9 for the sine (x^11 / 11!) and 2.5e-8,
// 0.4 of a half step of fp32 at 1, for the cosine (x^10 / 10!).
__device__ __forceinline__ void sincos_turn(uint64_t t, float &sin, float &cos) {
  const uint32_t quadrant = static_cast<uint32_t>((t + (uint64_t{1} << 61)) >> 62);
  const int32_t r = static_cast<int32_t>((t - (static_cast<uint64_t>(quadrant) << 62)) >> 32);
  const float x = static_cast<float>(r) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float x2 = x * x;
  float s = __builtin_fmaf(x2, 2.7557319224e-6f, -1.9841269841e-4f);
  s = __builtin_fmaf(s, x2, 8.3333333333e-3f);
  s = __builtin_fmaf(s, x2, -1.6666666667e-1f);
  s = __builtin_fmaf(s * x2, x, x);
  float c = __builtin_fmaf(x2, 2.4801587302e-5f, -1.3888888889e-3f);
  c = __builtin_fmaf(c, x2, 4.1666666667e-2f);
  c = __builtin_fmaf(c, x2, -0.5f);
  c = __builtin_fmaf(c, x2, 1.f);
  const float a = quadrant & 1 ? c : s, b = quadrant & 1 ? s : c;
  sin = quadrant & 2 ? -a : a;
  cos = (quadrant + 1) & 2 ? -b : b;
}

// U: units per lane (a unit is two runs of V elements).
template <int V, int U, int F>
__global__ __launch_bounds__(kThreads) void norm_rope_kernel(RopeArgs<F> a) {
  const int lane = threadIdx.x & 63;
  const int64_t wave0 = static_cast<int64_t>(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6);
  const int unit0 = lane & (a.lanes - 1), sub = lane / a.lanes, per = 64 / a.lanes;
  const int runs = a.dim / V;         // runs of V elements per head
  const int half = a.n_freqs / V;     // halves: rotated runs per half
  const int units = a.neighbours ? (runs + 1) / 2 : half + (runs - 2 * half + 1) / 2;

  const int64_t n_waves = a.n_tokens * a.chunks, stride = static_cast<int64_t>(gridDim.x) * (kThreads / 64);
  for (int64_t wave = wave0; wave < n_waves; wave += stride) {
    const int64_t token = wave / a.chunks;
    // this lane's runs, and the sines and cosines of its rotations
    int at[U][2];
    bool on[U][2], rot[U][2];
    float sn[U][V == 4 ? 4 : 1], cs[U][V == 4 ? 4 : 1];
    const int32_t pos = a.positions ? a.positions[token] : 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int unit = unit0 + u * 64;
      const bool paired = !a.neighbours && unit < half;
      const int r0 = paired ? unit : a.neighbours ? 2 * unit : 2 * half + 2 * (unit - half);
      const int r1 = paired ? half + unit : r0 + 1;
      on[u][0] = unit < units, on[u][1] = unit < units && r1 < runs;
      at[u][0] = on[u][0] ? r0 * V : 0, at[u][1] = on[u][1] ? r1 * V : 0;
      // neighbours, V == 4: each run holds two pairs; V == 1: the unit is a pair
      rot[u][0] = paired || (a.neighbours && (V == 4 ? 4 * r0 : r0) < 2 * a.n_freqs);
      rot[u][1] = paired || (a.neighbours && (V == 4 ? 4 * r1 : r1) < 2 * a.n_freqs);
#pragma unroll
      for (int i = 0; i < (V == 4 ? 4 : 1); ++i) {
        const int f = a.neighbours ? (V == 4 ? 2 * r0 + i : unit) : unit * V + i;
        const uint64_t t = f < a.n_freqs ? a.turn[f] * static_cast<uint64_t>(static_cast<int64_t>(pos)) : 0;
        sincos_turn(t, sn[u][i], cs[u][i]);
      }
    }
    const int slot = a.slots ? a.slots[token] : 0;

    int pass = static_cast<int>(wave % a.chunks) * a.chunk;
    const int pass_end = pass + a.chunk;
    int base = 0;
    for (int p = 0; p < a.n_parts; ++p) {
      const Part &part = a.part[p];
      const int end = base + part.passes;
      const bool stored = !part.slotted || (slot >= 0 && slot < a.n_slots);
      for (; pass < pass_end && pass < end; ++pass) {
        const int head = (pass - base) * per + sub;
        const bool live = head < part.heads;
        const int64_t x0 = token * part.xt + (live ? head : 0) * part.xh;
        float v[U][2][V];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[u][k][i] = 0.f;
            if (on[u][k]) load_run<V>(part.x, x0 + at[u][k], part.x_type, v[u][k]);
          }
        if (part.norm) {
          float sum = 0.f;
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int i = 0; i < V; ++i) sum = __builtin_fmaf(v[u][k][i], v[u][k][i], sum);
          for (int d = a.lanes / 2; d > 0; d /= 2) sum += __shfl_xor(sum, d);
          const float f = 1.f / sqrtf(__builtin_fmaf(sum, a.inv_dim, a.eps));
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float w[V];
#pragma unroll
              for (int i = 0; i < V; ++i) w[i] = 1.f;
              if (part.w && on[u][k]) {
#pragma unroll
                for (int i = 0; i < V; ++i) w[i] = part.w[at[u][k] + i];
              }
#pragma unroll
              for (int i = 0; i < V; ++i) v[u][k][i] *= f * w[i];
            }
        }
        if (part.rotate) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (V == 1 || !a.neighbours) {
              if (rot[u][0]) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                  const float x = v[u][0][i], y = v[u][1][i];
                  v[u][0][i] = x * cs[u][i] - y * sn[u][i];
                  v[u][1][i] = y * cs[u][i] + x * sn[u][i];
                }
              }
            } else if constexpr (V == 4) {
#pragma unroll
              for (int k = 0; k < 2; ++k)
                if (rot[u][k]) {
#pragma unroll
                  for (int i = 0; i < 4; i += 2) {
                    const float x = v[u][k][i], y = v[u][k][i + 1], c = cs[u][2 * k + i / 2], s = sn[u][2 * k + i / 2];
                    v[u][k][i] = x * c - y * s;
                    v[u][k][i + 1] = y * c + x * s;
                  }
                }
            }
          }
        }
        if (live && stored) {
          const int64_t y0 = (part.slotted ? slot : token) * part.yt + head * part.yh;
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              if (on[u][k]) store_run<V>(part.y, y0 + at[u][k], part.y_type, v[u][k]);
        }
      }
      base = end;
    }
  }
}

bool run_aligned(const void *p, int type, int64_t s0, int64_t s1) {
  const uintptr_t bytes = type == QMM_T_F32 ? 16 : 8;
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && s0 % 4 == 0 && s1 % 4 == 0;
}

// f / 2 pi in units of 2^-64, modulo 1, to within a unit: f is m 2^e with a
// 53-bit integer m, and m 2^65 / pi an integer product of 117 bits.
uint64_t to_turn(double f) {
  const uint64_t bits = __builtin_bit_cast(uint64_t, f);
  const int e = static_cast<int>(bits >> 52 & 0x7FF);
  if (e == 0) return 0;  // zero, or far below any angle
  const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | 0x10000000000000ull;
  const unsigned __int128 product = static_cast<unsigned __int128>(m) * 0xA2F9836E4E44152Aull;  // 2^65 / pi
  const int shift = 1077 - e;  // f = m 2^(e - 1075); 64 fraction bits, and 66 in the constant
  uint64_t t = 0;
  if (shift < 128)  // and above 47, |f| being at most 64
    t = static_cast<uint64_t>((product + (static_cast<unsigned __int128>(1) << (shift - 1))) >> shift);
  return f < 0 ? 0 - t : t;
}

template <int F>
hipError_t run(const qmm_head_part *parts, int n_parts, int64_t n_tokens, int64_t head_dim, float eps,
               const int32_t *positions, const double *freqs, int64_t n_freqs, int pairs, const int32_t *slots,
               int64_t n_slots, hipStream_t stream) {
  RopeArgs<F> a;
  bool wide = head_dim % 4 == 0 && n_freqs % (pairs == QMM_ROPE_HALVES ? 4 : 2) == 0;
  for (int p = 0; p < n_parts; ++p)
    wide = wide && run_aligned(parts[p].X, parts[p].x_type, parts[p].x_token_stride, parts[p].x_head_stride) &&
           run_aligned(parts[p].Y, parts[p].y_type, parts[p].y_row_stride, parts[p].y_head_stride);
  a.positions = positions, a.slots = slots, a.n_tokens = n_tokens;
  a.n_parts = n_parts, a.dim = static_cast<int>(head_dim), a.n_freqs = static_cast<int>(n_freqs);
  a.neighbours = pairs == QMM_ROPE_NEIGHBOURS, a.n_slots = static_cast<int>(n_slots);
  a.eps = eps, a.inv_dim = 1.f / static_cast<float>(head_dim);
  // a frequency in turns per position, modulo whole turns (positions are integers)
  for (int64_t i = 0; i < n_freqs; ++i) a.turn[i] = to_turn(freqs[i]);
  // two runs per lane, rounded up: one more unit than runs / 2 may be needed
  // where the rotated and the plain part both end in half a unit
  const int v = wide ? 4 : 1;
  const int runs = a.dim / v, half = a.n_freqs / v;
  const int units = a.neighbours ? (runs + 1) / 2 : half + (runs - 2 * half + 1) / 2;
  a.lanes = 1;
  while (a.lanes < units && a.lanes < 64) a.lanes *= 2;
  const int per = 64 / a.lanes;
  int64_t passes = 0;
  for (int p = 0; p < n_parts; ++p) {
    const qmm_head_part &s = parts[p];
    Part &d = a.part[p];
    d.x = s.X, d.y = s.Y, d.w = s.weight;
    d.xt = s.x_token_stride, d.xh = s.x_head_stride, d.yt = s.y_row_stride, d.yh = s.y_head_stride;
    // (a slotted part without slots has nothing to store, and need not exist)
    d.heads = s.slotted && n_slots == 0 ? 0 : static_cast<int>(s.n_heads);
    d.passes = (d.heads + per - 1) / per;
    d.x_type = s.x_type, d.y_type = s.y_type, d.norm = s.norm, d.rotate = s.rotate, d.slotted = s.slotted;
    passes += d.passes;
  }
  if (passes == 0) return hipSuccess;
  // few tokens: one pass per wavefront, to spread them over the GPU; many:
  // a whole token per wavefront, so that its sines are computed once
  a.chunk = static_cast<int>(std::max<int64_t>(1, std::min(passes, passes * n_tokens / 8192)));
  a.chunks = static_cast<int>((passes + a.chunk - 1) / a.chunk);
  const int64_t waves = n_tokens * a.chunks;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>((waves + kThreads / 64 - 1) / (kThreads / 64), 1 << 20)));
  if (wide) return launch(norm_rope_kernel<4, 1, F>, grid, dim3(kThreads), 0, stream, a);
  if (units <= 64) return launch(norm_rope_kernel<1, 1, F>, grid, dim3(kThreads), 0, stream, a);
  return launch(norm_rope_kernel<1, 4, F>, grid, dim3(kThreads), 0, stream, a);
}

}  // namespace

hipError_t launch_norm_rope(const qmm_head_part *parts, int n_parts, int64_t n_tokens, int64_t head_dim, float eps,
                            const int32_t *positions, const double *freqs, int64_t n_freqs, int pairs,
                            const int32_t *slots, int64_t n_slots, hipStream_t stream) {
  return (n_freqs <= kFewFreqs ? run<kFewFreqs> : run<kMaxFreqs>)(parts, n_parts, n_tokens, head_dim, eps, positions,
                                                                  freqs, n_freqs, pairs, slots, n_slots, stream);
}

}  // namespace qmm
