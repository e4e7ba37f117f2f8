// Keys and values into and out of the 4-bit paged cache (qmm_kv4_append,
// qmm_kv4_read; the layout stands in qmm_serve.h).
//
// Append. A lane holds 8 consecutive elements of a head, which are one dword of
// codes, both in the keys' and in the values' layout; a block of 32 is a quad
// of lanes, so its scale takes two exchanges. An element's rotation partner is
// read again (from the cache the first read filled) rather than exchanged,
// since it may lie at any distance.
//
// A code is a step function of x / d: where x lies near a border, an error of
// x chooses the neighbouring code, a whole step away. Norm, angle and rotation
// are therefore computed in 64 bits (at the rate of 32-bit arithmetic on this
// chip: 32.3 and 32.9 T fused multiply-adds a second), x is rounded to fp32 once, and from there on
// the decisions are exact: d is m scaled by a power of two and rounded once, and
// the reciprocal only finds the border next to x, d (n - 1/2), a product of 11
// and 5 bits, with which x is compared.
//
// Bound by vector instructions for many tokens: the 64-bit arithmetic and some 10
// instructions for a code. Sines are computed once for a token, a lane each, and lie in
// LDS with the norm's weights (eight in every lane: 163 us instead of 67 below). Measured:
// 16384 tokens of 8 heads of 128, fp32, normed and rotated, 59 us (153 MB, 2.6 TB/s;
// vector instructions fill two thirds of the cycles; loads issued a pass ahead: 65 us); one
// token 3.9 us. Read: the same tokens to fp16 25 us (86 MB, 3.4 TB/s; vector instructions fill 83 % of the cycles).
#include "common.h"
#include "launch.h"
#include "rope.h"
#include "serve.h"

#include <algorithm>

namespace qmm {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxTurns = 64;  // head_dim / 2
constexpr uint32_t kHalfNan = 0x7E00u;

struct AppendArgs {
  const void *k, *v;
  int64_t kt, kh, vt, vh;
  const float *w;
  const int32_t *positions, *slots;
  Kv4Cache cache;
  int64_t n_tokens, n_slots;
  double eps;
  int heads, type, norm, n_freqs, neighbours;
  int chunk, chunks;  // passes per wavefront; wavefronts per token for the keys, as many again for the values
  uint64_t turn[kMaxTurns];
};
struct ReadArgs {
  void *k, *v;
  int64_t kt, kh, vt, vh;
  const int32_t *slots;
  Kv4Cache cache;
  int64_t n_rows, n_slots, chunks;
  int heads, type, rows_shift;
};

__device__ __forceinline__ float load_one(const void *p, int64_t at, int type) {
  if (type == QMM_T_F32) return static_cast<const float *>(p)[at];
  const uint32_t u = static_cast<const uint16_t *>(p)[at];
  return type == QMM_T_BF16 ? __builtin_bit_cast(float, u << 16) : half_bits_to_float(u);
}
// 8 consecutive elements; WIDE: at a multiple of 16 bytes.
template <bool WIDE> __device__ __forceinline__ void load_eight(const void *p, int64_t at, int type, float x[8]) {
  if constexpr (WIDE) {
    if (type == QMM_T_F32) {
      const float4_t *f = reinterpret_cast<const float4_t *>(static_cast<const float *>(p) + at);
      const float4_t a = f[0], b = f[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
    } else {
      const u32x4_t u = *reinterpret_cast<const u32x4_t *>(static_cast<const uint16_t *>(p) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = u[i] & 0xFFFFu, hi = u[i] >> 16;
        x[2 * i] = type == QMM_T_BF16 ? __builtin_bit_cast(float, lo << 16) : half_bits_to_float(lo);
        x[2 * i + 1] = type == QMM_T_BF16 ? __builtin_bit_cast(float, hi << 16) : half_bits_to_float(hi);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = load_one(p, at + i, type);
  }
}

// Sine and cosine of 2 pi t / 2^64: the quadrant from the top bits, and Taylor
// polynomials on [-pi/4, pi/4], whose first omitted terms (x^17 / 17!, x^18 /
// 18!) are below 2^-53.
__device__ __forceinline__ void sincos_turn64(uint64_t t, double &sin, double &cos) {
  const uint32_t quadrant = static_cast<uint32_t>((t + (uint64_t{1} << 61)) >> 62);
  const int64_t r = static_cast<int64_t>(t - (static_cast<uint64_t>(quadrant) << 62));
  const double x = static_cast<double>(r) * 3.4061215800304986e-19;  // 2 pi / 2^64
  const double x2 = x * x;
  double s = -7.6471637318198164759e-13;                   // 1 / 15!
  s = __builtin_fma(s, x2, 1.6059043836821614599e-10);     // 1 / 13!
  s = __builtin_fma(s, x2, -2.5052108385441718775e-8);     // 1 / 11!
  s = __builtin_fma(s, x2, 2.7557319223985890653e-6);      // 1 / 9!
  s = __builtin_fma(s, x2, -1.9841269841269841270e-4);     // 1 / 7!
  s = __builtin_fma(s, x2, 8.3333333333333333333e-3);      // 1 / 5!
  s = __builtin_fma(s, x2, -1.6666666666666666667e-1);     // 1 / 3!
  s = __builtin_fma(s * x2, x, x);
  double c = 4.7794773323873852974e-14;                    // 1 / 16!
  c = __builtin_fma(c, x2, -1.1470745597729724714e-11);    // 1 / 14!
  c = __builtin_fma(c, x2, 2.0876756987868098979e-9);      // 1 / 12!
  c = __builtin_fma(c, x2, -2.7557319223985890653e-7);     // 1 / 10!
  c = __builtin_fma(c, x2, 2.4801587301587301587e-5);      // 1 / 8!
  c = __builtin_fma(c, x2, -1.3888888888888888889e-3);     // 1 / 6!
  c = __builtin_fma(c, x2, 4.1666666666666666667e-2);      // 1 / 4!
  c = __builtin_fma(c, x2, -0.5);
  c = __builtin_fma(c, x2, 1.0);
  const double a = quadrant & 1 ? c : s, b = quadrant & 1 ? s : c;
  sin = quadrant & 2 ? -a : a;
  cos = (quadrant + 1) & 2 ? -b : b;
}

// Codes (as a dword, element i in nibble i) and scale of a block whose 32
// elements lie 8 each in a quad of lanes.
__device__ __forceinline__ uint32_t block_codes(const float x[8], uint32_t &d_bits) {
  float most = x[0], zero = x[0] * 0.f;  // a NaN if one is infinite or a NaN
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    zero = __builtin_fmaf(x[i], 0.f, zero);
    most = __builtin_fabsf(x[i]) > __builtin_fabsf(most) ? x[i] : most;
  }
  int bad = zero != 0.f;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d <= 2; d *= 2) {  // the larger magnitude of the two, the lower lane's if they are equal
    const float other = __shfl_xor(most, d);
    const float a = __builtin_fabsf(most), b = __builtin_fabsf(other);
    most = b > a || (b == a && (lane & d)) ? other : most;
    bad |= __shfl_xor(bad, d);  // (by all lanes)
  }
  const _Float16 dh = static_cast<_Float16>(most * -0.125f);
  const float d = static_cast<float>(dh);
  bad |= !(__builtin_fabsf(d) < __builtin_inff());
  d_bits = bad ? kHalfNan : d == 0.f ? 0 : __builtin_bit_cast(uint16_t, dh);  // (a zero of either sign is +0)
  if (bad || d == 0.f) return 0x88888888u;
  const float inv = 1.f / d, step = __builtin_fabsf(d);
  float sum[2] = {0.f, 0.f};  // of 16^i times the codes, below 2^16
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    // floor(x / d + 1/2) is n or n - 1 for the integer n next to it, however the reciprocal was rounded
    const float n = __builtin_rintf(__builtin_fmaf(x[i], inv, 0.5f));
    const float y = d < 0.f ? -x[i] : x[i];
    const float q = y >= step * (n - 0.5f) ? n : n - 1.f;  // a border of 16 bits: exact
    sum[i / 4] = __builtin_fmaf(sum[i / 4], 16.f, __builtin_amdgcn_fmed3f(q, -8.f, 7.f) + 8.f);
  }
  return static_cast<uint32_t>(sum[0]) | static_cast<uint32_t>(sum[1]) << 16;
}

template <int D> __device__ __forceinline__ uint8_t *tile_of(const Kv4Cache &c, int slot, int head) {
  const int place = slot & (c.page_tokens - 1);
  return c.data + (slot >> c.page_shift) * c.page_bytes +
         (static_cast<int64_t>(head) * (c.page_tokens / kKv4Tile) + place / kKv4Tile) * kv4_tile_bytes(D);
}

// Element e of a rotated, normalised head is (x[e] A[e] + x[partner] B[e]) times
// the head's reciprocal norm, with A and B the same for every head of a token.
__device__ __forceinline__ int partner_of(const AppendArgs &a, int e) {
  if (e >= 2 * a.n_freqs) return e;
  return a.neighbours ? e ^ 1 : e < a.n_freqs ? e + a.n_freqs : e - a.n_freqs;
}
// A and B of a token, by one wavefront: a lane has one sine and cosine, which
// two elements share. Element e stands at (e % 8) (D / 8) + e / 8, since a lane
// reads 8 in a row.
template <int D> __device__ __forceinline__ void fill_turns(const AppendArgs &a, int position, double2 *turns, int lane) {
  auto at = [&](int e) -> double2 & { return turns[e % 8 * (D / 8) + e / 8]; };
  auto weight = [&](int e) { return a.norm && a.w ? static_cast<double>(a.w[e]) : 1.; };
  if (lane < a.n_freqs) {
    double sn, cs;
    sincos_turn64(a.turn[lane] * static_cast<uint64_t>(static_cast<int64_t>(position)), sn, cs);
    const int e = a.neighbours ? 2 * lane : lane, f = a.neighbours ? e + 1 : e + a.n_freqs;
    const double we = weight(e), wf = weight(f);
    at(e) = double2{cs * we, -sn * wf};
    at(f) = double2{cs * wf, sn * we};
  }
#pragma unroll
  for (int e = lane; e < D; e += 64)
    if (e >= 2 * a.n_freqs) at(e) = double2{weight(e), 0.};
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Workgroups are dealt to the 8 XCDs in turn, each with an L2 of its own. Runs of
// RUN go to the same one, so that the pieces of a line (neighbouring tokens') meet there.
template <int RUN> __device__ __forceinline__ uint32_t near_blocks(uint32_t block, uint32_t blocks) {
  if (block >= blocks / (8 * RUN) * (8 * RUN)) return block;
  return block / (8 * RUN) * (8 * RUN) + block % 8 * RUN + block / 8 % RUN;
}

template <int D, bool WIDE> __global__ __launch_bounds__(kThreads, 4) void append_kernel(AppendArgs a) {
  constexpr int kLanes = D / 8, kPer = 64 / kLanes;  // lanes per head, heads per pass of a wavefront
  constexpr int NB = D / 32;
  __shared__ double2 all_turns[kWaves][D];
  const int lane = threadIdx.x & 63, sub = lane / kLanes, l = lane % kLanes;
  const int own = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  double2 *turns = all_turns[own];
  const int64_t n_waves = a.n_tokens * 2 * a.chunks, stride = static_cast<int64_t>(gridDim.x) * kWaves;
  const int64_t first = static_cast<int64_t>(near_blocks<8>(blockIdx.x, gridDim.x)) * kWaves + own;
  for (int64_t wave = first; wave < n_waves; wave += stride) {
    const int64_t token = wave / (2 * a.chunks);
    const int part = static_cast<int>(wave % (2 * a.chunks));
    const bool values = part >= a.chunks;
    const bool rotate = !values && a.n_freqs > 0, turned = rotate || (!values && a.norm);
    const int slot = a.slots[token];
    const int position = rotate ? a.positions[token] : 0;
    if (slot < 0 || slot >= a.n_slots) continue;  // (the whole wavefront)
    const int t = slot & (kKv4Tile - 1);
    const int head0 = (values ? part - a.chunks : part) * a.chunk * kPer, head1 = min(a.heads, head0 + a.chunk * kPer);
    const void *src = values ? a.v : a.k;
    const int64_t token_at = token * (values ? a.vt : a.kt), apart = values ? a.vh : a.kh;
    if (turned) fill_turns<D>(a, position, turns, lane);
    for (int h0 = head0; h0 < head1; h0 += kPer) {
      const bool live = h0 + sub < head1;
      const int head = live ? h0 + sub : head1 - 1;
      const int64_t x0 = token_at + head * apart;
      float x[8];
      load_eight<WIDE>(src, x0 + 8 * l, a.type, x);
      if (turned) {
        float p[8];
        if (rotate) {
          if (WIDE && !a.neighbours) {
            load_eight<WIDE>(src, x0 + partner_of(a, 8 * l), a.type, p);
          } else if (a.neighbours && 2 * a.n_freqs == D) {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = x[i ^ 1];
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = load_one(src, x0 + partner_of(a, 8 * l + i), a.type);
          }
        }
        double scale = 1.;
        if (a.norm) {
          double sum = 0.;
#pragma unroll
          for (int i = 0; i < 8; ++i) sum = __builtin_fma(static_cast<double>(x[i]), static_cast<double>(x[i]), sum);
#pragma unroll
          for (int d = kLanes / 2; d > 0; d /= 2) sum += __shfl_xor(sum, d);
          scale = 1. / sqrt(sum * (1. / D) + a.eps);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const double2 turn = turns[i * kLanes + l];
          double y = static_cast<double>(x[i]) * turn.x;
          if (rotate) y = __builtin_fma(static_cast<double>(p[i]), turn.y, y);
          x[i] = static_cast<float>(y * scale);
        }
      }
      uint32_t d_bits;
      const uint32_t codes = block_codes(x, d_bits);
      if (live) {
        uint8_t *tile = tile_of<D>(a.cache, slot, head);
        const int b = l / 4, g = l % 4;
        uint8_t *to = values ? tile + 8 * D + t * (D / 2) + 4 * l : tile + 4 * ((16 * g + t) * NB + b);
        *reinterpret_cast<uint32_t *>(to) = codes;
        if (g == 0)
          *reinterpret_cast<uint16_t *>(tile + (values ? 17 : 16) * D + 2 * (16 * b + t)) =
              static_cast<uint16_t>(d_bits);
      }
    }
  }
}

template <bool WIDE> __device__ __forceinline__ void store_eight(void *p, int64_t at, int type, const float x[8]) {
  if (type == QMM_T_F32) {
    float *f = static_cast<float *>(p) + at;
    if constexpr (WIDE) {
      reinterpret_cast<float4_t *>(f)[0] = float4_t{x[0], x[1], x[2], x[3]};
      reinterpret_cast<float4_t *>(f)[1] = float4_t{x[4], x[5], x[6], x[7]};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = x[i];
    }
    return;
  }
  uint16_t *u = static_cast<uint16_t *>(p) + at;
  uint16_t y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    y[i] = type == QMM_T_BF16 ? __builtin_bit_cast(uint16_t, static_cast<__bf16>(x[i]))
                              : __builtin_bit_cast(uint16_t, static_cast<_Float16>(x[i]));
  if constexpr (WIDE) {
    u32x4_t w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = y[2 * i] | static_cast<uint32_t>(y[2 * i + 1]) << 16;
    *reinterpret_cast<u32x4_t *>(u) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = y[i];
  }
}

// A lane writes 8 elements. A row's lanes are those of its keys, then its values,
// head by head, in a.chunks wavefronts; where they are few, a wavefront has 2^a.rows_shift rows.
template <int D, bool WIDE> __global__ __launch_bounds__(kThreads) void read_kernel(ReadArgs a) {
  constexpr int kLanes = D / 8, NB = D / 32;
  const int lane = threadIdx.x & 63, lanes = a.heads * kLanes;  // of the keys or the values
  const int shift = 6 - a.rows_shift, sub = lane >> shift, mine = lane & ((1 << shift) - 1);
  const int64_t n = ((a.n_rows + (1 << a.rows_shift) - 1) >> a.rows_shift) * a.chunks;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kWaves;
  int64_t wave = static_cast<int64_t>(near_blocks<16>(blockIdx.x, gridDim.x)) * kWaves +
                 __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (; wave < n; wave += stride) {
    const int64_t first = a.chunks == 1 ? wave : wave / a.chunks;
    const int64_t row = (first << a.rows_shift) + sub;
    const int64_t item = (wave - first * a.chunks) * 64 + mine;
    const bool values = a.k == nullptr || item >= lanes;
    const int64_t at = values && a.k != nullptr ? item - lanes : item;
    if (row >= a.n_rows || at >= lanes || (values && a.v == nullptr)) continue;
    const int l = static_cast<int>(at % kLanes), head = static_cast<int>(at / kLanes);
    const int slot = a.slots[row];
    const int b = l / 4, g = l % 4;
    uint32_t codes = 0;
    float d = __builtin_bit_cast(float, 0x7FC00000u);
    if (slot >= 0 && slot < a.n_slots) {
      const uint8_t *tile = tile_of<D>(a.cache, slot, head);
      const int t = slot & (kKv4Tile - 1);
      codes = *reinterpret_cast<const uint32_t *>(values ? tile + 8 * D + t * (D / 2) + 4 * l
                                                         : tile + 4 * ((16 * g + t) * NB + b));
      d = half_bits_to_float(
          *reinterpret_cast<const uint16_t *>(tile + (values ? 17 : 16) * D + 2 * (16 * b + t)));
    }
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = d * static_cast<float>(static_cast<int>(codes >> (4 * j) & 15u) - 8);
    if (values)
      store_eight<WIDE>(a.v, row * a.vt + head * a.vh + 8 * l, a.type, x);
    else
      store_eight<WIDE>(a.k, row * a.kt + head * a.kh + 8 * l, a.type, x);
  }
}

// Runs of 8 elements at multiples of 16 bytes (strides of axes that have more than one element).
bool wide(const qmm_heads &h, int64_t tokens, int64_t heads) {
  return reinterpret_cast<uintptr_t>(h.data) % 16 == 0 && (tokens <= 1 || h.token_stride % 8 == 0) &&
         (heads <= 1 || h.head_stride % 8 == 0);
}

unsigned grid_for(int64_t groups) { return static_cast<unsigned>(std::min<int64_t>(groups, 1 << 20)); }

}  // namespace

hipError_t launch_kv4_append(int type, const qmm_heads &K, const qmm_heads &V, int64_t n_tokens, int64_t n_kv_heads,
                             int64_t head_dim, bool norm, const float *weight, double eps, const int32_t *positions,
                             const double *freqs, int64_t n_freqs, int pairs, const int32_t *slots,
                             const Kv4Cache &cache, hipStream_t stream) {
  AppendArgs a{};
  a.k = K.data, a.v = V.data, a.kt = K.token_stride, a.kh = K.head_stride, a.vt = V.token_stride, a.vh = V.head_stride;
  a.w = weight, a.positions = positions, a.slots = slots, a.cache = cache;
  a.n_tokens = n_tokens, a.n_slots = cache.n_pages * cache.page_tokens, a.eps = eps;
  a.heads = static_cast<int>(n_kv_heads), a.type = type, a.norm = norm, a.n_freqs = static_cast<int>(n_freqs);
  a.neighbours = pairs == QMM_ROPE_NEIGHBOURS;
  for (int64_t i = 0; i < n_freqs; ++i) a.turn[i] = to_turn(freqs[i]);
  const int64_t per = 64 / (head_dim / 8), passes = (n_kv_heads + per - 1) / per;
  // few tokens: one pass per wavefront, to spread them over the GPU; many: all
  // heads of a token, so that its sines are computed once
  a.chunk = static_cast<int>(std::max<int64_t>(1, std::min(passes, 2 * passes * n_tokens / 8192)));
  a.chunks = static_cast<int>((passes + a.chunk - 1) / a.chunk);
  const unsigned grid = grid_for((n_tokens * 2 * a.chunks + kWaves - 1) / kWaves);
  const bool w = wide(K, n_tokens, n_kv_heads) && wide(V, n_tokens, n_kv_heads) &&
                 (a.neighbours || n_freqs % 8 == 0);
  auto go = [&](auto kernel) { return launch(kernel, dim3(grid), dim3(kThreads), 0, stream, a); };
  if (head_dim == 128) return w ? go(append_kernel<128, true>) : go(append_kernel<128, false>);
  return w ? go(append_kernel<64, true>) : go(append_kernel<64, false>);
}

hipError_t launch_kv4_read(int type, const qmm_heads &K, const qmm_heads &V, int64_t n_rows, int64_t n_kv_heads,
                           int64_t head_dim, const int32_t *slots, const Kv4Cache &cache, hipStream_t stream) {
  ReadArgs a{};
  a.k = K.data, a.v = V.data, a.kt = K.token_stride, a.kh = K.head_stride, a.vt = V.token_stride, a.vh = V.head_stride;
  a.slots = slots, a.cache = cache, a.n_rows = n_rows, a.n_slots = cache.n_pages * cache.page_tokens;
  a.heads = static_cast<int>(n_kv_heads), a.type = type;
  const int64_t lanes = (K.data && V.data ? 2 : 1) * n_kv_heads * (head_dim / 8);
  while ((lanes << (a.rows_shift + 1)) <= 64) ++a.rows_shift;
  if ((lanes << a.rows_shift) != 64) a.rows_shift = 0;  // (three heads of 64)
  a.chunks = (lanes + 63) / 64;
  const int64_t waves = ((n_rows + (1 << a.rows_shift) - 1) >> a.rows_shift) * a.chunks;
  const unsigned grid = grid_for((waves + kWaves - 1) / kWaves);
  const bool w = (K.data == nullptr || wide(K, n_rows, n_kv_heads)) && (V.data == nullptr || wide(V, n_rows, n_kv_heads));
  auto go = [&](auto kernel) { return launch(kernel, dim3(grid), dim3(kThreads), 0, stream, a); };
  if (head_dim == 128) return w ? go(read_kernel<128, true>) : go(read_kernel<128, false>);
  return w ? go(read_kernel<64, true>) : go(read_kernel<64, false>);
}

}  // namespace qmm
