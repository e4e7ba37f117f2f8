// The next token of every row of logits (qmm_sample).
//
// All limits and the choice itself are prefixes of one order, by falling logit
// and then rising index, so the whole is three selections along it: the first
// top_k, the first whose mass reaches top_p of theirs, and the element where the
// mass passes u times that of what is left. No sort is needed: one histogram of
// counts and masses over 8192 equal ranges of the logits below the largest finds
// the range that holds a selection's place, and the few elements of that range are
// ranked by comparing each with each. Where a range holds more than kFew (many
// equal logits, or all but equal ones), the selection descends through the bits of
// the logits (as integers of the same order) instead, 11 at a time.
//
// Weights are 2^-t, t = (max - z) log2(e) / temperature, in 64 bits, and masses are
// sums of their fixed-point values (44 bits below the point): integers, whose sum
// does not depend on the order of atomic additions, and so exact that the place of
// a border moves by 10^-12 of the total. (A border decides a token; 32-bit sums
// would move one of 10^5 equally likely tokens' borders by a hundredth of a token.)
//
// A workgroup of 16 wavefronts has a row and reads it from L2 after the first
// time. Its passes are short loops: held in registers, a row of 32000 takes 32 a
// thread, whose passes are straight-line code that runs once, and fetching that
// takes longer (54 us) than the loads.
#include "common.h"
#include "launch.h"
#include "serve.h"

namespace qmm {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBits = 11;      // of a key, at a time
constexpr int kBins = 8192;    // ranges of logits
constexpr int kFew = 256;      // elements that are ranked one by one
constexpr int kPoint = 44;     // binary places of a weight
constexpr int kFractions = 64;  // of an octave, in the table of powers (k >> 6 below)

struct SampleArgs {
  const void *z;
  int64_t stride;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t *top_k;
  int32_t *tokens;
  float *probs;
  int vocab;
};

template <int TYPE> __device__ __forceinline__ float load_logit(const void *z, int64_t at) {
  float x;
  if constexpr (TYPE == QMM_T_F32) {
    x = static_cast<const float *>(z)[at];
  } else {
    const uint32_t u = static_cast<const uint16_t *>(z)[at];
    x = TYPE == QMM_T_BF16 ? __builtin_bit_cast(float, u << 16) : half_bits_to_float(u);
  }
  return fmaxf(x, -__builtin_inff());  // a NaN is below all others
}
// Four neighbouring logits, at any multiple of their size.
template <int TYPE> __device__ __forceinline__ void load_four(const void *z, int64_t at, float x[4]) {
  typedef uint16_t u16x4 __attribute__((ext_vector_type(4), aligned(2)));
  if constexpr (TYPE == QMM_T_F32) {
    const float4_a4 v = *reinterpret_cast<const float4_a4 *>(static_cast<const float *>(z) + at);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = v[k];
  } else {
    const u16x4 v = *reinterpret_cast<const u16x4 *>(static_cast<const uint16_t *>(z) + at);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      x[k] = TYPE == QMM_T_BF16 ? __builtin_bit_cast(float, static_cast<uint32_t>(v[k]) << 16) : half_bits_to_float(v[k]);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = fmaxf(x[k], -__builtin_inff());
}
// An integer that falls as x rises.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.f);  // (-0 is 0)
  return u >> 31 ? u : ~u & 0x7FFFFFFFu;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __builtin_bit_cast(float, key >> 31 ? key : ~key & 0x7FFFFFFFu);
}

// A row's weights.
struct Weights {
  double top, c;        // c: 64 log2(e) / temperature, so exponents come in 64ths of an octave
  const double *table;  // 2^(44 - j / 64)
  // 64 log2 of the largest weight over x's
  __device__ __forceinline__ double exponent(float x) const {
    const double d = top - static_cast<double>(x);
    return static_cast<double>(x) == top ? 0. : d < __builtin_inf() ? d * c : __builtin_inf();
  }
  // 2^(44 - t / 64) for t = d c, at most 46 octaves: whole octaves, 64ths of one from the
  // table, and the rest, half a 64th at most, as a Taylor polynomial in x = -rest ln 2 / 64,
  // whose first omitted term, x^4 / 24, is below 10^-10.
  __device__ __forceinline__ double power(double d, double c) const {
    constexpr double kMagic = 0x1.8p52;  // its sum with t ends in t's whole part
    constexpr double a1 = -0.010830424696249145, a2 = 5.864904955056169e-5, a3 = -2.1173137155464774e-7;
    const double whole = __builtin_fma(d, c, kMagic);
    const int k = static_cast<int>(__builtin_bit_cast(uint64_t, whole));
    const double rest = __builtin_fma(d, c, kMagic - whole);
    const double w = table[k & (kFractions - 1)];
    const double y = __builtin_fma(w * rest, __builtin_fma(__builtin_fma(rest, a3, a2), rest, a1), w);
    return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, y) - (static_cast<uint64_t>(k >> 6) << 52));
  }
  // The nearest whole number to a power.
  __device__ __forceinline__ static uint64_t fixed(double power) {
    return __builtin_bit_cast(uint64_t, power + 0x1p52) & 0xFFFFFFFFFFFFFull;
  }
  __device__ __forceinline__ double value(float x) const { return power(fmin(exponent(x), 46. * kFractions), 1.); }
  __device__ __forceinline__ uint64_t of(float x) const { return fixed(value(x)); }
};

// What a selection looks for: the last place with a count before it below `count`,
// or with a mass before it below (BELOW) or at most (UPTO) `mass`.
enum { COUNT, BELOW, UPTO };
struct Goal {
  int kind;
  uint32_t count;
  double mass;
  __device__ __forceinline__ bool reaches(uint32_t n, uint64_t m) const {
    return kind == COUNT ? n < count : kind == BELOW ? static_cast<double>(m) < mass : static_cast<double>(m) <= mass;
  }
};
struct Found {
  uint32_t key;     // the element's
  uint32_t ties;    // elements with it
  uint32_t before;  // elements and mass in front of the first of them
  uint64_t mass;
};

struct Shared {
  uint32_t n[kBins];
  uint64_t m[kBins];
  double table[kFractions];
  uint32_t wave_n[kWaves];
  uint64_t wave_m[kWaves], wave_m2[kWaves];
  float few_z[kFew];
  int few_i[kFew];
  uint64_t few_w[kFew];
  int bin, few;
  uint32_t before;
  uint64_t mass, result;
};

__device__ __forceinline__ uint64_t shfl_up64(uint64_t x, int d) {
  const uint32_t lo = __shfl_up(static_cast<uint32_t>(x), d), hi = __shfl_up(static_cast<uint32_t>(x >> 32), d);
  return static_cast<uint64_t>(hi) << 32 | lo;
}

// The last bin in which the goal's place lies; its start goes to before and mass. All threads call it.
template <int BINS> __device__ __forceinline__ int find_bin(Shared &s, const Goal &goal, uint32_t &before, uint64_t &mass) {
  constexpr int kPer = BINS / kThreads;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t n = 0;
  uint64_t m = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) n += s.n[threadIdx.x * kPer + i], m += s.m[threadIdx.x * kPer + i];
  uint32_t sn = n;
  uint64_t sm = m;
#pragma unroll 1
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t on = __shfl_up(sn, d);
    const uint64_t om = shfl_up64(sm, d);
    if (lane >= d) sn += on, sm += om;
  }
  if (lane == 63) s.wave_n[wave] = sn, s.wave_m[wave] = sm;
  if (threadIdx.x == 0) s.bin = -1;
  __syncthreads();
  uint32_t bn = before + sn - n;  // in front of this thread's bins
  uint64_t bm = mass + sm - m;
  for (int w = 0; w < wave; ++w) bn += s.wave_n[w], bm += s.wave_m[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int bin = threadIdx.x * kPer + i;
    if (s.n[bin] > 0 && goal.reaches(bn, bm)) atomicMax(&s.bin, bin);
    bn += s.n[bin], bm += s.m[bin];
  }
  __syncthreads();
  const int bin = s.bin;
  if (bin / kPer == static_cast<int>(threadIdx.x)) {
#pragma unroll
    for (int i = kPer - 1; i >= 0; --i) {
      bn -= s.n[threadIdx.x * kPer + i], bm -= s.m[threadIdx.x * kPer + i];
      if (threadIdx.x * kPer + i == bin) {
        s.before = bn, s.mass = bm;
        break;
      }
    }
  }
  __syncthreads();
  before = s.before, mass = s.mass;
  return bin;
}

// Histogram of the bits from `shift` to `high` of the row's keys whose upper bits are `prefix`.
template <int TYPE>
__device__ __forceinline__ void histogram(Shared &s, const void *z, int64_t at, int vocab, const Weights &w, uint32_t prefix,
                                          int shift, int high) {
  for (int i = threadIdx.x; i < 1 << kBits; i += kThreads) s.n[i] = 0, s.m[i] = 0;
  __syncthreads();
  const uint32_t mask = (1u << (high - shift)) - 1;
  for (int i = threadIdx.x; i < vocab; i += kThreads) {
    const float x = load_logit<TYPE>(z, at + i);
    const uint32_t key = key_of(x);
    if (high >= 32 || key >> high == prefix) {
      const uint32_t bin = key >> shift & mask;
      atomicAdd(&s.n[bin], 1u);
      atomicAdd(reinterpret_cast<unsigned long long *>(&s.m[bin]), static_cast<unsigned long long>(w.of(x)));
    }
  }
  __syncthreads();
}

// The element at a goal's place (all threads get it), by the bits of its key.
template <int TYPE>
__device__ __forceinline__ Found select(Shared &s, const void *z, int64_t at, int vocab, const Weights &w, const Goal &goal) {
  Found f{0, 0, 0, 0};
  int bin = 0, high = 32;
#pragma unroll 1
  for (int shift : {32 - kBits, 32 - 2 * kBits, 0}) {
    histogram<TYPE>(s, z, at, vocab, w, f.key, shift, high);
    bin = find_bin<1 << kBits>(s, goal, f.before, f.mass);
    f.key = f.key << (high - shift) | bin;
    high = shift;
  }
  f.ties = s.n[bin];
  __syncthreads();
  return f;
}

// The sum over the workgroup, in every thread.
__device__ __forceinline__ uint64_t sum_of(Shared &s, uint64_t a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll 1
  for (int d = 1; d < 64; d *= 2) {
    const uint64_t x = shfl_up64(a, d);
    if (lane >= d) a += x;
  }
  if (lane == 63) s.wave_m[wave] = a;
  __syncthreads();
  a = 0;
  for (int k = 0; k < kWaves; ++k) a += s.wave_m[k];
  __syncthreads();
  return a;
}

// A row's logits, in eights: two fours of a thread a pass of the loop, the next
// ones on their way meanwhile.
template <int TYPE> struct Row {
  const void *z;
  int64_t at;
  int vocab;
  // (loads that wait for nothing: a four that the row's end cuts is read again, one by one)
  __device__ __forceinline__ void read(int j, float x[4]) const {
    if (vocab >= 4) load_four<TYPE>(z, at + min(j, vocab - 4), x);
  }
  __device__ __forceinline__ void cut(int j, float x[4]) const {
    if (j + 3 < vocab) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = j + k < vocab ? load_logit<TYPE>(z, at + j + k) : -__builtin_inff();
  }
  template <class F> __device__ __forceinline__ void each(const F &f) const {
    constexpr int kStep = 4 * kThreads;
    int j = 4 * threadIdx.x;
    float a[4] = {}, b[4] = {};
    read(j, a), read(j + kStep, b);
#pragma unroll 1
    for (; j < vocab; j += 2 * kStep) {
      float c[4] = {}, d[4] = {};
      read(j + 2 * kStep, c), read(j + 3 * kStep, d);
      cut(j, a), cut(j + kStep, b);
#pragma unroll
      for (int k = 0; k < 4; ++k) f(a[k], j + k);
#pragma unroll
      for (int k = 0; k < 4; ++k) f(b[k], j + kStep + k);
#pragma unroll
      for (int k = 0; k < 4; ++k) a[k] = c[k], b[k] = d[k];
    }
  }
};

// The range of a logit: `scale` per unit below the largest. It rises as x falls.
// Ranges 8 t .. 8 t + 7 are thread t's, the i-th of them at kThreads i + t.
constexpr int kOwn = kBins / kThreads;
__device__ __forceinline__ float place_of(float top, float x, float scale) {
  return fminf((top - x) * scale, kBins - 1.f);
}
__device__ __forceinline__ int slot_of(int range) { return range % kOwn * kThreads + range / kOwn; }

// In front of a thread's ranges, behind them, and behind all.
struct Span {
  uint32_t n0, n1;
  uint64_t m0, m1, all;
};
__device__ __forceinline__ Span own_span(Shared &s) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t n = 0;
  uint64_t m = 0;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) n += s.n[i * kThreads + threadIdx.x], m += s.m[i * kThreads + threadIdx.x];
  uint32_t sn = n;
  uint64_t sm = m;
#pragma unroll 1
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t on = __shfl_up(sn, d);
    const uint64_t om = shfl_up64(sm, d);
    if (lane >= d) sn += on, sm += om;
  }
  if (lane == 63) s.wave_n[wave] = sn, s.wave_m[wave] = sm;
  __syncthreads();
  uint64_t all = 0;
  for (int k = 0; k < kWaves; ++k) {
    if (k < wave) sn += s.wave_n[k], sm += s.wave_m[k];
    all += s.wave_m[k];
  }
  __syncthreads();
  return {sn - n, sn, sm - m, sm, all};
}

// The mass up to and with the last element whose start a goal reaches, and that
// element's index (-1: its range has too many). The histogram of ranges is in s and
// stays.
template <int TYPE>
__device__ __forceinline__ uint64_t resolve(Shared &s, const Row<TYPE> &row, const Weights &w, float scale,
                                            const Span &span, const Goal &goal, int &index) {
  const float top = static_cast<float>(w.top);
  // starts rise from thread to thread, so one thread has the last that is reached
  if (goal.reaches(span.n0, span.m0) && (threadIdx.x == kThreads - 1 || !goal.reaches(span.n1, span.m1))) {
    uint32_t n = span.n0;
    uint64_t m = span.m0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const uint32_t own_n = s.n[i * kThreads + threadIdx.x];
      const uint64_t own_m = s.m[i * kThreads + threadIdx.x];
      // (without top_k only masses are counted, and a place in question has one)
      if ((own_n > 0 || own_m > 0) && goal.reaches(n, m)) s.bin = kOwn * threadIdx.x + i, s.before = n, s.mass = m;
      n += own_n, m += own_m;
    }
    s.few = 0;
  }
  __syncthreads();
  const float low = s.bin, high = low + 1.f;
  uint32_t before = s.before;
  uint64_t mass = s.mass;
  row.each([&](float x, int i) {
    const float place = place_of(top, x, scale);
    if (place >= low && place < high && i < row.vocab) {
      const int k = atomicAdd(&s.few, 1);
      if (k < kFew) s.few_z[k] = x, s.few_i[k] = i;
    }
  });
  __syncthreads();
  const int members = s.few;
  if (members > kFew) {
    index = -1;
    return 0;
  }
  const bool mine = static_cast<int>(threadIdx.x) < members;
  uint64_t own = 0;
  if (mine) s.few_w[threadIdx.x] = own = w.of(s.few_z[threadIdx.x]);
  if (threadIdx.x == 0) s.result = 0, s.before = 0;
  __syncthreads();
  if (mine) {
    const float x = s.few_z[threadIdx.x];
    const int i = s.few_i[threadIdx.x];
    for (int k = 0; k < members; ++k) {
      const bool first = s.few_z[k] > x || (s.few_z[k] == x && s.few_i[k] < i);
      before += first;
      mass += first ? s.few_w[k] : 0;
    }
    if (goal.reaches(before, mass)) {  // the last of those that it reaches has the largest sum, and the last place
      atomicMax(reinterpret_cast<unsigned long long *>(&s.result), static_cast<unsigned long long>(mass + own));
      atomicMax(&s.before, before);
    }
  }
  __syncthreads();
  if (mine && before == s.before && goal.reaches(before, mass)) s.few = s.few_i[threadIdx.x];
  __syncthreads();
  index = s.few;
  const uint64_t result = s.result;
  __syncthreads();
  return result;
}

// The index of the which-th element of logit `chosen`: wavefront by wavefront over blocks of the row.
template <int TYPE>
__device__ __forceinline__ int nth(Shared &s, const void *z, int64_t at, int vocab, float chosen, uint32_t which) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t seen = 0;
  for (int i0 = 0; i0 < vocab && seen <= which; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    const bool mine = i < vocab && load_logit<TYPE>(z, at + i) == chosen;
    const uint64_t mask = __ballot(mine);
    if (lane == 0) s.wave_n[wave] = __popcll(mask);
    __syncthreads();
    uint32_t before = seen;
    for (int k = 0; k < kWaves; ++k) {
      before += k < wave ? s.wave_n[k] : 0;
      seen += s.wave_n[k];
    }
    if (mine && before + __popcll(mask & ((uint64_t{1} << lane) - 1)) == which) s.few = i;
    __syncthreads();
  }
  return s.few;
}

template <int TYPE> __global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared &s = *reinterpret_cast<Shared *>(smem);
  const int row_i = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Row<TYPE> row{a.z, row_i * a.stride, a.vocab};
  // the largest logit and the smallest finite one
  float most = -__builtin_inff(), least = __builtin_inff();
  row.each([&](float x, int) {
    most = fmaxf(most, x);
    least = fminf(least, x > -__builtin_inff() ? x : __builtin_inff());
  });
  for (int i = threadIdx.x; i < kBins; i += kThreads) s.n[i] = 0, s.m[i] = 0;
  if (threadIdx.x < kFractions) {  // 2^44 times the powers 2^-1/2, 2^-1/4, .. 2^-1/64 of the index's bits
    constexpr double kRoots[] = {0x1.6a09e667f3bcdp-1, 0x1.ae89f995ad3adp-1, 0x1.d5818dcfba487p-1,
                                 0x1.ea4afa2a490dap-1, 0x1.f50765b6e4540p-1, 0x1.fa7c1819e90d8p-1};
    double p = 0x1p44;
#pragma unroll
    for (int b = 0; b < 6; ++b) p *= threadIdx.x >> (5 - b) & 1 ? kRoots[b] : 1.;
    s.table[threadIdx.x] = p;
  }
#pragma unroll
  for (int d = 32; d > 0; d /= 2) most = fmaxf(most, __shfl_xor(most, d)), least = fminf(least, __shfl_xor(least, d));
  if (lane == 0) s.few_z[wave] = most, s.few_z[kWaves + wave] = least;
  __syncthreads();
  for (int k = 0; k < kWaves; ++k) most = fmaxf(most, s.few_z[k]), least = fminf(least, s.few_z[kWaves + k]);
  __syncthreads();
  if (most == -__builtin_inff()) {  // nothing to choose from
    if (threadIdx.x == 0) {
      a.tokens[row_i] = -1;
      if (a.probs) a.probs[row_i] = __builtin_bit_cast(float, 0x7FC00000u);
    }
    return;
  }
  float temperature = a.temperature ? a.temperature[row_i] : 1.f;
  int64_t top_k = a.top_k ? a.top_k[row_i] : 0;
  const float top_p = a.top_p ? a.top_p[row_i] : 1.f, min_p = a.min_p ? a.min_p[row_i] : 0.f;
  float u = a.u[row_i];
  u = u > 0.f ? fminf(u, 0x1.fffffep-1f) : 0.f;
  if (!(temperature > 0.f)) temperature = 1.f, top_k = 1;  // the largest, the first of several
  const Weights w{static_cast<double>(most), 92.332482616893653 / static_cast<double>(temperature), s.table};
  // Ranges as fine as those logits allow that have a weight at all. Rows with an
  // infinity, or too wide for fp32, go by their bits.
  const double reach = 46. * kFractions / w.c;  // no weight from there on
  const float width = fminf(most - least, static_cast<float>(fmin(reach, 3e38)));
  const float scale = width > 0.f ? (kBins - 1.f) / width : 1.f;
  const bool by_range = most - least < 3e38f && scale < 3e38f && w.c > 0.;

  // masses of the ranges, of what min_p leaves, and of all
  const uint64_t limit = min_p > 0.f ? static_cast<uint64_t>(ceil(static_cast<double>(fminf(min_p, 1.f)) * 0x1p44)) : 0;
  uint64_t left = 0;
  const bool counted = top_k > 0 && top_k < a.vocab;
  row.each([&](float x, int i) {
    uint64_t m;
    if (by_range)
      m = Weights::fixed(w.power(fmin(w.top - static_cast<double>(x), reach), w.c));
    else
      m = w.of(x);
    left += m >= limit ? m : 0;
    const int at = by_range ? slot_of(static_cast<int>(place_of(most, x, scale))) : 0;
    if (counted && i < a.vocab) atomicAdd(&s.n[at], 1u);
    if (m) atomicAdd(reinterpret_cast<unsigned long long *>(&s.m[at]), static_cast<unsigned long long>(m));
  });
  __syncthreads();
  const Span span = own_span(s);
  left = limit > 0 ? sum_of(s, left) : span.all;

  // The three selections: COUNT and BELOW leave less of the mass, UPTO chooses.
  // Where a range has too many elements, they go by the bits from there on (whose
  // histograms take the ranges' place).
  bool ranges = by_range;
  uint64_t total = span.all;
#pragma unroll 1
  for (int kind = COUNT; kind <= UPTO; ++kind) {
    if (kind == COUNT && !counted) continue;
    if (kind == BELOW && !(top_p < 1.f)) continue;
    if (kind == UPTO && left < total) total = left;
    const double mass = static_cast<double>(kind == UPTO ? u : top_p) * static_cast<double>(total);
    const Goal goal{kind, static_cast<uint32_t>(top_k), kind == BELOW ? fmax(mass, 0.5) : mass};
    uint64_t kept = 0;
    int index = -1;
    if (ranges) kept = resolve(s, row, w, scale, span, goal, index);
    if (index < 0) {
      ranges = false;
      const Found f = select<TYPE>(s, a.z, row.at, a.vocab, w, goal);
      const float chosen = logit_of(f.key);
      const uint64_t one = w.of(chosen);
      // of the equal ones, those whose start the goal reaches
      const double rest = one ? (goal.mass - static_cast<double>(f.mass)) / static_cast<double>(one) : 0.;
      double n = kind == COUNT ? static_cast<double>(goal.count - f.before) : kind == BELOW ? ceil(rest) : floor(rest) + 1.;
      n = fmin(fmax(n, 1.), static_cast<double>(f.ties));
      kept = f.mass + static_cast<uint64_t>(n) * one;
      if (kind == UPTO) index = nth<TYPE>(s, a.z, row.at, a.vocab, chosen, static_cast<uint32_t>(n) - 1);
    }
    if (kind != UPTO) {
      total = kept < total ? kept : total;
    } else if (threadIdx.x == 0) {
      a.tokens[row_i] = index;
      if (a.probs) a.probs[row_i] = static_cast<float>(w.value(load_logit<TYPE>(a.z, row.at + index)) / static_cast<double>(total));
    }
  }
}

}  // namespace

hipError_t launch_sample(const SampleCall &c, hipStream_t stream) {
  SampleArgs a{c.logits, c.row_stride, c.u, c.temperature, c.top_p, c.min_p, c.top_k, c.tokens, c.probs, static_cast<int>(c.vocab)};
  auto go = [&](auto kernel) {
    return launch(kernel, dim3(static_cast<unsigned>(c.n_rows)), dim3(kThreads), sizeof(Shared), stream, a);
  };
  if (c.type == QMM_T_F32) return go(sample_kernel<QMM_T_F32>);
  if (c.type == QMM_T_F16) return go(sample_kernel<QMM_T_F16>);
  return go(sample_kernel<QMM_T_BF16>);
}

}  // namespace qmm
