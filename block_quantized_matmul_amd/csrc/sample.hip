// The next token of every row of logits (qmm_sample).
//
// All limits and the choice itself are prefixes of one order, by falling logit
// and then rising index, so the whole is three selections along it: the first
// top_k, the first whose mass reaches top_p of theirs, and the element where the
// mass passes u times that of what is left. No sort is needed: a selection
// descends through the logits' bits (as integers of the same order), 11 at a
// time, by a histogram of counts and masses of those that agree so far.
//
// Weights are 2^-t, t = (max - z) log2(e) / temperature, in 64 bits, and masses are
// sums of their fixed-point values (44 bits below the point): integers, whose sum
// does not depend on the order of atomic additions, and so exact that the place of
// a border moves by 10^-12 of the total. (A border decides a token; 32-bit sums
// would move one of 10^5 equally likely tokens' borders by a hundredth of a token.)
#include "common.h"
#include "launch.h"
#include "serve.h"

namespace qmm {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBits = 11, kBins = 1 << kBits;
constexpr int kPoint = 44;  // binary places of a weight

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
  return x != x ? -__builtin_inff() : x + 0.f;  // NaN is below all others, -0 is 0
}
// An integer that falls as x rises.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  return u >> 31 ? u : ~u & 0x7FFFFFFFu;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __builtin_bit_cast(float, key >> 31 ? key : ~key & 0x7FFFFFFFu);
}

// A row's weights.
struct Weights {
  double top, c;
  // log2 of the largest weight over x's
  __device__ __forceinline__ double exponent(float x) const {
    const double d = top - static_cast<double>(x);
    return static_cast<double>(x) == top ? 0. : d < __builtin_inf() ? d * c : __builtin_inf();
  }
  // 2^-t: a Taylor polynomial in f ln 2, |f| <= 1/2, whose first omitted term is below 10^-14
  __device__ __forceinline__ static double power(double t) {
    if (!(t < 1000.)) return 0.;
    const double n = __builtin_rint(t), x = (n - t) * 0.69314718055994530942;
    double p = 2.5052108385441718775e-8;  // 1 / 11!
    p = __builtin_fma(p, x, 2.7557319223985890653e-7);
    p = __builtin_fma(p, x, 2.7557319223985890653e-6);
    p = __builtin_fma(p, x, 2.4801587301587301587e-5);
    p = __builtin_fma(p, x, 1.9841269841269841270e-4);
    p = __builtin_fma(p, x, 1.3888888888888888889e-3);
    p = __builtin_fma(p, x, 8.3333333333333333333e-3);
    p = __builtin_fma(p, x, 4.1666666666666666667e-2);
    p = __builtin_fma(p, x, 1.6666666666666666667e-1);
    p = __builtin_fma(p, x, 0.5);
    p = __builtin_fma(p, x, 1.);
    p = __builtin_fma(p, x, 1.);
    return __builtin_ldexp(p, -static_cast<int>(n));
  }
  __device__ __forceinline__ static uint64_t fixed(double t) {
    return t < kPoint + 2. ? static_cast<uint64_t>(__builtin_fma(power(t), 0x1p44, 0.5)) : 0;
  }
  __device__ __forceinline__ uint64_t of(float x) const { return fixed(exponent(x)); }
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
  uint32_t wave_n[kWaves];
  uint64_t wave_m[kWaves];
  int bin;
  uint32_t before;
  uint64_t mass;
  float most;
};

__device__ __forceinline__ uint64_t shfl_up64(uint64_t x, int d) {
  const uint32_t lo = __shfl_up(static_cast<uint32_t>(x), d), hi = __shfl_up(static_cast<uint32_t>(x >> 32), d);
  return static_cast<uint64_t>(hi) << 32 | lo;
}

// The last bin in which the goal's place lies; its start goes to before and mass. All threads call it.
__device__ __forceinline__ int find_bin(Shared &s, const Goal &goal, uint32_t &before, uint64_t &mass) {
  constexpr int kPer = kBins / kThreads;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t n = 0;
  uint64_t m = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) n += s.n[threadIdx.x * kPer + i], m += s.m[threadIdx.x * kPer + i];
  uint32_t sn = n;
  uint64_t sm = m;
#pragma unroll
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
  for (int i = threadIdx.x; i < kBins; i += kThreads) s.n[i] = 0, s.m[i] = 0;
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

// The element at a goal's place (all threads get it).
template <int TYPE>
__device__ __forceinline__ Found select(Shared &s, const void *z, int64_t at, int vocab, const Weights &w, const Goal &goal) {
  Found f{0, 0, 0, 0};
  int bin = 0, high = 32;
#pragma unroll 1
  for (int shift : {32 - kBits, 32 - 2 * kBits, 0}) {
    histogram<TYPE>(s, z, at, vocab, w, f.key, shift, high);
    bin = find_bin(s, goal, f.before, f.mass);
    f.key = f.key << (high - shift) | bin;
    high = shift;
  }
  f.ties = s.n[bin];
  __syncthreads();
  return f;
}

template <int TYPE> __global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a) {
  __shared__ Shared s;
  const int row = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t at = row * a.stride;
  // the largest logit
  float most = -__builtin_inff();
  for (int i = threadIdx.x; i < a.vocab; i += kThreads) most = fmaxf(most, load_logit<TYPE>(a.z, at + i));
#pragma unroll
  for (int d = 32; d > 0; d /= 2) most = fmaxf(most, __shfl_xor(most, d));
  if (lane == 0) s.wave_n[wave] = __builtin_bit_cast(uint32_t, most);
  __syncthreads();
  for (int k = 0; k < kWaves; ++k) most = fmaxf(most, __builtin_bit_cast(float, s.wave_n[k]));
  __syncthreads();
  if (most == -__builtin_inff()) {  // nothing to choose from
    if (threadIdx.x == 0) {
      a.tokens[row] = -1;
      if (a.probs) a.probs[row] = __builtin_bit_cast(float, 0x7FC00000u);
    }
    return;
  }
  float temperature = a.temperature ? a.temperature[row] : 1.f;
  int64_t top_k = a.top_k ? a.top_k[row] : 0;
  const float top_p = a.top_p ? a.top_p[row] : 1.f, min_p = a.min_p ? a.min_p[row] : 0.f;
  float u = a.u[row];
  u = u > 0.f ? fminf(u, 0x1.fffffep-1f) : 0.f;
  if (!(temperature > 0.f)) temperature = 1.f, top_k = 1;  // the largest, the first of several
  const Weights w{static_cast<double>(most), 1.4426950408889634074 / static_cast<double>(temperature)};

  // mass of what min_p leaves, and of all
  const double limit = min_p > 0.f ? fmax(0., -log2(static_cast<double>(min_p))) : __builtin_inf();
  uint64_t all = 0, left = 0;
  for (int i = threadIdx.x; i < a.vocab; i += kThreads) {
    const double t = w.exponent(load_logit<TYPE>(a.z, at + i));
    const uint64_t m = Weights::fixed(t);
    all += m;
    left += t <= limit ? m : 0;
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint64_t x = shfl_up64(all, d), y = shfl_up64(left, d);
    if (lane >= d) all += x, left += y;
  }
  if (lane == 63) s.wave_m[wave] = all, s.m[wave] = left;
  __syncthreads();
  all = left = 0;
  for (int k = 0; k < kWaves; ++k) all += s.wave_m[k], left += s.m[k];
  __syncthreads();

  uint64_t total = all;
  if (top_k > 0 && top_k < a.vocab) {
    const Found f = select<TYPE>(s, a.z, at, a.vocab, w, Goal{COUNT, static_cast<uint32_t>(top_k), 0.});
    total = f.mass + (static_cast<uint32_t>(top_k) - f.before) * w.of(logit_of(f.key));
  }
  if (top_p < 1.f) {
    const Goal goal{BELOW, 0, fmax(static_cast<double>(top_p) * static_cast<double>(total), 0.5)};
    const Found f = select<TYPE>(s, a.z, at, a.vocab, w, goal);
    // of the equal ones, those with a mass before them below the goal
    const uint64_t one = w.of(logit_of(f.key));
    double n = one ? ceil((goal.mass - static_cast<double>(f.mass)) / static_cast<double>(one)) : 1.;
    n = fmin(fmax(n, 1.), static_cast<double>(f.ties));
    const uint64_t kept = f.mass + static_cast<uint64_t>(n) * one;
    total = kept < total ? kept : total;
  }
  total = left < total ? left : total;
  const Goal goal{UPTO, 0, static_cast<double>(u) * static_cast<double>(total)};
  const Found f = select<TYPE>(s, a.z, at, a.vocab, w, goal);
  const float chosen = logit_of(f.key);
  const uint64_t one = w.of(chosen);
  const double n = one ? floor((goal.mass - static_cast<double>(f.mass)) / static_cast<double>(one)) : 0.;
  const uint32_t which = static_cast<uint32_t>(fmin(fmax(n, 0.), static_cast<double>(f.ties - 1)));
  // the which-th element of that logit, by index: wavefront by wavefront over blocks of the row
  uint32_t seen = 0;
  for (int i0 = 0; i0 < a.vocab; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    const bool mine = i < a.vocab && load_logit<TYPE>(a.z, at + i) == chosen;
    const uint64_t mask = __ballot(mine);
    if (lane == 0) s.wave_n[wave] = __popcll(mask);
    __syncthreads();
    uint32_t before = seen, block = 0;
    for (int k = 0; k < kWaves; ++k) {
      before += k < wave ? s.wave_n[k] : 0;
      block += s.wave_n[k];
    }
    if (mine && before + __popcll(mask & ((uint64_t{1} << lane) - 1)) == which) a.tokens[row] = i;
    seen += block;
    __syncthreads();
    if (seen > which) break;  // (the same for all)
  }
  if (threadIdx.x == 0 && a.probs)
    a.probs[row] = static_cast<float>(Weights::power(w.exponent(chosen)) / (static_cast<double>(total) * 0x1p-44));
}

}  // namespace

hipError_t launch_sample(const SampleCall &c, hipStream_t stream) {
  SampleArgs a{c.logits, c.row_stride, c.u, c.temperature, c.top_p, c.min_p, c.top_k, c.tokens, c.probs, static_cast<int>(c.vocab)};
  const dim3 grid(static_cast<unsigned>(c.n_rows));
  if (c.type == QMM_T_F32) return launch(sample_kernel<QMM_T_F32>, grid, dim3(kThreads), 0, stream, a);
  if (c.type == QMM_T_F16) return launch(sample_kernel<QMM_T_F16>, grid, dim3(kThreads), 0, stream, a);
  return launch(sample_kernel<QMM_T_BF16>, grid, dim3(kThreads), 0, stream, a);
}

}  // namespace qmm
