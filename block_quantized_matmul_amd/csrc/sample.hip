// The next token of every row of logits (qmm_sample).
//
// All limits and the choice itself are prefixes of one order, by falling logit
// and then rising index, so the whole is three selections along it: the first
// top_k, the first whose mass reaches top_p of theirs, and the element where the
// mass passes u times that of what is left. No sort is needed: one histogram of
// counts and masses over 1024 equal ranges of the logits below the largest finds
// the range that holds a selection's place, and the few elements of that range are
// ranked by comparing each with each, after dividing the range again, or equal
// elements by index, where they are more than kFew. Rows that this does not fit (with
// infinities, or most elements in few ranges) descend through the bits of the logits
// (as integers of the same order) instead, 11 at a time.
//
// Weights are 2^-t, t = (max - z) log2(e) / temperature, in 64 bits, and masses are
// sums of their fixed-point values (44 bits below the point): integers, whose sum
// does not depend on the order of atomic additions, and so exact that the place of
// a border moves by 10^-12 of the total. (A border decides a token; 32-bit sums
// would move one of 10^5 equally likely tokens' borders by a hundredth of a token.)
//
// Bound by latency: the logits are few, and the steps follow from each other. A row
// is divided into chunks of 8192, a workgroup each, in three launches: the largest
// logits; the histograms, which the row's last workgroup adds; the elements of the
// ranges in question, among which the row's last workgroup chooses. Where a
// selection's place is not known before the one in front of it, its bounds are, and
// the ranges between them are few.
//
// Measured (fp32): one row of 32000 2.7 + 11 + 8 us (a workgroup of 16 wavefronts for
// the row, which reads it five times: 33); 64 rows 4 + 16 + 19 (41); 37 rows of 130001,
// flat, so that ranges have hundreds of elements: 6 + 24 + 30 (116). With 2048 ranges
// these are 25, 44 and 67 us in all instead of 22, 39 and 60; with up to 256 elements
// ranked all together, and then 2048 ranges, 24, 39 and 84.
#include "common.h"
#include "launch.h"
#include "serve.h"

#include <algorithm>
#include <type_traits>

namespace qmm {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBits = 11;      // of a key, at a time
constexpr int kBins = kThreads;  // ranges of logits, one a thread
constexpr int kChunk = 8 * kThreads;
constexpr int kList = 16384;   // elements of a row that are looked at in the end
constexpr int kAtOnce = 8;
constexpr int kQuick = 64;      // of those: elements that are ranked all together, by one wavefront
constexpr int kFew = 512;      // elements that are ranked one by one
constexpr int kFractions = 64;  // of an octave, in the table of powers (k >> 6 below)

struct SampleArgs {
  const void *z;
  int64_t stride;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t *top_k;
  int32_t *tokens;
  float *probs;
  int vocab, chunks, room;
  // workspace
  struct RowState *rows;  // [n_rows]
  struct Element *list;   // [n_rows][room]
  struct Part *parts;     // [n_rows][chunks]
  struct Top *tops;       // [n_rows][chunks]
};
struct alignas(8) Element {
  float z;
  int i;
};
// What workgroups of one launch write and others of it read (`put` and `get`: the
// parts, the lists and the counters) shares no line with what they read in the ordinary
// way, whatever the workspace's alignment. A line that an L2 has taken in for the one
// is then never asked for the other.
constexpr int kLine = 128;
struct Part {  // a chunk's
  uint64_t m[kBins];
  uint32_t n[kBins];
  uint64_t left;  // mass that min_p leaves
  uint8_t apart[kLine];
};
struct Top {  // a chunk's largest logit, and its smallest finite one
  float most, least;
};
enum { COUNT, BELOW, UPTO };
struct RowState {
  uint32_t arrived[2];  // workgroups, of the second and third launch
  uint32_t listed;
  uint8_t apart[kLine + 4];
  uint64_t m[kBins + 1];  // mass and count in front of every range
  uint32_t n[kBins + 1];
  int lo[3], hi[3];       // ranges that may hold a selection's place; none where it is known
  uint64_t left;
  uint8_t behind[kLine];
};
static_assert(offsetof(RowState, m) - offsetof(RowState, listed) >= kLine + sizeof(uint32_t) &&
              sizeof(RowState) - offsetof(RowState, left) >= kLine + sizeof(uint64_t) &&
              sizeof(Part) - offsetof(Part, left) >= kLine + sizeof(uint64_t) && sizeof(RowState) % 8 == 0);

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
  // whose first omitted term, x^6 / 720, is below 2^-54. (Without the last two, x^4 / 24 =
  // 2^-34.7 of the weight would be left out, which moves borders by more than the sums do.)
  __device__ __forceinline__ double power(double d, double c) const {
    constexpr double kMagic = 0x1.8p52;  // its sum with t ends in t's whole part
    constexpr double a1 = -0.010830424696249145, a2 = 5.864904955056169e-5, a3 = -2.1173137155464774e-7,
                     a4 = 5.732851688640402e-10, a5 = -1.2417843701716925e-12;
    const double whole = __builtin_fma(d, c, kMagic);
    const int k = static_cast<int>(__builtin_bit_cast(uint64_t, whole));
    const double rest = __builtin_fma(d, c, kMagic - whole);
    const double w = table[k & (kFractions - 1)];
    double sum = __builtin_fma(rest, a5, a4);
    sum = __builtin_fma(sum, rest, a3);
    sum = __builtin_fma(sum, rest, a2);
    sum = __builtin_fma(sum, rest, a1);
    const double y = __builtin_fma(w * rest, sum, w);
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
  uint32_t n[1 << kBits];
  uint64_t m[(1 << kBits) + 1];
  double table[kFractions];
  uint32_t wave_n[kWaves];
  uint64_t wave_m[kWaves];
  float few_z[kFew + kAtOnce];
  int few_i[kFew + kAtOnce];
  uint64_t few_w[kFew + kAtOnce];
  struct alignas(16) {
    float z;
    int i;
    uint64_t w;
  } quick[kQuick];
  int bin, few;
  int bins[3];
  uint32_t before, listed, at;
  uint64_t mass, result;
};

__device__ __forceinline__ uint64_t shfl_up64(uint64_t x, int d) {
  const uint32_t lo = __shfl_up(static_cast<uint32_t>(x), d), hi = __shfl_up(static_cast<uint32_t>(x >> 32), d);
  return static_cast<uint64_t>(hi) << 32 | lo;
}

__device__ __forceinline__ uint64_t shfl64(uint64_t x, int l) {
  const uint32_t lo = __shfl(static_cast<uint32_t>(x), l), hi = __shfl(static_cast<uint32_t>(x >> 32), l);
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

// The eight logits of a thread in a chunk: fours at 4 t and 4 (1024 + t), -infinity behind the row's end.
template <int TYPE> __device__ __forceinline__ void load_eight(const void *z, int64_t row_at, int vocab, int chunk, float x[8]) {
  const int j = chunk * kChunk + 4 * threadIdx.x;
  if (vocab >= 4) {  // (loads that wait for nothing: a four that the row's end cuts is read again, one by one)
    load_four<TYPE>(z, row_at + min(j, vocab - 4), x);
    load_four<TYPE>(z, row_at + min(j + kChunk / 2, vocab - 4), x + 4);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = j + h * (kChunk / 2);
    if (at + 3 < vocab) continue;
#pragma unroll
    for (int k = 0; k < 4; ++k) x[4 * h + k] = at + k < vocab ? load_logit<TYPE>(z, row_at + at + k) : -__builtin_inff();
  }
}
__device__ __forceinline__ int index_of(int chunk, int k) {
  return chunk * kChunk + k / 4 * (kChunk / 2) + 4 * static_cast<int>(threadIdx.x) + k % 4;
}

// The range of a logit: `scale` per unit below the largest. It rises as x falls.
__device__ __forceinline__ float place_of(float top, float x, float scale) {
  return fminf((top - x) * scale, kBins - 1.f);
}

// What the steps of a row work with: its largest logit (-infinity: there is nothing
// to choose from), the limits, and the division into ranges.
struct Row {
  float most, scale, u, top_p;
  double c, reach;  // reach: no weight from there on
  int64_t top_k;
  uint64_t limit;   // weights that min_p leaves
  bool counted, by_range;
};
__device__ __forceinline__ Row row_of(Shared &s, const SampleArgs &a, int row) {
  const int lane = threadIdx.x & 63;
  Row r;
  float most = -__builtin_inff(), least = __builtin_inff();
  for (int k = lane; k < a.chunks; k += 64) {
    const Top top = a.tops[static_cast<int64_t>(row) * a.chunks + k];
    most = fmaxf(most, top.most), least = fminf(least, top.least);
  }
#pragma unroll
  for (int d = 32; d > 0; d /= 2) most = fmaxf(most, __shfl_xor(most, d)), least = fminf(least, __shfl_xor(least, d));
  float temperature = a.temperature ? a.temperature[row] : 1.f;
  r.most = most;
  r.top_k = a.top_k ? a.top_k[row] : 0;
  r.top_p = a.top_p ? a.top_p[row] : 1.f;
  const float min_p = a.min_p ? a.min_p[row] : 0.f, u = a.u[row];
  r.u = u > 0.f ? fminf(u, 0x1.fffffep-1f) : 0.f;
  if (!(temperature > 0.f)) temperature = 1.f, r.top_k = 1;  // the largest, the first of several
  r.counted = r.top_k > 0 && r.top_k < a.vocab;
  r.limit = min_p > 0.f ? static_cast<uint64_t>(ceil(static_cast<double>(fminf(min_p, 1.f)) * 0x1p44)) : 0;
  r.c = 92.332482616893653 / static_cast<double>(temperature);
  // Ranges as fine as those logits allow that have a weight at all. Rows with an
  // infinity, or too wide for fp32, go by their bits.
  r.reach = 46. * kFractions / r.c;
  const float width = fminf(most - least, static_cast<float>(fmin(r.reach, 3e38)));
  r.scale = width > 0.f ? (kBins - 1.f) / width : 1.f;
  r.by_range = most - least < 3e38f && r.scale < 3e38f && r.c > 0.;
  if (threadIdx.x < kFractions) {  // 2^44 times the powers 2^-1/2, 2^-1/4, .. 2^-1/64 of the index's bits
    constexpr double kRoots[] = {0x1.6a09e667f3bcdp-1, 0x1.ae89f995ad3adp-1, 0x1.d5818dcfba487p-1,
                                 0x1.ea4afa2a490dap-1, 0x1.f50765b6e4540p-1, 0x1.fa7c1819e90d8p-1};
    double p = 0x1p44;
#pragma unroll
    for (int b = 0; b < 6; ++b) p *= threadIdx.x >> (5 - b) & 1 ? kRoots[b] : 1.;
    s.table[threadIdx.x] = p;
  }
  return r;
}

// In front of the threads' counts and masses, in order, and (all) behind the last.
__device__ __forceinline__ void scan(Shared &s, uint32_t &n, uint64_t &m, uint32_t &all_n, uint64_t &all_m) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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
  // the wavefronts' sums, by every wavefront
  uint32_t wn = lane < kWaves ? s.wave_n[lane] : 0;
  uint64_t wm = lane < kWaves ? s.wave_m[lane] : 0;
#pragma unroll 1
  for (int d = 1; d < kWaves; d *= 2) {
    const uint32_t on = __shfl_up(wn, d);
    const uint64_t om = shfl_up64(wm, d);
    if (lane >= d) wn += on, wm += om;
  }
  all_n = __shfl(wn, kWaves - 1), all_m = shfl64(wm, kWaves - 1);
  const uint32_t before_n = __shfl(wn, max(wave - 1, 0));
  const uint64_t before_m = shfl64(wm, max(wave - 1, 0));
  n = sn - n + (wave > 0 ? before_n : 0), m = sm - m + (wave > 0 ? before_m : 0);
  __syncthreads();
}

// What workgroups of one launch give each other goes through their XCDs' L2s, both
// ways: a release and an acquire would write back and empty them (256 workgroups: 90 us).
template <class T> __device__ __forceinline__ void put(T *at, T v) {
  __hip_atomic_store(at, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T> __device__ __forceinline__ T get(const T *at) {
  return __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ Element get(const Element *at) {
  return __builtin_bit_cast(Element, get(reinterpret_cast<const uint64_t *>(at)));
}
// Whether this workgroup is the last of the row's to come here, all of whose `put`s
// are done then. The workgroups' numbers (below 2^20 together) are added: in s.at.
__device__ __forceinline__ bool last_here(Shared &s, uint32_t *arrived, int chunks, uint32_t number) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint32_t mine = (1u << 20) + number;
    s.at = __hip_atomic_fetch_add(arrived, mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + mine;
  }
  __syncthreads();
  return s.at >> 20 == static_cast<uint32_t>(chunks);
}

__device__ __forceinline__ Goal goal_of(const Row &r, int kind, uint64_t total) {
  const double mass = static_cast<double>(kind == UPTO ? r.u : r.top_p) * static_cast<double>(total);
  return Goal{kind, static_cast<uint32_t>(r.top_k), kind == BELOW ? fmax(mass, 0.5) : mass};
}

// Counts and masses in front of a range and behind it. Starts rise, so there is one
// range whose start is the last that a goal reaches.
struct Range {
  uint32_t n0, n1;
  uint64_t m0, m1;
  __device__ __forceinline__ bool is_last(const Goal &goal, int bin) const {
    return goal.reaches(n0, m0) && (bin == kBins - 1 || !goal.reaches(n1, m1));
  }
};
// The mass up to and with the last element whose start a goal reaches, and that
// element's index (-1: not by ranges), of the elements in the row's list.
__device__ __forceinline__ uint64_t resolve(Shared &s, const Element *list, int listed, const Element &own_element,
                                            const Range &own_range, const Row &r, const Weights &w, int per,
                                            const Goal &goal, int &index) {
  index = -1;
  const int t = threadIdx.x;
  if (own_range.is_last(goal, t)) s.bin = t, s.before = own_range.n0, s.mass = own_range.m0;
  if (t == 0) s.few = 0;
  __syncthreads();
  const int bin = s.bin;
  uint32_t before = s.before;
  uint64_t mass = s.mass;
  auto element = [&](int k) { return k < kThreads ? own_element : get(list + k); };  // k % kThreads = t
  // the elements of that range, then of one of its 1024 parts, then (equal ones) of one part of the indexes
  int sub = -1, part = -1;
  int members = 0;
#pragma unroll 1
  for (int depth = 0; depth < 3; ++depth) {
    auto fine = [&](const Element &e) {
      return min(static_cast<int>((place_of(r.most, e.z, r.scale) - static_cast<float>(bin)) * kThreads), kThreads - 1);
    };
    auto inside = [&](const Element &e) {
      return static_cast<int>(place_of(r.most, e.z, r.scale)) == bin && (sub < 0 || fine(e) == sub) &&
             (part < 0 || e.i / per == part);
    };
    for (int k = t; k < listed; k += kThreads) {
      const Element e = element(k);
      if (!inside(e)) continue;
      const int at = atomicAdd(&s.few, 1);
      if (at < kFew) s.few_z[at] = e.z, s.few_i[at] = e.i;
    }
    __syncthreads();
    members = s.few;
    // (ranking takes 0.08 us per element, dividing again 4 us)
    if (members <= (sub < 0 ? kFew / 16 : kFew)) break;
    const bool by_index = sub >= 0;
    if (part >= 0) return 0;
    if (by_index) {  // equal ones only
      if (t == 0) s.bin = 0;
      __syncthreads();
      const float first = s.few_z[0];
      bool other = false;
      for (int k = t; k < listed; k += kThreads) {
        const Element e = element(k);
        other = other || (inside(e) && e.z != first);
      }
      if (other) s.bin = 1;
      __syncthreads();
      if (s.bin) return 0;
    }
    s.n[t] = 0, s.m[t] = 0;
    __syncthreads();
    for (int k = t; k < listed; k += kThreads) {
      const Element e = element(k);
      if (!inside(e)) continue;
      const int at = by_index ? e.i / per : fine(e);
      atomicAdd(&s.n[at], 1u);
      atomicAdd(reinterpret_cast<unsigned long long *>(&s.m[at]), static_cast<unsigned long long>(w.of(e.z)));
    }
    __syncthreads();
    uint32_t n = s.n[t], all_n;
    uint64_t m = s.m[t], all_m;
    const uint32_t own_n = n;
    const uint64_t own_m = m;
    scan(s, n, m, all_n, all_m);
    n += before, m += mass;
    if (goal.reaches(n, m) && (t == kThreads - 1 || !goal.reaches(n + own_n, m + own_m))) s.bin = t, s.before = n, s.mass = m;
    if (t == 0) s.few = 0;
    __syncthreads();
    part = by_index ? s.bin : -1;
    sub = by_index ? sub : s.bin;
    before = s.before, mass = s.mass;
  }
  __syncthreads();
  if (members == 0 || members > kFew) return 0;
  const bool mine = t < members;
  uint64_t own = 0;
  if (mine) {
    s.few_w[t] = own = w.of(s.few_z[t]);
  } else if (t < members + kAtOnce) {  // behind all others, without a weight
    s.few_z[t] = -__builtin_inff(), s.few_i[t] = 0x7FFFFFFF, s.few_w[t] = 0;
  }
  if (t == 0) s.result = 0, s.before = 0;
  __syncthreads();
  if (mine) {
    const float x = s.few_z[t];
    const int i = s.few_i[t];
    for (int k0 = 0; k0 < members; k0 += kAtOnce) {
#pragma unroll
      for (int k = k0; k < k0 + kAtOnce; ++k) {
        const bool first = s.few_z[k] > x || (s.few_z[k] == x && s.few_i[k] < i);
        before += first;
        mass += first ? s.few_w[k] : 0;
      }
    }
    if (goal.reaches(before, mass)) {  // the last of those that it reaches has the largest sum, and the last place
      atomicMax(reinterpret_cast<unsigned long long *>(&s.result), static_cast<unsigned long long>(mass + own));
      atomicMax(&s.before, before);
    }
  }
  __syncthreads();
  if (mine && before == s.before && goal.reaches(before, mass)) s.few = s.few_i[t];
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

// The three selections among few elements in question, as nearly always, by one
// wavefront, which finds each one's place and its start at once. (The others of
// the workgroup end: 16 take turns at every instruction.)
__device__ __forceinline__ void pick_few(Shared &s, const SampleArgs &a, int row, const Element *list, int listed,
                                         const RowState &st, const Row &r, const Weights &w) {
  const int t = threadIdx.x;
  if (t >= kQuick) return;
  const bool mine = t < listed;
  const Element e = mine ? get(list + t) : Element{-__builtin_inff(), 0x7FFFFFFF};
  const int bin = static_cast<int>(place_of(r.most, e.z, r.scale));
  const uint64_t own = mine ? w.of(e.z) : 0;
  uint32_t n = st.n[bin];
  uint64_t m = st.m[bin], total = st.m[kBins];
  const uint64_t left = st.left;
  s.quick[t] = {e.z, e.i, own};
  if (t < 3) s.bins[t] = -1;
  __syncthreads();
  uint32_t with = 0;  // in front of it in its range
  for (int k0 = 0; k0 < listed; k0 += kAtOnce) {
#pragma unroll
    for (int k = k0; k < k0 + kAtOnce; ++k) {
      const auto o = s.quick[k];
      // (what is in front of it is not in a later range)
      const bool first = (o.z > e.z || (o.z == e.z && o.i < e.i)) && place_of(r.most, o.z, r.scale) >= static_cast<float>(bin);
      with += first;
      m += first ? o.w : 0;
    }
  }
  n += with;
  const int pos = bin * kQuick + static_cast<int>(with);  // rises along the order
#pragma unroll 1
  for (int kind = COUNT; kind <= UPTO; ++kind) {
    if (kind == COUNT && (!r.counted || st.hi[COUNT] < 0)) continue;
    if (kind == BELOW && !(r.top_p < 1.f)) continue;
    if (kind == UPTO) total = min(total, left);
    int last = mine && goal_of(r, kind, total).reaches(n, m) ? pos : -1;
#pragma unroll
    for (int d = 32; d > 0; d /= 2) last = max(last, __shfl_xor(last, d));
    if ((t & 63) == 0 && last >= 0) atomicMax(&s.bins[kind], last);
    __syncthreads();
    const bool is_last = mine && pos == s.bins[kind];
    if (kind == UPTO) {
      if (is_last) {
        a.tokens[row] = e.i;
        if (a.probs) a.probs[row] = static_cast<float>(w.value(e.z) / static_cast<double>(total));
      }
      break;
    }
    if (is_last) s.mass = m + own;
    __syncthreads();
    total = min(total, s.mass);
  }
}

// A chunk's largest logit and its smallest finite one.
template <int TYPE> __global__ __launch_bounds__(kThreads) void sample_top_kernel(SampleArgs a) {
  __shared__ float high[kWaves], low[kWaves];
  const int row = blockIdx.x, chunk = blockIdx.y;
  float x[8], most = -__builtin_inff(), least = __builtin_inff();
  load_eight<TYPE>(a.z, row * a.stride, a.vocab, chunk, x);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    most = fmaxf(most, x[k]);
    least = fminf(least, x[k] > -__builtin_inff() ? x[k] : __builtin_inff());
  }
#pragma unroll
  for (int d = 32; d > 0; d /= 2) most = fmaxf(most, __shfl_xor(most, d)), least = fminf(least, __shfl_xor(least, d));
  if ((threadIdx.x & 63) == 0) high[threadIdx.x >> 6] = most, low[threadIdx.x >> 6] = least;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int k = 1; k < kWaves; ++k) most = fmaxf(most, high[k]), least = fminf(least, low[k]);
  a.tops[static_cast<int64_t>(row) * a.chunks + chunk] = {most, least};
  if (chunk == 0) {
    RowState &st = a.rows[row];
    st.arrived[0] = st.arrived[1] = st.listed = 0;
  }
}

// A chunk's histogram; the row's last workgroup adds the chunks' and bounds the selections' places.
template <int TYPE> __global__ __launch_bounds__(kThreads) void sample_mass_kernel(SampleArgs a) {
  __shared__ Shared s;
  const int row = blockIdx.x, chunk = blockIdx.y, t = threadIdx.x;
  float x[8];
  load_eight<TYPE>(a.z, row * a.stride, a.vocab, chunk, x);
  const Row r = row_of(s, a, row);
  if (r.most == -__builtin_inff()) return;  // nothing to choose from
  s.n[t] = 0, s.m[t] = 0;
  __syncthreads();
  const Weights w{static_cast<double>(r.most), r.c, s.table};
  uint64_t left = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint64_t m;
    if (r.by_range)
      m = Weights::fixed(w.power(fmin(w.top - static_cast<double>(x[k]), r.reach), r.c));
    else
      m = w.of(x[k]);
    left += m >= r.limit ? m : 0;
    const int at = r.by_range ? static_cast<int>(place_of(r.most, x[k], r.scale)) : 0;
    if (r.counted && index_of(chunk, k) < a.vocab) atomicAdd(&s.n[at], 1u);
    if (m) atomicAdd(reinterpret_cast<unsigned long long *>(&s.m[at]), static_cast<unsigned long long>(m));
  }
  __syncthreads();
  Part *parts = a.parts + static_cast<int64_t>(row) * a.chunks;
  RowState &st = a.rows[row];
  put(&parts[chunk].n[t], s.n[t]), put(&parts[chunk].m[t], s.m[t]);
  if (r.limit > 0) left = sum_of(s, left);
  if (t == 0) put(&parts[chunk].left, left);
  if (!last_here(s, &st.arrived[0], a.chunks, 0)) return;

  uint32_t own_n = 0, all_n;  // of range t
  uint64_t own_m = 0, all_m;
#pragma unroll 4
  for (int k = 0; k < a.chunks; ++k) own_n += get(&parts[k].n[t]), own_m += get(&parts[k].m[t]);
  left = 0;
  if (r.limit > 0 && t < a.chunks) left = get(&parts[t].left);  // (a row has at most 64)
  if (r.limit > 0) left = sum_of(s, left);
  uint32_t n = own_n;
  uint64_t m = own_m;
  scan(s, n, m, all_n, all_m);
  if (r.limit == 0) left = all_m;
  const Range range{n, n + own_n, m, m + own_m};
  st.n[t] = n, st.m[t] = m;
  s.m[t] = m;
  if (t == 0) {
    st.n[kBins] = all_n, st.m[kBins] = s.m[kBins] = all_m;
    st.left = left;
  }
  // The last range whose start each selection reaches, for the least and the most that
  // the ones before it can leave.
  uint64_t lo_total = all_m, hi_total = all_m;
#pragma unroll 1
  for (int kind = COUNT; kind <= UPTO; ++kind) {
    int lo = 0, hi = -1;
    if (kind == UPTO) lo_total = min(lo_total, left), hi_total = min(hi_total, left);
    if (kind == COUNT ? r.counted : kind == BELOW ? r.top_p < 1.f : true) {
      if (t < 2) s.bins[t] = 0;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const Goal goal = goal_of(r, kind, k ? hi_total : lo_total);
        if (range.is_last(goal, t)) s.bins[k] = t;
      }
      __syncthreads();
      lo = s.bins[0], hi = s.bins[1];
      lo_total = min(lo_total, s.m[lo]), hi_total = min(hi_total, s.m[hi + 1]);
      // where top_k ends among elements without a weight, it leaves all the mass (peaked
      // rows, whose last range has most of the elements)
      if (kind == COUNT && s.m[lo] == s.m[hi + 1]) hi = -1;
      __syncthreads();
    }
    if (t == 0) st.lo[kind] = lo, st.hi[kind] = hi;
  }
}

// The elements of the ranges in question; the row's last workgroup makes the three
// selections: COUNT and BELOW leave less of the mass, UPTO chooses.
template <int TYPE> __global__ __launch_bounds__(kThreads) void sample_pick_kernel(SampleArgs a) {
  __shared__ Shared s;
  const int row = blockIdx.x, chunk = blockIdx.y, t = threadIdx.x;
  const int64_t row_at = row * a.stride;
  float x[8];
  load_eight<TYPE>(a.z, row_at, a.vocab, chunk, x);
  if (t == 0) s.listed = 0;
  const Row r = row_of(s, a, row);
  if (r.most == -__builtin_inff()) {
    if (chunk == 0 && t == 0) {
      a.tokens[row] = -1;
      if (a.probs) a.probs[row] = __builtin_bit_cast(float, 0x7FC00000u);
    }
    return;
  }
  RowState &st = a.rows[row];
  Element *list = a.list + static_cast<int64_t>(row) * a.room;
  const int lo[3] = {st.lo[0], st.lo[1], st.lo[2]}, hi[3] = {st.hi[0], st.hi[1], st.hi[2]};
  __syncthreads();
  if (r.by_range) {
    uint32_t take = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int at = static_cast<int>(place_of(r.most, x[k], r.scale));
      const bool in = (at >= lo[0] && at <= hi[0]) || (at >= lo[1] && at <= hi[1]) || (at >= lo[2] && at <= hi[2]);
      if (in && index_of(chunk, k) < a.vocab) take |= 1u << k;
    }
    uint32_t place = take ? atomicAdd(&s.listed, __popc(take)) : 0;
    __syncthreads();
    if (t == 0) s.at = s.listed ? atomicAdd(&st.listed, s.listed) : 0;
    __syncthreads();
    place += s.at;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (take >> k & 1) {
        if (place < kList)
          put(reinterpret_cast<uint64_t *>(list + place), __builtin_bit_cast(uint64_t, Element{x[k], index_of(chunk, k)}));
        ++place;
      }
  }
  if (!last_here(s, &st.arrived[1], a.chunks, s.listed)) return;

  const Weights w{static_cast<double>(r.most), r.c, s.table};
  const uint32_t listed = s.at & 0xFFFFFu;
  // Where ranges do not do, the selections go by the bits from there on.
  bool ranges = r.by_range && listed <= kList;
  if (ranges && listed <= kQuick) {
    pick_few(s, a, row, list, static_cast<int>(listed), st, r, w);
    return;
  }
  const int per = (a.vocab + kThreads - 1) / kThreads;  // indexes of a part, at most kFew
  const Range own_range{st.n[t], st.n[t + 1], st.m[t], st.m[t + 1]};
  const Element own_element = t < static_cast<int>(min(listed, static_cast<uint32_t>(kList))) ? get(list + t) : Element{0.f, 0};
  const uint64_t left = st.left;
  uint64_t total = st.m[kBins];
#pragma unroll 1
  for (int kind = COUNT; kind <= UPTO; ++kind) {
    if (kind == COUNT && (!r.counted || (ranges && st.hi[COUNT] < 0))) continue;
    if (kind == BELOW && !(r.top_p < 1.f)) continue;
    if (kind == UPTO) total = min(total, left);
    const Goal goal = goal_of(r, kind, total);
    uint64_t kept = 0;
    int index = -1;
    if (ranges) kept = resolve(s, list, listed, own_element, own_range, r, w, per, goal, index);
    if (index < 0) {
      ranges = false;
      const Found f = select<TYPE>(s, a.z, row_at, a.vocab, w, goal);
      const float chosen = logit_of(f.key);
      const uint64_t one = w.of(chosen);
      // of the equal ones, those whose start the goal reaches
      const double rest = one ? (goal.mass - static_cast<double>(f.mass)) / static_cast<double>(one) : 0.;
      double n = kind == COUNT ? static_cast<double>(goal.count - f.before) : kind == BELOW ? ceil(rest) : floor(rest) + 1.;
      n = fmin(fmax(n, 1.), static_cast<double>(f.ties));
      kept = f.mass + static_cast<uint64_t>(n) * one;
      if (kind == UPTO) index = nth<TYPE>(s, a.z, row_at, a.vocab, chosen, static_cast<uint32_t>(n) - 1);
    }
    if (kind != UPTO) {
      total = kept < total ? kept : total;
    } else if (t == 0) {
      a.tokens[row] = index;
      if (a.probs) a.probs[row] = static_cast<float>(w.value(load_logit<TYPE>(a.z, row_at + index)) / static_cast<double>(total));
    }
  }
}

int64_t chunks_of(int64_t vocab) { return (vocab + kChunk - 1) / kChunk; }
// Of a row's list: all that it can have, in whole lines.
int64_t room_of(int64_t vocab) { return std::min<int64_t>(kList, (vocab + 15) / 16 * 16); }

}  // namespace

int64_t sample_workspace_bytes(int64_t n_rows, int64_t vocab) {
  return n_rows * static_cast<int64_t>(sizeof(RowState) + room_of(vocab) * sizeof(Element) +
                                       chunks_of(vocab) * (sizeof(Part) + sizeof(Top)));
}

hipError_t launch_sample(const SampleCall &c, void *workspace, hipStream_t stream) {
  SampleArgs a{c.logits, c.row_stride, c.u, c.temperature, c.top_p, c.min_p, c.top_k, c.tokens, c.probs, static_cast<int>(c.vocab)};
  a.chunks = static_cast<int>(chunks_of(c.vocab)), a.room = static_cast<int>(room_of(c.vocab));
  a.rows = static_cast<RowState *>(workspace);
  a.list = reinterpret_cast<Element *>(a.rows + c.n_rows);
  a.parts = reinterpret_cast<Part *>(a.list + c.n_rows * a.room);
  a.tops = reinterpret_cast<Top *>(a.parts + c.n_rows * a.chunks);
  const dim3 grid(static_cast<unsigned>(c.n_rows), static_cast<unsigned>(a.chunks));
  auto go = [&](auto type) {
    constexpr int T = decltype(type)::value;
    hipError_t e = launch(sample_top_kernel<T>, grid, dim3(kThreads), 0, stream, a);
    if (e == hipSuccess) e = launch(sample_mass_kernel<T>, grid, dim3(kThreads), 0, stream, a);
    return e != hipSuccess ? e : launch(sample_pick_kernel<T>, grid, dim3(kThreads), 0, stream, a);
  };
  if (c.type == QMM_T_F32) return go(std::integral_constant<int, QMM_T_F32>{});
  if (c.type == QMM_T_F16) return go(std::integral_constant<int, QMM_T_F16>{});
  return go(std::integral_constant<int, QMM_T_BF16>{});
}

}  // namespace qmm
