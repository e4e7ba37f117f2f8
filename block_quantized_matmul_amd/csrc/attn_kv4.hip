// Attention of a decode batch over a 4-bit paged cache (qmm_attn_kv4; the
// cache's layout stands in qmm_serve.h).
//
// Bound by memory: 1.125 bytes per key and element for 4 group flops. What can
// keep it from that is the arithmetic that turns codes into operands, so the
// kernel spends as little as it can on a code:
//
//  * A dword of 8 codes becomes an operand of v_mfma_f32_16x16x32_f16 in five
//    instructions (one shift, four masks): a nibble n in the low bits of a half
//    is the subnormal n 2^-24, one in bits 4..7 is 16 n 2^-24, and the matrix
//    cores take subnormals exactly. The 16 is taken out of the other operand,
//    the 2^-24 out of the result, and the zero point 8 is a constant per column:
//    -8 sum q starts the scores' sum, 8 sum p is a column of its own, taken off in
//    the end. (Sums of subnormals are cut off downwards by some 2^-21 of their terms;
//    the difference of two such sums is not. With -8 sum p added, 60000 keys' outputs
//    were 7e-7 of the values too low, a third of their fp16 rounding.)
//  * A block's scale belongs to a key and 32 elements. The matrix cores' 16
//    columns hold H = 16 / NB query heads of the group times the NB = D / 32
//    blocks: column (h, b) of the first operand has q_h's elements of block b
//    and zeros elsewhere, so a lane gets the part of its score that block b
//    contributes, multiplies it by the key's one scale, and adds over the quad
//    of lanes (pair for D = 64) that holds the row. In the second product column
//    (h, b) is w_h d_b, the weight times the value's scale, and the rows of
//    block b are kept of its results. So scales cost one multiplication per
//    lane and key, not one per element.
//  * The scores' C layout (a lane has keys 4 g .. 4 g + 3 of a tile, g = lane /
//    16) is the second product's B layout if the values are read in the same
//    order of keys. Keys lie in the cache as the first operand needs them and are
//    loaded straight into registers, 16 bytes per lane (8 for D = 64); values
//    are copied to LDS and read by columns (ds_read_b64_tr_b4: 16 lanes take a
//    16 x 16 block of nibbles), the rows' addresses giving the order.
//
// Weights are binary16 in the second product, relative to two references: the
// row's maximum m (as in attn_core.h) and for each column an exponent E that
// follows the largest weight times scale, p = 2^(c x - c m - E) d, so that no product
// leaves binary16's range above, and those that do below are too small to count
// (whatever the scales alone: a key without a weight may have any). Each p is two
// numbers, the nearest and what is left, so that outputs are off by their own rounding
// alone (rms 2.0e-4 in fp16, 1.65e-3 in bf16; with the first number alone fp16 outputs
// of 700 and of 60000 keys by 2.8e-4). That costs 2 us of 49 and of 25 (below).
//
// Four wavefronts take chunks of 64 keys in turn, each with the next chunk on
// its way while it computes; they join through LDS. Where rows are few, their
// keys are split over workgroups, in ranges of one length for all rows, and a
// second launch joins them.
//
// Measured: 48 rows of up to 8000 keys (192000 in all), 8 KV heads of 128, groups of 4,
// bf16: 51 us + 5 for the join, 221 MB at 4.4 TB/s; 3 rows of up to 60000, 16 heads of
// 64, fp16: 27 + 5 us, 103 MB at 3.8 TB/s. Matrix cores are busy in 83 and 74 % of the
// cycles, vector instructions fill 52 and 67 %, and registers hold two to four wavefronts
// a SIMD, so waits are not always covered; a second chunk on its way is not built.
#include "attn_core.h"
#include "launch.h"
#include "serve.h"

#include <algorithm>

namespace qmm {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kChunk = 64;       // keys
constexpr int kTiles = kChunk / kKv4Tile;
// Tables of fewer than 5 x 256 keys are not worth a second launch: one row of 700 keys
// whole 9.5 us, divided 11.8; of 1000 10.0 and 12.0; of 1200 11.3 and 12.2 (in a graph,
// without the host's part, 8.2 and 9.1; 9.6 and 9.0; 11.1 and 9.1). The host does not
// know the lengths, so a short row in a wide table is divided.
constexpr int kFewestUnits = 5;
constexpr int kFewGroups = 1024;  // fewer workgroups than this, four per CU on 256 CUs: rows are split
// Workgroups of a CU that its registers hold: as many as run at once are wanted.
// Kernel and join of 48 rows of up to 8000 keys, of which 768 run at once, in 512, 768,
// 1024, 1536, 2048, 4096 workgroups: 66, 55, 61, 57, 61, 68 us; of 3 rows of 60000, of
// which 1024 do: 38, 32, 32, 36, 38, 49.
constexpr int resident(int64_t head_dim, int64_t columns) { return columns == 2 ? 2 : head_dim == 128 ? 3 : 4; }
constexpr float kWeightSlack = 4.f;  // weights up to 2^4
constexpr int kProductTop = 7;       // the largest product is in [2^7, 2^8) when the exponent is taken,
constexpr float kProductMost = 32768.f;  // and up to 2^15 before it follows
constexpr int kLeastExponent = -100;  // where it starts: weights up to 2^4 times scales below 2^16 stay within fp32

struct Kv4Args {
  const void *q;
  void *o;
  int64_t qt, qh, ot, oh;
  const uint8_t *cache;
  int64_t page_bytes, table_stride;
  const int32_t *tables, *lengths;
  float *part_o;   // [units][n_heads][D]
  float4_t *part;  // likewise: reference m, sum l, factor c
  int *first;      // [n_rows + 1]: a row's first unit
  int n_rows, n_heads, group, n_kv, tiles, want, cap;  // want: units of equal length wanted, or 0: rows are not split
  int n_pages, page_shift;
  float c0;  // scale * log2(e)
};

__device__ __forceinline__ int chunks_in(int n) { return n / kChunk + (n % kChunk != 0); }  // (n up to 2^31 - 1)
// Chunks of row r's keys; a length that the table does not hold is none.
__device__ __forceinline__ int chunks_of(const Kv4Args &a, int r) {
  const int n = r < a.n_rows ? a.lengths[r] : 0;
  return n < 0 || n > a.cap ? 0 : chunks_in(n);
}
// A unit of work is a range of a row's keys, all about the same length over all
// rows, whatever their lengths: every workgroup sums the lengths to get it, and
// counts the units of the rows before its own.
struct Unit {
  int row, split, used;  // unit `split` of the row's `used`; used = 0: none
};
__device__ __forceinline__ Unit find_unit(const Kv4Args &a, int unit, int lane) {
  if (a.want == 0) return Unit{unit, 0, 1};
  const int chunks0 = chunks_of(a, lane);
  int64_t total = chunks0;
  for (int r = 64; r < a.n_rows; r += 64) total += chunks_of(a, r + lane);
#pragma unroll
  for (int d = 1; d < 64; d *= 2) total += __shfl_xor(total, d);
  const int each = static_cast<int>(max(static_cast<int64_t>(kWaves), (total + a.want - 1) / a.want));
  int before = 0;
  for (int r0 = 0; r0 < a.n_rows; r0 += 64) {
    const int r = r0 + lane;
    const int chunks = r0 == 0 ? chunks0 : chunks_of(a, r);
    const int units = r >= a.n_rows ? 0 : max(1, chunks / each + (chunks % each != 0));
    int upto = units;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int other = __shfl_up(upto, d);
      upto += lane >= d ? other : 0;
    }
    const int first = before + upto - units;
    if (unit == 0 && r < a.n_rows) a.first[r] = first;
    const uint64_t here = __ballot(unit >= first && unit < first + units);
    before += __builtin_amdgcn_readlane(upto, 63);
    if (here != 0 && unit != 0) {
      const int l = __builtin_ctzll(here);
      return Unit{r0 + l, unit - __builtin_amdgcn_readlane(first, l), __builtin_amdgcn_readlane(units, l)};
    }
  }
  if (unit != 0) return Unit{0, 0, 0};
  a.first[a.n_rows] = before;
  return Unit{0, 0, max(1, __builtin_amdgcn_readfirstlane(chunks0) / each + (__builtin_amdgcn_readfirstlane(chunks0) % each != 0))};
}

// 8 codes as halves: element order 0, 4, 1, 5, 2, 6, 3, 7, in units of 2^-24
// (elements 0, 4, 2, 6) and 2^-20 (1, 5, 3, 7).
__device__ __forceinline__ half8_t unpack_codes(uint32_t v) {
  const uint32_t u = v >> 8;
  return __builtin_bit_cast(half8_t, u32x4_t{v & 0x000F000Fu, v & 0x00F000F0u, u & 0x000F000Fu, u & 0x00F000F0u});
}
__device__ __forceinline__ int code_of(int j) { return (j & 1) * 4 + j / 2; }    // the element at place j
__device__ __forceinline__ bool times16(int j) { return (j / 2) & 1; }           // whether it is 16 times as large

// 16 bytes per lane from base + offset, the lane's own, into LDS at lds + 16 lane.
__device__ __forceinline__ void dma_lane_to_lds(const uint8_t *base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset), "s"(base), "s"(lds)
               : "memory", "m0");
}

__device__ __forceinline__ float max_over_rows(float x) {  // over lanes l, l ^ 16, l ^ 32, l ^ 48
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const float2_t two = both_halves(fmaxf(__builtin_bit_cast(float, static_cast<uint32_t>(r[0])),
                                         __builtin_bit_cast(float, static_cast<uint32_t>(r[1]))));
  return fmaxf(two.x, two.y);
}
__device__ __forceinline__ float sum_over_rows(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const float2_t two = both_halves(__builtin_bit_cast(float, static_cast<uint32_t>(r[0])) +
                                   __builtin_bit_cast(float, static_cast<uint32_t>(r[1])));
  return two.x + two.y;
}
// The same value, but one that the compiler does not compute ahead of the loop
// and then keep in scratch memory, whose loads would wait for all others.
__device__ __forceinline__ uint32_t here(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}
template <int CTRL> __device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}
// Sum over the NB neighbouring lanes of a row's blocks, in every one of them.
template <int NB> __device__ __forceinline__ float sum_over_blocks(float x) {
  x += dpp<0xB1>(x);                             // quad_perm 1, 0, 3, 2
  if constexpr (NB == 4) x += dpp<0x4E>(x);      // quad_perm 2, 3, 0, 1
  return x;
}
__device__ __forceinline__ float half_at(u32x2_t v, int r) {
  return half_bits_to_float(r < 2 ? (r & 1 ? v.x >> 16 : v.x & 0xFFFFu) : (r & 1 ? v.y >> 16 : v.y & 0xFFFFu));
}

// One column tile's query heads and running state.
template <int D> struct Column {
  static constexpr int NB = D / 32;
  half8_t q[NB];      // the first product's operand for block b: zeros but in columns (h, b)
  float start;        // -8 sum q, where the scores' sum starts
  float c;            // weights are 2^(c x - c m) for raw scores x
  float m, mu_e, l;   // reference, its Reference::mu plus E, this lane's part of the sum
  int e;              // E
  float4_t o[D / 16];  // outputs 16 dt + 4 g + r of column lane % 16, in units of 2^(E - 24), but for
  float4_t zero;      // 8 sum p, to be taken from each
};

template <class E, int D> __device__ __forceinline__ void start_column(Column<D> &s, const Kv4Args &a, int row, int head0,
                                                                       int heads, int lane) {
  constexpr int NB = D / 32;
  const int col = lane & 15, g = lane >> 4, b = col % NB;
  const int head = head0 + min(col / NB, heads - 1);
  const typename E::v8 in = *reinterpret_cast<const typename E::v8 *>(static_cast<const typename E::one *>(a.q) +
                                                                      row * a.qt + head * a.qh + 32 * b + 8 * g);
  float f[8], most = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = static_cast<float>(in[j]), most = fmaxf(most, __builtin_fabsf(f[j]));
  most = max_over_rows(most);
  most = fmaxf(most, dpp<0xB1>(most));
  if constexpr (NB == 4) most = fmaxf(most, dpp<0x4E>(most));
  // the row's largest element in [2^12, 2^13), a power of two away from its value
  const int ex = most > 0.f && most < __builtin_inff() ? (__builtin_amdgcn_frexp_expf(most) - 1) : 0;
  half8_t q;
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = __builtin_ldexpf(f[code_of(j)], 12 - ex - (times16(j) ? 4 : 0));
    q[j] = static_cast<_Float16>(x);
    sum += static_cast<float>(q[j]) * (times16(j) ? 16.f : 1.f);
  }
#pragma unroll
  for (int k = 0; k < NB; ++k) s.q[k] = k == b ? q : half8_t{};
  s.start = -8.f * 0x1p-24f * sum_over_rows(sum);
  // Within fp32's normal range: scores so large that this clips it differ by more
  // than 2^80 or not at all, and so small that it does are all the same.
  s.c = fminf(fmaxf(__builtin_ldexpf(a.c0, 12 + ex), 0x1p-126f), 0x1p126f);
  s.m = -__builtin_inff();
  s.mu_e = s.l = 0.f;
  s.e = kLeastExponent;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) s.o[i] = float4_t{};
  s.zero = float4_t{};
}

// Weights of a chunk's raw scores x (a lane's keys 16 t + 4 g + r), times the
// values' scales, as the second product's operands of its two steps, and what
// their rounding leaves.
template <int D>
__device__ __forceinline__ void weigh(Column<D> &s, float x[kTiles][4], const u32x2_t dv[kTiles], half8_t p[2][2]) {
  float mx = fmaxf(x[0][0], x[0][1]);
#pragma unroll
  for (int i = 2; i < 4 * kTiles; ++i) mx = fmaxf(mx, x[i / 4][i % 4]);
  mx = max_over_rows(mx);
  float f = 1.f;  // from sums relative to the old m to those relative to the new one
  const bool moved = __any((mx - s.m) * s.c > kWeightSlack);
  if (moved) {
    const float m = fmaxf(s.m, mx);
    f = rescaling(s.m, m, s.c);
    s.m = m, s.l *= f;
    s.mu_e = Reference(m, s.c).mu + static_cast<float>(s.e);
  }
  const float sub = Reference(s.m, s.c).sub;
  if (__any(sub != 0.f)) {
#pragma unroll
    for (int i = 0; i < 4 * kTiles; ++i) x[i / 4][i % 4] -= sub;
  }
  float sum[2] = {0.f, 0.f}, most = 0.f;  // (a NaN is not above others: its column is NaNs whatever E)
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int j = 4 * (t & 1) + r;  // the key's place in its step: one whose codes count 16 times has a 16th of the weight
      const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][r], s.c, -s.mu_e - (times16(j) ? 4.f : 0.f)));
      sum[times16(j)] += w;
      x[t][r] = __builtin_fmaf(w, half_at(dv[t], r), 0.f);
      most = fmaxf(most, __builtin_fabsf(x[t][r]));
    }
  s.l += __builtin_ldexpf(__builtin_fmaf(sum[1], 16.f, sum[0]), s.e);
  if (moved || __any(most > kProductMost)) {
    // The largest product so far: the chunk's, or one before, which was 2^7 at least when E was taken. Without
    // any, E starts again.
    most = fmaxf(__builtin_ldexpf(f, kProductTop), max_over_rows(most));
    const int least = kLeastExponent - s.e;
    const int up = most > 0.f ? max(__builtin_amdgcn_frexp_expf(most) - 1 - kProductTop, least) : least;
    s.e += up, s.mu_e += static_cast<float>(up);
    const float down = __builtin_ldexpf(1.f, -up);
#pragma unroll
    for (int i = 0; i < 4 * kTiles; ++i) x[i / 4][i % 4] *= down;
    f *= down;
    s.zero *= f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) s.o[i] *= f;
  }
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) p[0][t >> 1][4 * (t & 1) + r] = static_cast<_Float16>(x[t][r]);
  float minus = -1.f;
  asm("" : "+s"(minus));  // (or the subtraction's operand is converted by an instruction of its own)
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    const u32x4_t u = __builtin_bit_cast(u32x4_t, p[0][t >> 1]);
    const u32x2_t four = t & 1 ? u32x2_t{u.z, u.w} : u32x2_t{u.x, u.y};
#pragma unroll
    for (int r = 0; r < 4; ++r)
      p[1][t >> 1][4 * (t & 1) + r] = static_cast<_Float16>(__builtin_fmaf(half_at(four, r), minus, x[t][r]));
  }
}

template <class E, int D, int CT>
__global__ __launch_bounds__(kThreads, resident(D, CT)) void attn_kv4_kernel(Kv4Args a) {
  typedef typename E::one one;
  constexpr int NB = D / 32, H = 16 / NB;
  constexpr int kBuffer = kChunk * D / 2;  // bytes of a chunk's value codes
  constexpr int kRow = D / 2;
  constexpr int kJoin = CT * 10 * 64 * 4;  // bytes a wavefront leaves for the join
  __shared__ __align__(1024) uint8_t lds[kWaves * (2 * kBuffer > kJoin ? 2 * kBuffer : kJoin)];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  // KV heads are the fastest index, so that workgroups on the same keys share an XCD's L2
  const int kv = blockIdx.x % a.n_kv, ct0 = blockIdx.x / a.n_kv % a.tiles * CT, unit = blockIdx.x / a.n_kv / a.tiles;
  const Unit u = find_unit(a, unit, lane);
  const int row = u.row, split = u.split, used = u.used;
  if (used == 0) return;
  const int len = __builtin_amdgcn_readfirstlane(a.lengths[row]);
  const bool bad_len = len < 0 || len > a.cap;
  const int n = bad_len ? 0 : len;
  const int chunks = chunks_in(n);
  const int lo = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<int64_t>(split) * chunks / used));
  const int hi = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<int64_t>(split + 1) * chunks / used));
  const int mine = max(0, (hi - lo - wave + kWaves - 1) / kWaves);  // chunks lo + wave, + kWaves, ..

  Column<D> s[CT];
#pragma unroll
  for (int k = 0; k < CT; ++k) {
    const int first = min((ct0 + k) * H, a.group - 1);
    start_column<E, D>(s[k], a, row, kv * a.group + first, min(H, a.group - first), lane);
  }
  bool poison = bad_len;

  if (mine > 0) {
    const int32_t *table = a.tables + row * a.table_stride;
    const int last_tile = (n - 1) / kKv4Tile;
    const int tile_shift = a.page_shift - 4;  // tiles per page
    const int64_t head_off = (static_cast<int64_t>(kv) << tile_shift) * kv4_tile_bytes(D);
    const uint32_t buf0 = lds_addr(lds) + wave * 2 * kBuffer;
    // the pages of the next 16 of the wavefront's chunks, four tiles each
    int ids = 0;
    auto fetch_ids = [&](int i) {
      const int c = min(lo + wave + kWaves * (i + lane / kTiles), hi - 1);
      const int id = table[min(c * kTiles + lane % kTiles, last_tile) >> tile_shift];
      const bool bad = id < 0 || id >= a.n_pages;
      poison = poison || __any(bad);
      ids = bad ? 0 : id;
    };
    uint32_t kc[kTiles][NB];
    u32x2_t dk[kTiles], dv[kTiles];
    const uint8_t *base[kTiles];
    auto locate = [&](int i) {
      const int c = lo + wave + kWaves * i;
      if ((i & 15) == 0) fetch_ids(i);
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        const int id = __builtin_amdgcn_readlane(ids, (i & 15) * kTiles + t);
        const int tile = min(c * kTiles + t, last_tile) & ((1 << tile_shift) - 1);
        base[t] = a.cache + static_cast<int64_t>(id) * a.page_bytes + head_off + tile * kv4_tile_bytes(D);
      }
    };
    const int scale_at = 2 * (16 * (col % NB) + 4 * g);
    auto load_keys = [&]() {
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        if constexpr (NB == 4) {
          const u32x4_t v = *reinterpret_cast<const u32x4_t *>(base[t] + 16 * lane);
#pragma unroll
          for (int b = 0; b < NB; ++b) kc[t][b] = v[b];
        } else {
          const u32x2_t v = *reinterpret_cast<const u32x2_t *>(base[t] + 8 * lane);
#pragma unroll
          for (int b = 0; b < NB; ++b) kc[t][b] = v[b];
        }
        dk[t] = *reinterpret_cast<const u32x2_t *>(base[t] + 16 * D + scale_at);
      }
    };
    // Rows of the values' codes, the 16-byte chunk c of a row of tile t at c ^ t, so that
    // the 16 rows of a read (four of each tile) lie on different banks
    auto copy_values = [&](int buffer) {
      const uint32_t to = buf0 + buffer * kBuffer, l = here(lane);
      if constexpr (D == 128) {
        const uint32_t at = 8 * D + 16 * l;  // row l / 4, chunk l % 4
#pragma unroll
        for (int t = 0; t < kTiles; ++t) dma_lane_to_lds(base[t], at ^ (16 * t), to + t * 1024);
      } else {
#pragma unroll
        for (int t = 0; t < kTiles; t += 2) {  // two tiles, each by half of the lanes
          const uint32_t at = 8 * D + ((16 * l % 512) ^ (16 * (l / 32)));
          if (lane < 32) dma_lane_to_lds(base[t], at, to + t * 512);
          if (lane >= 32) dma_lane_to_lds(base[t + 1], at, to + t * 512);
        }
      }
    };
    auto load_scales = [&]() {
#pragma unroll
      for (int t = 0; t < kTiles; ++t) dv[t] = *reinterpret_cast<const u32x2_t *>(base[t] + 17 * D + scale_at);
    };
    // this lane's row of a read by columns: nibble i of the result, of step i / 8, is place j of the operand
    const int ri = lane & 15, rj = (ri & 3) * 2 + ((ri >> 2) & 1);
    const int r_tile = 2 * (ri >> 3) + (rj >> 2), r_row = 16 * r_tile + 4 * g + (rj & 3);
    const uint32_t v_at = r_row * kRow + 16 * (r_tile & (D / 32 - 1));
    const half8_t eights = __builtin_bit_cast(half8_t, u32x4_t{0x00080008u, 0x00800080u, 0x00080008u, 0x00800080u});

    locate(0);
    load_keys();
    copy_values(0);
    load_scales();
    for (int i = 0; i < mine; ++i) {
      wait_loads<0>();
      float x[CT][kTiles][4];
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        float4_t acc[CT];
#pragma unroll
        for (int k = 0; k < CT; ++k) acc[k] = float4_t{s[k].start, s[k].start, s[k].start, s[k].start};
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const half8_t keys = unpack_codes(kc[t][b]);
#pragma unroll
          for (int k = 0; k < CT; ++k) acc[k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(keys, s[k].q[b], acc[k], 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < CT; ++k)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            x[k][t][r] = sum_over_blocks<NB>(__builtin_fmaf(acc[k][r], half_at(dk[t], r), 0.f));
      }
      const int left = n - (lo + wave + kWaves * i) * kChunk;
      if (left < kChunk) {  // places past the length: no weight, and no scale, which may be a NaN
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          const int keep = left - 16 * t - 4 * static_cast<int>(here(g));
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (r >= keep) {
#pragma unroll
              for (int k = 0; k < CT; ++k) x[k][t][r] = -__builtin_inff();
            }
          dv[t].x = keep >= 2 ? dv[t].x : keep == 1 ? dv[t].x & 0xFFFFu : 0;
          dv[t].y = keep >= 4 ? dv[t].y : keep == 3 ? dv[t].y & 0xFFFFu : 0;
        }
      }
      const bool more = i + 1 < mine;
      if (more) {
        locate(i + 1);
        load_keys();
        wait_reads();
        copy_values((i + 1) & 1);
      }
      half8_t p[CT][2][2];
#pragma unroll
      for (int k = 0; k < CT; ++k) weigh<D>(s[k], x[k], dv, p[k]);
      if (more) load_scales();
      const uint32_t va = here(buf0 + (i & 1) * kBuffer + v_at);
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt) {
        typedef int int2_t __attribute__((ext_vector_type(2)));
        const int2_t v = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
            reinterpret_cast<__attribute__((address_space(3))) int2_t *>((va ^ (16 * (dt / 2))) + 8 * (dt & 1)));
#pragma unroll
        for (int step = 0; step < 2; ++step) {
          const half8_t values = unpack_codes(static_cast<uint32_t>(v[step]));
#pragma unroll
          for (int k = 0; k < CT; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              s[k].o[dt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(values, p[k][h][step], s[k].o[dt], 0, 0, 0);
        }
      }
#pragma unroll
      for (int step = 0; step < 2; ++step)
#pragma unroll
        for (int k = 0; k < CT; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            s[k].zero = __builtin_amdgcn_mfma_f32_16x16x32_f16(eights, p[k][h][step], s[k].zero, 0, 0, 0);
    }
  }

  // The wavefronts' parts: a lane has outputs 32 b + 16 k + 4 g + r of its column's head.
  __syncthreads();
  float *mine_at = reinterpret_cast<float *>(lds) + wave * (kJoin / 4);
#pragma unroll
  for (int k = 0; k < CT; ++k) {
    const int b = col % NB;
    const float unit_v = __builtin_ldexpf(1.f, s[k].e + 24);
    float *at = mine_at + k * 640 + lane;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float v = s[k].o[i][r];
#pragma unroll
        for (int q = 1; q < NB; ++q) v = b == q ? s[k].o[2 * q + i][r] : v;
        at[(4 * i + r) * 64] = (v - s[k].zero[r]) * unit_v;
      }
    const float l = sum_over_rows(s[k].l);
    at[8 * 64] = s[k].m;
    at[9 * 64] = poison ? __builtin_bit_cast(float, 0x7FC00000u) : l;
  }
  __syncthreads();
  if (wave >= CT) return;
  const int k = wave;
  const int in_group = (ct0 + k) * H + col / NB;
  if (in_group >= a.group) return;
  const float *at = reinterpret_cast<const float *>(lds) + k * 640 + lane;
  float c = s[0].c;
  if constexpr (CT == 2) c = k == 1 ? s[1].c : c;
  float m = at[8 * 64], l = 0.f, v[8];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) m = fmaxf(m, at[w * (kJoin / 4) + 8 * 64]);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const float *from = at + w * (kJoin / 4);
    const float f = rescaling(from[8 * 64], m, c);
    l = __builtin_fmaf(from[9 * 64], f, l);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_fmaf(from[i * 64], f, v[i]);
  }
  const int head = kv * a.group + in_group, e0 = 32 * (col % NB) + 4 * g;
  if (used == 1) {
    const float f = len == 0 ? 0.f : 1.f / l;  // with keys, but no weight, 0 / 0
    one *out = static_cast<one *>(a.o) + row * a.ot + head * a.oh + e0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      typename E::v4 y;
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] = static_cast<one>(E::limit(len == 0 ? 0.f : v[4 * i + r] * f));
      *reinterpret_cast<typename E::v4 *>(out + 16 * i) = y;
    }
  } else {
    const int64_t item = static_cast<int64_t>(unit) * a.n_heads + head;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<float4_t *>(a.part_o + item * D + e0 + 16 * i) =
          float4_t{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
    if (col % NB == 0 && g == 0) a.part[item] = float4_t{m, l, c, 0.f};
  }
}

// Joins the units of a row's head: a wavefront, D / 4 lanes per unit with four
// outputs each, so that 2 (D = 64: 4) units are summed at a time.
template <class E, int D> __global__ __launch_bounds__(kThreads) void attn_kv4_join_kernel(Kv4Args a) {
  typedef typename E::one one;
  constexpr int kFours = D / 4, kAtOnce = 64 / kFours;
  const int lane = threadIdx.x & 63;
  const int item = __builtin_amdgcn_readfirstlane(static_cast<int>(blockIdx.x * kWaves + (threadIdx.x >> 6)));
  if (item >= a.n_rows * a.n_heads) return;
  const int row = item / a.n_heads, head = item % a.n_heads;
  const int first = a.first[row], used = a.first[row + 1] - first;
  if (used == 1) return;  // written already
  const float4_t *part = a.part + static_cast<int64_t>(first) * a.n_heads + head;
  const float *part_o = a.part_o + (static_cast<int64_t>(first) * a.n_heads + head) * D + 4 * (lane % kFours);
  float m = -__builtin_inff();
  for (int k = lane; k < used; k += 64) m = fmaxf(m, part[static_cast<int64_t>(k) * a.n_heads][0]);
#pragma unroll
  for (int d = 1; d < 64; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
  float l = 0.f;
  float4_t v{};
#pragma unroll 4
  for (int k = lane / kFours; k < used; k += kAtOnce) {
    const float4_t p = part[static_cast<int64_t>(k) * a.n_heads];
    const float4_t o = *reinterpret_cast<const float4_t *>(part_o + static_cast<int64_t>(k) * a.n_heads * D);
    const float f = rescaling(p[0], m, p[2]);
    l = __builtin_fmaf(p[1], f, l);
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf(o[r], f, v[r]);
  }
#pragma unroll
  for (int d = kFours; d < 64; d *= 2) {
    l += __shfl_xor(l, d);
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] += __shfl_xor(v[r], d);
  }
  if (lane >= kFours) return;
  typename E::v4 y;
#pragma unroll
  for (int r = 0; r < 4; ++r) y[r] = static_cast<one>(E::limit(v[r] * (1.f / l)));
  *reinterpret_cast<typename E::v4 *>(static_cast<one *>(a.o) + row * a.ot + head * a.oh + 4 * lane) = y;
}

// Outputs: means of values up to 8 times binary16's largest scale. Where the
// rounding of the weights alone takes one past binary16's largest value, it is that.
struct OutF16 : ElemF16 {
  __device__ static __forceinline__ float limit(float x) {
    return __builtin_fabsf(x) < largest * 1.001f ? __builtin_amdgcn_fmed3f(x, -largest, largest) : x;
  }
};

template <class E, int D> hipError_t run(const Kv4Args &a, const Kv4Plan &p, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.units * p.tiles * a.n_kv));
  const hipError_t e = p.columns == 2 ? launch(attn_kv4_kernel<E, D, 2>, grid, dim3(kThreads), 0, stream, a)
                                      : launch(attn_kv4_kernel<E, D, 1>, grid, dim3(kThreads), 0, stream, a);
  if (e != hipSuccess || p.want == 0) return e;
  return launch(attn_kv4_join_kernel<E, D>, dim3(static_cast<unsigned>((a.n_rows * a.n_heads + kWaves - 1) / kWaves)),
                dim3(kThreads), 0, stream, a);
}

}  // namespace

Kv4Plan kv4_plan(int64_t n_rows, int64_t n_q_heads, int64_t n_kv_heads, int64_t head_dim, int64_t cap) {
  const int64_t group = n_q_heads / n_kv_heads, per = 16 / (head_dim / 32);
  Kv4Plan p{};
  const int64_t columns = (group + per - 1) / per;
  p.columns = columns > 1 ? 2 : 1;
  p.tiles = (columns + p.columns - 1) / p.columns;
  const int64_t per_unit = n_kv_heads * p.tiles, most = cap / (kWaves * kChunk);
  p.units = n_rows;
  if (n_rows > 0 && n_rows * per_unit < kFewGroups && most >= kFewestUnits) {
    // half a range per row more, since a row's last is short on average
    p.want = std::max(n_rows, 256 * resident(head_dim, p.columns) / per_unit - n_rows / 2);
    // sum_r max(1, ceil(chunks_r / each)), each at least total / want and kWaves
    p.units = std::min(p.want + n_rows, n_rows * (most + 1));
  }
  return p;
}

int64_t kv4_workspace_bytes(const Kv4Plan &p, int64_t n_rows, int64_t n_q_heads, int64_t head_dim) {
  // a unit's head: its outputs, reference, sum, factor and a spare
  return p.want == 0 ? 0 : p.units * n_q_heads * (head_dim + 4) * 4 + (n_rows + 1 + 3) / 4 * 16;
}

hipError_t launch_attn_kv4(int type, const qmm_heads &Q, const qmm_heads &O, int64_t n_rows, int64_t n_q_heads,
                           int64_t n_kv_heads, int64_t head_dim, const Kv4Cache &cache, const int32_t *tables,
                           int64_t table_stride, int64_t table_width, const int32_t *lengths, float scale,
                           void *workspace, hipStream_t stream) {
  const int64_t cap = table_width * cache.page_tokens;
  const Kv4Plan p = kv4_plan(n_rows, n_q_heads, n_kv_heads, head_dim, cap);
  Kv4Args a{};
  a.q = Q.data, a.o = O.data, a.qt = Q.token_stride, a.qh = Q.head_stride, a.ot = O.token_stride, a.oh = O.head_stride;
  a.cache = cache.data, a.page_bytes = cache.page_bytes, a.tables = tables, a.table_stride = table_stride;
  a.lengths = lengths;
  a.part_o = static_cast<float *>(workspace);
  a.part = reinterpret_cast<float4_t *>(a.part_o + p.units * n_q_heads * head_dim);
  a.first = reinterpret_cast<int *>(a.part + p.units * n_q_heads);
  a.n_rows = static_cast<int>(n_rows), a.n_heads = static_cast<int>(n_q_heads);
  a.group = static_cast<int>(n_q_heads / n_kv_heads), a.n_kv = static_cast<int>(n_kv_heads);
  a.tiles = static_cast<int>(p.tiles), a.want = static_cast<int>(p.want), a.cap = static_cast<int>(cap);
  a.n_pages = static_cast<int>(cache.n_pages), a.page_shift = cache.page_shift;
  a.c0 = scale * 1.4426950408889634f;
  auto by_dim = [&](auto elem) {
    typedef decltype(elem) E;
    return head_dim == 128 ? run<E, 128>(a, p, stream) : run<E, 64>(a, p, stream);
  };
  return type == QMM_T_F16 ? by_dim(OutF16{}) : by_dim(ElemBF16{});
}

}  // namespace qmm
