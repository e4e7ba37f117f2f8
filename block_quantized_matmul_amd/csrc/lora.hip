// Low-rank adapters of many requests beside a shared projection (qmm_lora).
//
//   V[t] = A_a X[t]        (rank values, a = ids[t])
//   Y[t] = base[t] + s_a B_a V[t]
//
// Two launches on the matrix cores over tiles of 16 tokens; both are bound by
// memory (X, base and Y pass once, the adapters' bytes are few), or by
// latency where the batch is small. An fp16 X is multiplied as it is; an fp32
// X, and V in the second launch, run on the fp32 matrix instruction with A and
// B widened, so nothing is rounded to fewer than 32 bits.
//
// What a tile is:
//  * up to kGroupTokens tokens (a decode batch: neighbours rarely share an
//    adapter), up to 16 tokens of one adapter. The workgroups of token t count
//    the earlier tokens with its id; if their number is a multiple of 16 they
//    take t and the next 15 tokens with that id, else they leave. No launch
//    sorts anything, and all adapters run at once;
//  * more tokens (prompts: the tokens of a request stand together), 16
//    consecutive tokens. A tile that does hold several adapters takes them one
//    after another and keeps, in each token's column, its own adapter's result.
// Columns do not mix, so a non-finite value of another token or adapter stays
// out in both.
//
// The first launch splits k and leaves partial sums of V in the workspace,
// which the second adds in order (no atomics).
#include "attn.h"
#include "common.h"
#include "launch.h"

#include <algorithm>

namespace qmm {

namespace {

constexpr int kThreads = 256;
constexpr int kTok = 16;            // tokens per tile
constexpr int kGroupTokens = 512;   // largest batch in tiles by adapter
constexpr int kGroupSlab = 64;      // k per wavefront and round, tiles by adapter
constexpr int kMaxSplits = 256;     // ranges of k, tiles by adapter
constexpr int kRankGroup = 64;      // ranks per workgroup of the first launch
constexpr int kTileWaves = 2048;    // wavefronts the first launch aims at, consecutive tiles

// Tiles by adapter: the tokens of workgroup `t`'s tile, by their ids' order in
// the batch, in slot[0 .. 15] of LDS (-1 behind the last). False if t does
// not begin a tile. One wavefront scans the batch, 64 ids at a time.
__device__ __forceinline__ bool group_of(const int32_t *ids, int n_tokens, int t, int *slot, int &id) {
  __shared__ int begins;
  id = ids[t];
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    if (lane < kTok) slot[lane] = -1;
    int before = 0, rank = 0;  // same id: in the chunks so far, and before t
    bool own = false;
    for (int i0 = 0; i0 < n_tokens; i0 += 64) {
      const int i = i0 + lane;
      const bool same = i < n_tokens && ids[i] == id;
      const uint64_t mask = __ballot(same);
      if (i0 <= t && t < i0 + 64) {
        rank = before + __popcll(mask & ((uint64_t{1} << (t - i0)) - 1));
        own = rank % kTok == 0;
        if (!own) break;
      }
      if (own) {
        const int at = before + __popcll(mask & ((uint64_t{1} << lane) - 1)) - rank;
        if (same && at >= 0 && at < kTok) slot[at] = i;
        if (before + __popcll(mask) - rank >= kTok) break;
      }
      before += __popcll(mask);
    }
    if (lane == 0) begins = own;
  }
  __syncthreads();
  return begins != 0;
}

// The adapters of a tile's tokens, one after another: f(a, mine) with mine
// true in the lanes whose token (lane % 16) has id a. Ids outside
// [0, n_adapters) are left out.
template <class F> __device__ __forceinline__ void each_adapter(int id, int n_adapters, F f) {
  uint32_t left = static_cast<uint32_t>(__ballot(id >= 0 && id < n_adapters)) & 0xFFFFu;
  while (left != 0) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
    const bool mine = id == a;
    left &= ~static_cast<uint32_t>(__ballot(mine));
    f(a, mine);
  }
}

struct DownArgs {
  const void *x;
  const _Float16 *a;
  const int32_t *ids;
  float *v;  // [splits][n_tokens][rank]
  int64_t n_tokens, k, range;  // range: k per split
  int n_adapters, rank;
};

// V^T = A X^T on one wavefront: 16 RT ranks of one adapter, the tokens of the
// lanes' columns, k from begin to end (multiples of 32). The C layout gives a
// lane four consecutive ranks of token lane % 16. Operand element j of lane
// group g = lane / 16 is the same k for both operands; which k it is does not
// matter to the sum, so an fp32 lane takes 4 consecutive k per load and four
// products. Loads run kSteps operands ahead.
template <bool XF16, int RT> struct Down {
  static constexpr int kStep = XF16 ? 32 : 16;  // k per load
  static constexpr int kPer = XF16 ? 8 : 4;     // k per lane and load
  static constexpr int kSteps = 4;
  typedef typename std::conditional<XF16, half8_t, float4_t>::type xvec;
  typedef typename std::conditional<XF16, half8_t, half4_t>::type avec;
  struct Chunk {
    xvec x[kSteps];
    avec a[kSteps][RT];
  };
  const typename std::conditional<XF16, _Float16, float>::type *x;  // this lane's
  const _Float16 *a[RT];

  __device__ __forceinline__ Down(const DownArgs &p, int64_t token, int adapter, int rank0, int lane)
      : x(static_cast<decltype(x)>(p.x) + token * p.k + kPer * (lane >> 4)) {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int j = rank0 + 16 * r + (lane & 15);
      a[r] = p.a + (static_cast<int64_t>(adapter) * p.rank + (j < p.rank ? j : p.rank - 1)) * p.k + kPer * (lane >> 4);
    }
  }
  __device__ __forceinline__ void load(Chunk &c, int s, int64_t k) const {
    c.x[s] = *reinterpret_cast<const xvec *>(x + k);
#pragma unroll
    for (int r = 0; r < RT; ++r) c.a[s][r] = *reinterpret_cast<const avec *>(a[r] + k);
  }
  __device__ __forceinline__ void multiply(const Chunk &c, int s, float4_t acc[RT]) const {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      if constexpr (XF16) {
        acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_f16(c.a[s][r], c.x[s], acc[r], 0, 0, 0);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[r] = __builtin_amdgcn_mfma_f32_16x16x4f32(static_cast<float>(c.a[s][r][i]), c.x[s][i], acc[r], 0, 0, 0);
      }
    }
  }
  __device__ __forceinline__ void load(Chunk &c, int64_t k) const {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) load(c, s, k + s * kStep);
  }
  __device__ __forceinline__ void multiply(const Chunk &c, float4_t acc[RT]) const {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) multiply(c, s, acc);
  }
  __device__ __forceinline__ void operator()(int64_t begin, int64_t end, float4_t acc[RT]) const {
    constexpr int kChunk = kSteps * kStep;
    Chunk c[2];
    int64_t k = begin;
    if (k + kChunk <= end) {
      load(c[0], k);
      for (; k + 3 * kChunk <= end; k += 2 * kChunk) {
        load(c[1], k + kChunk);
        multiply(c[0], acc);
        load(c[0], k + 2 * kChunk);
        multiply(c[1], acc);
      }
      if (k + 2 * kChunk <= end) {
        load(c[1], k + kChunk);
        multiply(c[0], acc);
        multiply(c[1], acc);
        k += 2 * kChunk;
      } else {
        multiply(c[0], acc);
        k += kChunk;
      }
    }
    for (; k < end; k += kStep) {
      load(c[0], 0, k);
      multiply(c[0], 0, acc);
    }
  }
};

// Four ranks j .. j + 3 of a token's V, of which those below `rank` exist.
__device__ __forceinline__ void store_v(float *o, int j, int rank, float4_t v) {
  if (rank % 4 == 0) {
    if (j < rank) *reinterpret_cast<float4_t *>(o + j) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j + e < rank) o[j + e] = v[e];
  }
}

// Tiles by adapter: one workgroup per (token, split, ranks); its wavefronts
// split the k range again and add up through LDS, in order.
template <bool XF16, int RT> __global__ __launch_bounds__(kThreads) void lora_down_group_kernel(DownArgs p) {
  __shared__ int slot[kTok];
  __shared__ float4_t sum[4][RT][64];
  int id;
  if (!group_of(p.ids, static_cast<int>(p.n_tokens), blockIdx.x, slot, id)) return;
  if (id < 0 || id >= p.n_adapters) return;  // no product: the second launch reads no V either
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int mine = slot[lane & 15];
  const int rank0 = blockIdx.z * kRankGroup;
  const Down<XF16, RT> down(p, mine < 0 ? blockIdx.x : mine, __builtin_amdgcn_readfirstlane(id), rank0, lane);
  const int64_t part = p.range / 4;
  const int64_t begin = blockIdx.y * p.range + wave * part;
  const int64_t end = begin + part < p.k ? begin + part : p.k;
  float4_t acc[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = float4_t{};
  down(begin, end, acc);
#pragma unroll
  for (int r = 0; r < RT; ++r) sum[wave][r][lane] = acc[r];
  __syncthreads();
  for (int i = threadIdx.x; i < RT * 64; i += kThreads) {
    const int r = i >> 6, l = i & 63, t = slot[l & 15];
    if (t < 0) continue;
    store_v(p.v + (blockIdx.y * p.n_tokens + t) * p.rank, rank0 + 16 * r + 4 * (l >> 4), p.rank,
            ((sum[0][r][l] + sum[1][r][l]) + sum[2][r][l]) + sum[3][r][l]);
  }
}

// Consecutive tiles: one wavefront per (tile, split, ranks).
template <bool XF16, int RT> __global__ __launch_bounds__(kThreads) void lora_down_kernel(DownArgs p) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (static_cast<int64_t>(blockIdx.x) * 4 + wave) * kTok + (lane & 15);
  const int64_t token = t < p.n_tokens ? t : p.n_tokens - 1;
  const int id = t < p.n_tokens ? p.ids[token] : -1;
  const int rank0 = blockIdx.z * kRankGroup;
  const int64_t begin = blockIdx.y * p.range;
  const int64_t end = begin + p.range < p.k ? begin + p.range : p.k;
  float4_t out[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) out[r] = float4_t{};
  each_adapter(id, p.n_adapters, [&](int a, bool mine) {
    const Down<XF16, RT> down(p, token, a, rank0, lane);
    float4_t acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = float4_t{};
    down(begin, end, acc);
#pragma unroll
    for (int r = 0; r < RT; ++r)
      if (mine) out[r] = acc[r];
  });
  if (t >= p.n_tokens || id < 0 || id >= p.n_adapters) return;
#pragma unroll
  for (int r = 0; r < RT; ++r)
    store_v(p.v + (blockIdx.y * p.n_tokens + t) * p.rank, rank0 + 16 * r + 4 * (lane >> 4), p.rank, out[r]);
}

struct UpArgs {
  const _Float16 *b;
  const float *v, *scales, *base;
  const int32_t *ids;
  float *y;
  int64_t n_tokens, n_rows;
  int n_adapters, rank, splits;
  int steps, chunks;  // steps per wavefront, workgroups per token tile
  bool b_vec, y_vec;      // rows of B, and of base and Y, allow 8- and 16-byte accesses
};

// Four values from p[0..3], of which those before `n` exist; `vec`: all or
// none of them, at once.
template <class V4, class T> __device__ __forceinline__ V4 load4(const T *p, int64_t n, bool vec) {
  V4 v{};
  if (vec) {
    if (n > 0) v = *reinterpret_cast<const V4 *>(p);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) v[i] = p[i];
  }
  return v;
}

// Y^T = B V^T: a lane holds four consecutive rows of token lane % 16; RQ: 16s
// of the rank. The workgroup adds up its tokens' V once; then each wavefront
// goes over its rows in steps of 16 RS, the next step's base and B on their
// way.
template <int RQ, bool GROUP, int RS> __global__ __launch_bounds__(kThreads) void lora_up_kernel(UpArgs p) {
  constexpr int kRow = 16 * RQ + 4;  // floats; padded so that 16 rows start on different banks
  __shared__ __align__(16) float vs[kTok * kRow];
  __shared__ int slot[kTok];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, grp = lane >> 4;
  const int tile = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
  if constexpr (GROUP) {
    int id;
    if (!group_of(p.ids, static_cast<int>(p.n_tokens), tile, slot, id)) return;
  } else {
    if (threadIdx.x < kTok) {
      const int64_t t = static_cast<int64_t>(tile) * kTok + threadIdx.x;
      slot[threadIdx.x] = t < p.n_tokens ? static_cast<int>(t) : -1;
    }
    __syncthreads();
  }
  // V of the tile, scaled: thread (token, four ranks)
  for (int i = threadIdx.x; i < kTok * 4 * RQ; i += kThreads) {
    const int c = i / (4 * RQ), j = 4 * (i % (4 * RQ)), t = slot[c];
    const int id = t < 0 ? -1 : p.ids[t];
    float4_t v{};
    if (id >= 0 && id < p.n_adapters) {
      const float *src = p.v + static_cast<int64_t>(t) * p.rank + j;
      const int64_t step = p.n_tokens * p.rank;
      for (int s = 0; s < p.splits; s += 8) {  // eight loads on their way at once
        float4_t part[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          part[e] = load4<float4_t>(src + (s + e) * step, s + e < p.splits ? p.rank - j : 0, p.rank % 4 == 0);
#pragma unroll
        for (int e = 0; e < 8; ++e) v += part[e];
      }
      v *= p.scales ? p.scales[id] : 1.f;
    }
    *reinterpret_cast<float4_t *>(vs + c * kRow + j) = v;
  }
  __syncthreads();

  const bool live = slot[col] >= 0;
  const int64_t token = live ? slot[col] : slot[0];
  const int id = live ? p.ids[token] : -1;
  const bool valid = id >= 0 && id < p.n_adapters;
  float4_t v[RQ];
#pragma unroll
  for (int q = 0; q < RQ; ++q) v[q] = *reinterpret_cast<const float4_t *>(vs + col * kRow + 16 * q + 4 * grp);

  const uint32_t with = static_cast<uint32_t>(__ballot(valid)) & 0xFFFFu;  // columns with an adapter
  const int first_id = with ? __builtin_amdgcn_readlane(id, __builtin_ctz(with)) : 0;
  const bool one_adapter = __all(!valid || id == first_id);
  // a step: RS tiles of 16 rows, 16 RS consecutive values of each token's row
  struct Step {
    float4_t y[RS];
    half4_t b[RS][RQ];
  };
  const int64_t row_base = (static_cast<int64_t>(chunk) * 4 + wave) * p.steps * (16 * RS);
  auto load_b = [&](Step &t, int64_t row0, int a) {
#pragma unroll
    for (int i = 0; i < RS; ++i) {
      const int64_t r = row0 + 16 * i + col;
      const _Float16 *b = p.b + (a * p.n_rows + (r < p.n_rows ? r : p.n_rows - 1)) * p.rank + 4 * grp;
#pragma unroll
      for (int q = 0; q < RQ; ++q) t.b[i][q] = load4<half4_t>(b + 16 * q, p.rank - 16 * q - 4 * grp, p.b_vec);
    }
  };
  auto load = [&](Step &t, int64_t row0) {
#pragma unroll
    for (int i = 0; i < RS; ++i) {
      const int64_t r4 = row0 + 16 * i + 4 * grp;
      t.y[i] = load4<float4_t>(p.base + token * p.n_rows + r4, p.base && live ? p.n_rows - r4 : 0, p.y_vec);
    }
    if (with && one_adapter) load_b(t, row0, first_id);
  };
  auto add_product = [&](Step &t, bool mine) {
#pragma unroll
    for (int i = 0; i < RS; ++i) {
      float4_t acc{};
#pragma unroll
      for (int q = 0; q < RQ; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc = __builtin_amdgcn_mfma_f32_16x16x4f32(static_cast<float>(t.b[i][q][e]), v[q][e], acc, 0, 0, 0);
      if (mine) t.y[i] += acc;
    }
  };
  auto finish = [&](Step &t, int64_t row0) {
    if (with && one_adapter)
      add_product(t, valid);
    else if (with)
      each_adapter(id, p.n_adapters, [&](int a, bool mine) {
        load_b(t, row0, a);
        add_product(t, mine);
      });
#pragma unroll
    for (int i = 0; i < RS; ++i) {
      if (id != -1 && !valid) {
        const float nan = __builtin_bit_cast(float, 0x7FC00000u);
        t.y[i] = float4_t{nan, nan, nan, nan};
      }
      const int64_t r4 = row0 + 16 * i + 4 * grp, left = live ? p.n_rows - r4 : 0;
      float *o = p.y + token * p.n_rows + r4;
      if (p.y_vec) {
        if (left > 0) *reinterpret_cast<float4_t *>(o) = t.y[i];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < left) o[e] = t.y[i][e];
      }
    }
  };
  const int64_t row_end = row_base + p.steps * (16 * RS) < p.n_rows ? row_base + p.steps * (16 * RS) : p.n_rows;
  if (row_base >= row_end) return;
  Step t[2];
  int64_t row = row_base;
  load(t[0], row);
  for (; row + 32 * RS < row_end; row += 32 * RS) {
    load(t[1], row + 16 * RS);
    finish(t[0], row);
    load(t[0], row + 32 * RS);
    finish(t[1], row + 16 * RS);
  }
  if (row + 16 * RS < row_end) {
    load(t[1], row + 16 * RS);
    finish(t[0], row);
    finish(t[1], row + 16 * RS);
  } else {
    finish(t[0], row);
  }
}

bool by_adapter(int64_t n_tokens) { return n_tokens <= kGroupTokens; }
// k per split: a multiple of 128 (4 wavefronts of 32) by adapter, of 32 else.
int64_t split_range(int64_t n_tokens, int64_t k) {
  if (by_adapter(n_tokens)) return std::max<int64_t>(4 * kGroupSlab, (k + 128 * kMaxSplits - 1) / (128 * kMaxSplits) * 128);
  const int64_t waves = (n_tokens + kTok - 1) / kTok;
  const int64_t want = std::min(std::max<int64_t>(1, kTileWaves / waves), std::max<int64_t>(1, k / 256));
  return (k + 32 * want - 1) / (32 * want) * 32;
}

}  // namespace

int lora_splits(int64_t n_tokens, int64_t k, int64_t) {
  const int64_t range = split_range(n_tokens, k);
  return static_cast<int>((k + range - 1) / range);
}

hipError_t launch_lora(const void *X, bool x_f16, int64_t n_tokens, int64_t k, const void *A, const void *B,
                       int64_t n_adapters, int64_t rank, int64_t n_rows, const float *scales, const int32_t *ids,
                       const float *base, float *Y, float *partial, hipStream_t stream) {
  const bool group = by_adapter(n_tokens);
  const int splits = lora_splits(n_tokens, k, rank);
  const int64_t tiles = group ? n_tokens : (n_tokens + kTok - 1) / kTok;
  const DownArgs d{X, static_cast<const _Float16 *>(A), ids, partial, n_tokens, k, split_range(n_tokens, k),
                   static_cast<int>(n_adapters), static_cast<int>(rank)};
  const dim3 grid(static_cast<unsigned>(group ? tiles : (tiles + 3) / 4), splits,
                  static_cast<unsigned>((rank + kRankGroup - 1) / kRankGroup));
  auto down = [&](auto xf16, auto rt) {
    constexpr bool X16 = decltype(xf16)::value;
    constexpr int RT = decltype(rt)::value;
    return launch(group ? lora_down_group_kernel<X16, RT> : lora_down_kernel<X16, RT>, grid, dim3(kThreads), 0, stream,
                  d);
  };
  auto by_rank = [&](auto xf16) {
    if (rank <= 16) return down(xf16, std::integral_constant<int, 1>{});
    if (rank <= 32) return down(xf16, std::integral_constant<int, 2>{});
    return down(xf16, std::integral_constant<int, 4>{});
  };
  const hipError_t e = x_f16 ? by_rank(std::true_type{}) : by_rank(std::false_type{});
  if (e != hipSuccess) return e;

  // Steps of 64 rows per wavefront (256 bytes of a token's row), of 16 where
  // there are few; several steps where there are workgroups enough, since
  // each workgroup first adds up its tokens' V.
  const int64_t rs = rank > 64 || n_rows * tiles < 4096 * 64 ? 1 : 4;
  const int64_t all = (n_rows + 64 * rs - 1) / (64 * rs);  // steps of a workgroup's four wavefronts
  const int64_t steps = std::max({int64_t{1}, std::min<int64_t>(16 / rs, all * tiles / 1024), (all * tiles) >> 23});
  const int64_t chunks = (all + steps - 1) / steps;
  const UpArgs u{static_cast<const _Float16 *>(B), partial, scales, base, ids, Y, n_tokens, n_rows,
                 static_cast<int>(n_adapters), static_cast<int>(rank), splits, static_cast<int>(steps),
                 static_cast<int>(chunks), rank % 4 == 0 && reinterpret_cast<uintptr_t>(B) % 8 == 0,
                 n_rows % 4 == 0 && reinterpret_cast<uintptr_t>(Y) % 16 == 0 && reinterpret_cast<uintptr_t>(base) % 16 == 0};
  const dim3 ugrid(static_cast<unsigned>(chunks * tiles));
  auto up = [&](auto rq, auto r) {
    constexpr int RQ = decltype(rq)::value, RS = decltype(r)::value;
    return launch(group ? lora_up_kernel<RQ, true, RS> : lora_up_kernel<RQ, false, RS>, ugrid, dim3(kThreads), 0,
                  stream, u);
  };
  auto by_rows = [&](auto rq) {
    return rs == 4 ? up(rq, std::integral_constant<int, 4>{}) : up(rq, std::integral_constant<int, 1>{});
  };
  if (rank <= 16) return by_rows(std::integral_constant<int, 1>{});
  if (rank <= 32) return by_rows(std::integral_constant<int, 2>{});
  if (rank <= 64) return by_rows(std::integral_constant<int, 4>{});
  return up(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
}

}  // namespace qmm
