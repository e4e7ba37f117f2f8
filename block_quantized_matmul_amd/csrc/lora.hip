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
//  * more tokens (prompts: the tokens of a request stand together), 64
//    consecutive tokens, so that an operand of A or B serves four products. A
//    tile that does hold several adapters deals them to two workgroups, which
//    take theirs one after another and keep, in each token's column, its own
//    adapter's result.
// Columns do not mix, so a non-finite value of another token or adapter stays
// out in both.
//
// The first launch splits k and leaves partial sums of V in the workspace,
// which the second adds in order (no atomics; for consecutive tiles a launch
// between them does).
//
// Measured: 1 token, 4096 x 4096, rank 16, fp32 X 7 us for both launches in a
// graph (latency); 64 tokens on 32 adapters, 4096 to 11008 rows, 15 us (22 MB,
// of which 15 are the adapters: 4.5 us at a copy's rate; the rest is the two
// launches' latencies: ids, then operands, then the sum); 2048 fp16 tokens of
// 9 requests, 11008 to 4096 rows, rank 64, 61 us: down 25 (45 MB, 1.8 TB/s),
// sum 5, up 32 (67 MB, 2.1 TB/s; its fp32 products alone are 7); 8192 fp32
// tokens, 4096 x 4096, rank 32, 119 us (402 MB, 3.4 TB/s).
#include "attn.h"
#include "common.h"
#include "launch.h"

#include <algorithm>

namespace qmm {

namespace {

constexpr int kThreads = 256;
constexpr int kTok = 16;            // tokens per product
constexpr int kSub = 4;             // products' tokens per consecutive tile
// Largest batch in tiles by adapter. The host does not know the ids, so this
// weighs decode batches of many adapters against prompts. 4096 x 4096, rank 16,
// us by adapter / in consecutive tiles: 200 tokens on 32 adapters at random 17 /
// 39, on 8 17 / 18, in 9 runs 17 / 14, on one 20 / 12; 512 tokens 29 / 48, 28 /
// 22, 29 / 14, 53 / 14; 1000 tokens 49 / 84, 48 / 35, 51 / 19, 89 / 17. What is
// left is a step up for batches of many adapters at random: 512 tokens on 32
// 29 us, 513 59.
constexpr int kGroupTokens = 512;
// Ranges of k, tiles by adapter: bounds the workspace, for k beyond 131072 only.
// 1 token of 262144 to 1024 rows 22 us, 14 with 64 ranges, 38 with 1024; of
// 1048576 26, 27, 72.
constexpr int kMaxSplits = 256;
// Workgroups among which a consecutive tile's adapters are dealt: most tiles
// have one adapter, and those where requests meet two. 2048 tokens of 9
// requests 61 us, with one workgroup for all of a tile's adapters 66, with four
// 67 (the workgroups that leave at once cost more than they save).
constexpr int kShares = 2;
constexpr int kRankGroup = 64;      // ranks per workgroup of the first launch
// Workgroups the first launch aims at, consecutive tiles: 2048 tokens, 11008 to
// 4096 rows, rank 64 63 us, 64 with 256, 72 with 1024; 8192 tokens, 4096 x 4096,
// rank 32 119, 124, 117.
constexpr int kTileGroups = 512;

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

// The adapters of a tile's tokens, one after another: f(a), the lanes whose
// token t (of TT, in column lane % 16) has adapter a being those with
// id[t] == a. Ids outside [0, n_adapters) are left out.
template <int TT, class F> __device__ __forceinline__ void each_adapter(const int id[TT], int n_adapters, F f) {
  uint32_t left[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t)
    left[t] = static_cast<uint32_t>(__ballot(id[t] >= 0 && id[t] < n_adapters)) & 0xFFFFu;
  for (;;) {
    int a = -1;
#pragma unroll
    for (int t = 0; t < TT; ++t)
      if (a < 0 && left[t] != 0) a = __builtin_amdgcn_readlane(id[t], __builtin_ctz(left[t]));
    if (a < 0) return;
#pragma unroll
    for (int t = 0; t < TT; ++t) left[t] &= ~static_cast<uint32_t>(__ballot(id[t] == a));
    f(a);
  }
}
// Consecutive tiles: the tokens (as bits) whose adapters fall to this share of
// a tile's workgroups, the tile's adapters being dealt to its kShares shares
// in the order of their first tokens. Lane l of the wavefront has token l's id.
__device__ __forceinline__ uint64_t share_of(int id, int n_adapters, int share) {
  static_assert(kTok * kSub == 64, "a lane per token");
  uint64_t left = __ballot(id >= 0 && id < n_adapters), mine = 0;
  for (int j = 0; left != 0; j = (j + 1) % kShares) {
    const uint64_t with = __ballot(id == __builtin_amdgcn_readlane(id, __builtin_ctzll(left)));
    if (j == share) mine |= with;
    left &= ~with;
  }
  return mine;
}
// Consecutive tiles: workgroup b's share, tile and part of the tile's work, of
// `parts` (padded). The parts are the fastest index, so that one XCD
// (workgroups go round them) gets the same parts of all tiles: its L2 then
// holds those of the adapters, and the XCDs have equal work. The last share
// comes first: where a tile has one adapter, its workgroups leave at once.
__device__ __forceinline__ void tile_of(int b, int parts, int tiles, int &share, int &tile, int &part) {
  part = b % parts;
  tile = b / parts % tiles;
  share = kShares - 1 - b / parts / tiles;
}

struct DownArgs {
  const void *x;
  const _Float16 *a;
  const int32_t *ids;
  float *v;  // [splits][n_tokens][rank]
  int64_t n_tokens, k, range;  // range: k per split
  int n_adapters, rank, splits;
  int parts;  // consecutive tiles: splits, padded
};

// V^T = A X^T on one wavefront: 16 RT ranks of one adapter, TT tokens in each
// of the lanes' columns, k from begin to end (multiples of 32). The C layout
// gives a lane four consecutive ranks of token lane % 16. Operand element j of lane
// group g = lane / 16 is the same k for both operands; which k it is does not
// matter to the sum, so an fp32 lane takes 4 consecutive k per load and four
// products. Loads run kSteps operands ahead.
template <bool XF16, int RT, int TT> struct Down {
  static constexpr int kStep = XF16 ? 32 : 16;  // k per load
  static constexpr int kPer = XF16 ? 8 : 4;     // k per lane and load
  static constexpr int kSteps = TT > 1 ? 2 : 4;
  typedef typename std::conditional<XF16, half8_t, float4_t>::type xvec;
  typedef typename std::conditional<XF16, half8_t, half4_t>::type avec;
  struct Chunk {
    xvec x[kSteps][TT];
    avec a[kSteps][RT];
  };
  typedef typename std::conditional<XF16, _Float16, float>::type xone;
  const xone *x[TT];  // this lane's
  const _Float16 *a[RT];

  __device__ __forceinline__ Down(const DownArgs &p, const int64_t token[TT], int adapter, int rank0, int lane) {
#pragma unroll
    for (int t = 0; t < TT; ++t)
      x[t] = static_cast<const xone *>(p.x) + token[t] * p.k + kPer * (lane >> 4);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int j = rank0 + 16 * r + (lane & 15);
      a[r] = p.a + (static_cast<int64_t>(adapter) * p.rank + (j < p.rank ? j : p.rank - 1)) * p.k + kPer * (lane >> 4);
    }
  }
  __device__ __forceinline__ void load(Chunk &c, int s, int64_t k) const {
#pragma unroll
    for (int t = 0; t < TT; ++t) c.x[s][t] = *reinterpret_cast<const xvec *>(x[t] + k);
#pragma unroll
    for (int r = 0; r < RT; ++r) c.a[s][r] = *reinterpret_cast<const avec *>(a[r] + k);
  }
  __device__ __forceinline__ void multiply(const Chunk &c, int s, float4_t (&acc)[RT][TT]) const {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        if constexpr (XF16) {
          acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(c.a[s][r], c.x[s][t], acc[r][t], 0, 0, 0);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(static_cast<float>(c.a[s][r][i]), c.x[s][t][i],
                                                             acc[r][t], 0, 0, 0);
        }
      }
  }
  __device__ __forceinline__ void load(Chunk &c, int64_t k) const {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) load(c, s, k + s * kStep);
    __builtin_amdgcn_sched_barrier(0);  // the loads go out before the products of the other buffer
  }
  __device__ __forceinline__ void multiply(const Chunk &c, float4_t (&acc)[RT][TT]) const {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) multiply(c, s, acc);
    __builtin_amdgcn_sched_barrier(0);
  }
  __device__ __forceinline__ void operator()(int64_t begin, int64_t end, float4_t (&acc)[RT][TT]) const {
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

// One workgroup per (tile, split, ranks); its wavefronts split the k range
// again and add up through LDS, in order.
template <bool XF16, int RT, bool GROUP>
__global__ __launch_bounds__(kThreads, GROUP || RT < 4 ? 2 : 1) void lora_down_kernel(DownArgs p) {
  constexpr int TT = GROUP ? 1 : kSub;
  __shared__ float4_t sum[4][RT][TT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rank0 = blockIdx.y * kRankGroup;
  __shared__ int slot[kTok * TT];
  int split;
  int id[TT];
  int64_t token[TT];
  if constexpr (GROUP) {
    split = blockIdx.x / static_cast<int>(p.n_tokens);
    const int t = blockIdx.x % static_cast<int>(p.n_tokens);
    if (!group_of(p.ids, static_cast<int>(p.n_tokens), t, slot, id[0])) return;
    if (id[0] < 0 || id[0] >= p.n_adapters) return;  // no product: the second launch reads no V either
    token[0] = slot[lane & 15] < 0 ? t : slot[lane & 15];
  } else {
    const int tiles = static_cast<int>((p.n_tokens + kTok * TT - 1) / (kTok * TT));
    int tile, share;
    tile_of(blockIdx.x, p.parts, tiles, share, tile, split);
    if (split >= p.splits) return;
    const int64_t t0 = static_cast<int64_t>(tile) * (kTok * TT);
    const int own = t0 + lane < p.n_tokens ? p.ids[t0 + lane] : -1;
    const uint64_t mine = share_of(own, p.n_adapters, share);
    if (mine == 0) return;
    if (wave == 0) slot[lane] = mine >> lane & 1 ? static_cast<int>(t0) + lane : -1;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int at = kTok * t + (lane & 15);
      const int a = __shfl(own, at);
      id[t] = mine >> at & 1 ? a : -1;
      token[t] = t0 + (mine >> at & 1 ? at : __builtin_ctzll(mine));
    }
  }
  const int64_t part = p.range / 4;
  const int64_t begin = split * p.range + wave * part;
  const int64_t end = begin + part < p.k ? begin + part : p.k;
  each_adapter<TT>(id, p.n_adapters, [&](int a) {
    const Down<XF16, RT, TT> down(p, token, a, rank0, lane);
    float4_t acc[RT][TT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[r][t] = float4_t{};
    down(begin, end, acc);
#pragma unroll
    for (int t = 0; t < TT; ++t)
      if (id[t] == a) {
#pragma unroll
        for (int r = 0; r < RT; ++r) sum[wave][r][t][lane] = acc[r][t];
      }
  });
  __syncthreads();
  for (int i = threadIdx.x; i < RT * TT * 64; i += kThreads) {
    const int r = i / (TT * 64), t = i / 64 % TT, l = i & 63, tok = slot[kTok * t + (l & 15)];
    if (tok < 0) continue;
    store_v(p.v + (split * p.n_tokens + tok) * p.rank, rank0 + 16 * r + 4 * (l >> 4), p.rank,
            ((sum[0][r][t][l] + sum[1][r][t][l]) + sum[2][r][t][l]) + sum[3][r][t][l]);
  }
}

struct UpArgs {
  const _Float16 *b;
  const float *v, *scales, *base;
  const int32_t *ids;
  float *y;
  int64_t n_tokens, n_rows;
  int n_adapters, rank, splits;
  int steps, chunks;  // steps per wavefront, workgroups per token tile
  int parts;          // consecutive tiles: chunks, padded
};

// Four values from p[at .. at + 3] of n. VEC: n and at are multiples of 4 and
// p allows one access; past the end the last four are read instead, without a
// branch, so that many loads can be on their way. Otherwise those that exist,
// and zeros.
template <class V4, bool VEC, class T> __device__ __forceinline__ V4 load4(const T *p, int64_t at, int64_t n) {
  if constexpr (VEC) return *reinterpret_cast<const V4 *>(p + (at < n ? at : n - 4));
  V4 v{};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (at + i < n) v[i] = p[at + i];
  return v;
}

// Adds up the partial sums of V, in order, into those of the first split:
// before the second launch on consecutive tiles, whose workgroups on one tile
// would each read all of them again.
__global__ __launch_bounds__(kThreads) void lora_sum_kernel(float *v, int64_t n, int splits) {
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n; i += stride) {
    float sum = 0.f;
    for (int s = 0; s < splits; s += 8) {
      float part[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) part[e] = s + e < splits ? v[(s + e) * n + i] : 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += part[e];
    }
    v[i] = sum;
  }
}

// Y^T = B V^T: a lane holds four consecutive rows of its tokens (columns
// lane % 16). RQ: 16s of the rank; RS: 16s of the rows of a step, which are
// consecutive in each token's row. The workgroup adds up its tokens' V once;
// then each wavefront goes over its rows, the next step's base and B on their
// way. VEC: the rows of B and V allow 8- and 16-byte accesses, those of base
// and Y 16-byte ones.
template <int RQ, bool GROUP, int RS, bool VEC>
__global__ __launch_bounds__(kThreads, RQ <= 4 ? 2 : 1) void lora_up_kernel(UpArgs p) {
  constexpr int TT = GROUP ? 1 : kSub;
  constexpr int kRow = 16 * RQ + 4;  // floats; padded so that 16 rows start on different banks
  __shared__ __align__(16) float vs[kTok * TT * kRow];
  __shared__ int slot[kTok * TT], adapter[kTok * TT];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, grp = lane >> 4;
  int chunk;
  int any;  // one of the tile's tokens
  if constexpr (GROUP) {
    chunk = blockIdx.x % p.chunks;
    any = blockIdx.x / p.chunks;
    int id;
    if (!group_of(p.ids, static_cast<int>(p.n_tokens), any, slot, id)) return;
    if (threadIdx.x < kTok) adapter[threadIdx.x] = slot[threadIdx.x] >= 0 ? id : -1;
  } else {
    const int tiles = static_cast<int>((p.n_tokens + kTok * TT - 1) / (kTok * TT));
    int tile, share;
    tile_of(blockIdx.x, p.parts, tiles, share, tile, chunk);
    if (chunk >= p.chunks) return;
    const int64_t t = static_cast<int64_t>(tile) * (kTok * TT) + lane;
    const int own = t < p.n_tokens ? p.ids[t] : -1;
    uint64_t mine = share_of(own, p.n_adapters, share);
    // tokens without a product go with the first share
    if (share == 0) mine |= __ballot(t < p.n_tokens && (own < 0 || own >= p.n_adapters));
    if (mine == 0) return;
    if (wave == 0) {
      slot[lane] = mine >> lane & 1 ? static_cast<int>(t) : -1;
      adapter[lane] = mine >> lane & 1 ? own : -1;
    }
    any = static_cast<int>(t) - lane + __builtin_ctzll(mine);
  }
  __syncthreads();
  int id[TT];
  bool live[TT], valid[TT];
  const float *base[TT];  // the lanes' token rows
  float *out[TT];
  int first_id = -1;  // the first valid id, -1 if there is none
  bool one_adapter = true;
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int s = slot[kTok * t + col];
    live[t] = s >= 0;
    const int64_t token = live[t] ? s : any;
    id[t] = adapter[kTok * t + col];
    valid[t] = id[t] >= 0 && id[t] < p.n_adapters;
    base[t] = p.base ? p.base + token * p.n_rows : nullptr;
    out[t] = p.y + token * p.n_rows;
    const uint32_t with = static_cast<uint32_t>(__ballot(valid[t])) & 0xFFFFu;
    if (first_id < 0 && with) first_id = __builtin_amdgcn_readlane(id[t], __builtin_ctz(with));
    one_adapter = one_adapter && __all(!valid[t] || id[t] == first_id);
  }
  struct Step {
    float4_t y[RS][TT];
    half4_t b[RS][RQ];
  };
  auto load_b = [&](Step &s, int64_t row0, int a) {
#pragma unroll
    for (int i = 0; i < RS; ++i) {
      const int64_t r = row0 + 16 * i + col;
      const _Float16 *b = p.b + (a * p.n_rows + (r < p.n_rows ? r : p.n_rows - 1)) * p.rank;
#pragma unroll
      for (int q = 0; q < RQ; ++q) s.b[i][q] = load4<half4_t, VEC>(b, 16 * q + 4 * grp, p.rank);
    }
  };
  auto load = [&](Step &s, int64_t row0) {
    if (p.base) {
#pragma unroll
      for (int i = 0; i < RS; ++i)
#pragma unroll
        for (int t = 0; t < TT; ++t) s.y[i][t] = load4<float4_t, VEC>(base[t], row0 + 16 * i + 4 * grp, p.n_rows);
    } else {
#pragma unroll
      for (int i = 0; i < RS; ++i)
#pragma unroll
        for (int t = 0; t < TT; ++t) s.y[i][t] = float4_t{};
    }
    if (first_id >= 0 && one_adapter) load_b(s, row0, first_id);
    __builtin_amdgcn_sched_barrier(0);
  };
  const int64_t row_base = (static_cast<int64_t>(chunk) * 4 + wave) * p.steps * (16 * RS);
  const int64_t row_end = row_base + p.steps * (16 * RS) < p.n_rows ? row_base + p.steps * (16 * RS) : p.n_rows;
  Step s[2];
  int64_t row = row_base;
  if (row < row_end) load(s[0], row);

  // V of the tile, scaled: thread (token, four ranks), all loads on their way
  // at once (what the workspace holds for a token without an adapter is read
  // too, and dropped)
  constexpr int kItems = kTok * TT * 4 * RQ, kEach = (kItems + kThreads - 1) / kThreads;
  constexpr int kParts = GROUP ? 8 : 1;  // partial sums per round
  float4_t sum[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) sum[e] = float4_t{};
  const int64_t v_step = p.n_tokens * p.rank;
  for (int part = 0; part < p.splits; part += kParts) {
    float4_t add[kEach][kParts];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = threadIdx.x + e * kThreads < kItems ? threadIdx.x + e * kThreads : 0;
      const int t = slot[i / (4 * RQ)] < 0 ? any : slot[i / (4 * RQ)];
#pragma unroll
      for (int u = 0; u < kParts; ++u)
        add[e][u] = load4<float4_t, VEC>(
            p.v + (part + u < p.splits ? part + u : p.splits - 1) * v_step + static_cast<int64_t>(t) * p.rank,
            4 * (i % (4 * RQ)), p.rank);
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e)
#pragma unroll
      for (int u = 0; u < kParts; ++u) sum[e] += part + u < p.splits ? add[e][u] : float4_t{};
  }
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = threadIdx.x + e * kThreads, c = i / (4 * RQ), j = 4 * (i % (4 * RQ));
    if (i < kItems) {
      const int a = adapter[c];
      const bool with = a >= 0 && a < p.n_adapters && j < p.rank;
      const float scale = with && p.scales ? p.scales[a] : 1.f;
      *reinterpret_cast<float4_t *>(vs + c * kRow + j) = with ? sum[e] * scale : float4_t{};
    }
  }
  __syncthreads();
  if (row >= row_end) return;
  constexpr bool kHold = RQ <= 4;  // V's operands fit the registers
  float4_t held[kHold ? TT : 1][kHold ? RQ : 1];
  if constexpr (kHold) {
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int q = 0; q < RQ; ++q)
        held[t][q] = *reinterpret_cast<const float4_t *>(vs + (kTok * t + col) * kRow + 16 * q + 4 * grp);
  }
  auto add_product = [&](Step &s, int a) {
#pragma unroll
    for (int i = 0; i < RS; ++i)
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        float4_t acc{};
#pragma unroll
        for (int q = 0; q < RQ; ++q) {
          float4_t v;
          if constexpr (kHold)
            v = held[t][q];
          else
            v = *reinterpret_cast<const float4_t *>(vs + (kTok * t + col) * kRow + 16 * q + 4 * grp);
          // ranks past the last meet a zero of V, and are made zeros here too (a repeated value may be infinite)
          const half4_t w = 16 * q + 4 * grp < p.rank ? s.b[i][q] : half4_t{};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(static_cast<float>(w[e]), v[e], acc, 0, 0, 0);
        }
        if (id[t] == a) s.y[i][t] += acc;
      }
  };
  auto finish = [&](Step &s, int64_t row0) {
    if (first_id >= 0 && one_adapter)
      add_product(s, first_id);
    else if (first_id >= 0)
      each_adapter<TT>(id, p.n_adapters, [&](int a) {
        load_b(s, row0, a);
        add_product(s, a);
      });
#pragma unroll
    for (int i = 0; i < RS; ++i)
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        if (id[t] != -1 && !valid[t]) {
          const float nan = __builtin_bit_cast(float, 0x7FC00000u);
          s.y[i][t] = float4_t{nan, nan, nan, nan};
        }
        const int64_t r4 = row0 + 16 * i + 4 * grp;
        if constexpr (VEC) {
          if (live[t] && r4 < p.n_rows) *reinterpret_cast<float4_t *>(out[t] + r4) = s.y[i][t];
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (live[t] && r4 + e < p.n_rows) out[t][r4 + e] = s.y[i][t][e];
        }
      }
  };
  for (; row + 32 * RS < row_end; row += 32 * RS) {
    load(s[1], row + 16 * RS);
    finish(s[0], row);
    load(s[0], row + 32 * RS);
    finish(s[1], row + 16 * RS);
  }
  if (row + 16 * RS < row_end) {
    load(s[1], row + 16 * RS);
    finish(s[0], row);
    finish(s[1], row + 16 * RS);
  } else {
    finish(s[0], row);
  }
}

// Workgroups per tile, such that those of a part fall to one XCD of eight, or
// to as few as they can.
int64_t padded(int64_t parts) {
  if (parts >= 8) return (parts + 7) / 8 * 8;
  return parts > 4 ? 8 : parts > 2 ? 4 : parts;
}
bool by_adapter(int64_t n_tokens) { return n_tokens <= kGroupTokens; }
// k per split: a multiple of 128, 32 for each of a workgroup's wavefronts. By
// adapter, each split is a partial sum that the second launch's workgroups
// read, a round of eight at a time: two rounds of loads of 64 k per wavefront,
// or one where ranks are many and k short. 8 tokens, 4096 to 11008 rows, rank
// 16 8.9 us with 512 k per split, 9.7 with 256, 9.9 with 1024; 1 token, the
// same with rank 64 11.1, 9.6, 14.7; 8 tokens, 11008 to 4096, rank 64 15.4,
// 16.6, 18.4. (The header's qmm_lora_workspace_max_bytes follows from these.)
int64_t split_range(int64_t n_tokens, int64_t k, int64_t rank) {
  const int64_t tiles = (n_tokens + kTok * kSub - 1) / (kTok * kSub);
  int64_t want;
  if (by_adapter(n_tokens))
    want = std::min<int64_t>(kMaxSplits, rank > 32 ? std::max(k / 512, std::min<int64_t>(k / 256, 16)) : k / 512);
  else
    want = std::min(kTileGroups / tiles, k / 256);
  want = std::max<int64_t>(want, 1);
  return (k + 128 * want - 1) / (128 * want) * 128;
}

}  // namespace

int lora_splits(int64_t n_tokens, int64_t k, int64_t rank) {
  const int64_t range = split_range(n_tokens, k, rank);
  return static_cast<int>((k + range - 1) / range);
}

hipError_t launch_lora(const void *X, bool x_f16, int64_t n_tokens, int64_t k, const void *A, const void *B,
                       int64_t n_adapters, int64_t rank, int64_t n_rows, const float *scales, const int32_t *ids,
                       const float *base, float *Y, float *partial, hipStream_t stream) {
  const bool group = by_adapter(n_tokens);
  const int splits = lora_splits(n_tokens, k, rank);
  // workgroups per split or chunk: every token's (most leave at once), or every tile's
  const int64_t groups = group ? n_tokens : (n_tokens + kTok * kSub - 1) / (kTok * kSub);
  const int64_t parts = padded(splits);
  const DownArgs d{X, static_cast<const _Float16 *>(A), ids, partial, n_tokens, k, split_range(n_tokens, k, rank),
                   static_cast<int>(n_adapters), static_cast<int>(rank), splits, static_cast<int>(parts)};
  const dim3 grid(static_cast<unsigned>(group ? groups * splits : groups * parts * kShares),
                  static_cast<unsigned>((rank + kRankGroup - 1) / kRankGroup));
  auto down = [&](auto xf16, auto rt) {
    constexpr bool X16 = decltype(xf16)::value;
    constexpr int RT = decltype(rt)::value;
    return launch(group ? lora_down_kernel<X16, RT, true> : lora_down_kernel<X16, RT, false>, grid, dim3(kThreads), 0,
                  stream, d);
  };
  auto by_rank = [&](auto xf16) {
    if (rank <= 16) return down(xf16, std::integral_constant<int, 1>{});
    if (rank <= 32) return down(xf16, std::integral_constant<int, 2>{});
    return down(xf16, std::integral_constant<int, 4>{});
  };
  const hipError_t e = x_f16 ? by_rank(std::true_type{}) : by_rank(std::false_type{});
  if (e != hipSuccess) return e;

  if (!group && splits > 1) {
    const int64_t n = n_tokens * rank;
    const int64_t blocks = std::min<int64_t>((n + kThreads - 1) / kThreads, 4096);
    const hipError_t f =
        launch(lora_sum_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, partial, n, splits);
    if (f != hipSuccess) return f;
  }

  // Steps of 64 rows by adapter (256 bytes of a token's row), of 16 where
  // there are few or for consecutive tiles, whose step has 64 tokens (rank 16,
  // us in steps of 64 / 16: 64 tokens to 11008 rows 15.6 / 17.4, 256 to 4096
  // 24.6 / 26.5, up to 16 tokens the same; rank 64: 64 to 11008 46.5 / 40.6, 8 to
  // 11008 16.2 / 14.8); several
  // steps where there are workgroups enough, since each workgroup first adds
  // up its tokens' V. On consecutive tiles V is little for ranks up to 32, and
  // more workgroups balance better: 2048 tokens, 11008 rows, rank 16 72 us with
  // 2048 wanted, 64 with 4096; 4096 rows, rank 64 60 with 2048, 53 with 1024.
  const bool vec = rank % 4 == 0 && reinterpret_cast<uintptr_t>(B) % 8 == 0 && n_rows % 4 == 0 &&
                   reinterpret_cast<uintptr_t>(Y) % 16 == 0 && reinterpret_cast<uintptr_t>(base) % 16 == 0;
  const int64_t rs = !group || !vec || rank > 64 || n_rows * groups < 4096 * 64 ? 1 : 4;
  const int64_t all = (n_rows + 64 * rs - 1) / (64 * rs);  // steps of a workgroup's four wavefronts
  const int64_t want = group || rank > 32 ? 1024 : 4096;
  const int64_t steps = std::max({int64_t{1}, std::min<int64_t>(16 / rs, all * groups / want), (all * groups) >> 22});
  const int64_t chunks = (all + steps - 1) / steps;
  const UpArgs u{static_cast<const _Float16 *>(B), partial, scales, base, ids, Y, n_tokens, n_rows,
                 static_cast<int>(n_adapters), static_cast<int>(rank), group ? splits : 1, static_cast<int>(steps),
                 static_cast<int>(chunks), static_cast<int>(padded(chunks))};
  const dim3 ugrid(static_cast<unsigned>(group ? groups * chunks : groups * padded(chunks) * kShares));
  auto up = [&](auto rq) {
    constexpr int RQ = decltype(rq)::value;
    constexpr int RS = RQ <= 4 ? 4 : 1;
    if (rs > 1) return launch(lora_up_kernel<RQ, true, RS, true>, ugrid, dim3(kThreads), 0, stream, u);
    if (vec)
      return launch(group ? lora_up_kernel<RQ, true, 1, true> : lora_up_kernel<RQ, false, 1, true>, ugrid,
                    dim3(kThreads), 0, stream, u);
    return launch(group ? lora_up_kernel<RQ, true, 1, false> : lora_up_kernel<RQ, false, 1, false>, ugrid,
                  dim3(kThreads), 0, stream, u);
  };
  if (rank <= 16) return up(std::integral_constant<int, 1>{});
  if (rank <= 32) return up(std::integral_constant<int, 2>{});
  if (rank <= 64) return up(std::integral_constant<int, 4>{});
  return up(std::integral_constant<int, 16>{});
}

}  // namespace qmm
