// Low-rank adapters of many requests beside a shared projection (qmm_lora).
//
//   V[t] = A_a X[t]        (rank values, a = ids[t])
//   Y[t] = base[t] + s_a B_a V[t]
//
// Two launches on the matrix cores, both over tiles of 16 tokens. Both are
// bound by memory: X, base and Y pass once, and the adapters' own bytes are
// small. A tile whose tokens use several adapters takes them one after
// another and keeps, in each token's column, the result of the token's own
// (columns do not mix, so neither does a non-finite value of another
// adapter). Tokens of one request stand together in a batch, so a prompt's
// tiles have one adapter, and a decode batch has few tiles.
//
// The first launch splits k over its wavefronts and, where tiles are few, over
// workgroups: each range leaves its partial V in the workspace, and the
// second adds them in order (no atomics). An fp16 X is multiplied as it is;
// an fp32 X, and V in the second launch, run on the fp32 matrix instruction
// with A and B widened, so nothing is rounded to fewer than 32 bits.
#include "attn.h"
#include "common.h"
#include "launch.h"

#include <algorithm>

namespace qmm {

namespace {

constexpr int kThreads = 256;
constexpr int kTok = 16;        // tokens per tile
constexpr int kSlab = 256;      // k per wavefront and round, many tiles
constexpr int kSlabFew = 64;    // the same, few tiles
constexpr int kRankGroup = 64;  // ranks per workgroup of the first launch

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
  int64_t n_tokens, k;
  int n_adapters, rank, splits, rounds;  // rounds: slabs per wavefront
};

// V^T = A X^T: the C layout gives a lane four consecutive ranks of token
// lane % 16. Operand element j of lane group g = lane / 16 is the same k for
// both operands; which k it is does not matter to the sum, so an fp32 lane
// takes 4 consecutive k per load and four steps.
template <bool XF16, int RT, int SLAB>
__global__ __launch_bounds__(kThreads) void lora_down_kernel(DownArgs p) {
  constexpr int kStep = XF16 ? 32 : 16;  // k per load
  constexpr int kSteps = SLAB / kStep;
  typedef typename std::conditional<XF16, half8_t, float4_t>::type xvec;
  typedef typename std::conditional<XF16, half8_t, half4_t>::type avec;
  constexpr int kPer = XF16 ? 8 : 4;  // k per lane and load
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * kTok;
  const int split = blockIdx.y, rank0 = blockIdx.z * kRankGroup;
  const int col = lane & 15, grp = lane >> 4;
  const int64_t token = tok0 + col < p.n_tokens ? tok0 + col : p.n_tokens - 1;
  const int id = tok0 + col < p.n_tokens ? p.ids[token] : -1;
  const int64_t begin = (static_cast<int64_t>(split) * 4 + wave) * p.rounds * SLAB;
  const int64_t end = begin + static_cast<int64_t>(p.rounds) * SLAB < p.k ? begin + static_cast<int64_t>(p.rounds) * SLAB : p.k;

  float4_t out[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) out[r] = float4_t{};
  each_adapter(id, p.n_adapters, [&](int a, bool mine) {
    float4_t acc[RT];
    const _Float16 *arow[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      acc[r] = float4_t{};
      const int j = rank0 + 16 * r + col;
      arow[r] = p.a + (static_cast<int64_t>(a) * p.rank + (j < p.rank ? j : p.rank - 1)) * p.k + kPer * grp;
    }
    const int64_t x0 = token * p.k + kPer * grp;
    auto slab = [&](int64_t k0, auto full) {
      xvec x[kSteps];
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        if (full || k0 + s * kStep < end) {
          if constexpr (XF16)
            x[s] = *reinterpret_cast<const half8_t *>(static_cast<const _Float16 *>(p.x) + x0 + k0 + s * kStep);
          else
            x[s] = *reinterpret_cast<const float4_t *>(static_cast<const float *>(p.x) + x0 + k0 + s * kStep);
        }
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        if (full || k0 + s * kStep < end) {
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const avec w = *reinterpret_cast<const avec *>(arow[r] + k0 + s * kStep);
            if constexpr (XF16) {
              acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, x[s], acc[r], 0, 0, 0);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc[r] = __builtin_amdgcn_mfma_f32_16x16x4f32(static_cast<float>(w[i]), x[s][i], acc[r], 0, 0, 0);
            }
          }
        }
    };
    for (int64_t k0 = begin; k0 < end; k0 += SLAB) {
      if (k0 + SLAB <= end)
        slab(k0, std::true_type{});
      else
        slab(k0, std::false_type{});
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
      if (mine) out[r] = acc[r];
  });

  // the four wavefronts' ranges, added in order
  __shared__ float4_t sum[4][RT][64];
#pragma unroll
  for (int r = 0; r < RT; ++r) sum[wave][r][lane] = out[r];
  __syncthreads();
  for (int i = threadIdx.x; i < RT * 64; i += kThreads) {
    const int r = i >> 6, l = i & 63;
    const float4_t v = ((sum[0][r][l] + sum[1][r][l]) + sum[2][r][l]) + sum[3][r][l];
    const int j = rank0 + 16 * r + 4 * (l >> 4);
    const int64_t t = tok0 + (l & 15);
    if (t >= p.n_tokens) continue;
    float *o = p.v + (split * p.n_tokens + t) * p.rank;
    if (p.rank % 4 == 0) {
      if (j < p.rank) *reinterpret_cast<float4_t *>(o + j) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j + e < p.rank) o[j + e] = v[e];
    }
  }
}

struct UpArgs {
  const _Float16 *b;
  const float *v, *scales, *base;
  const int32_t *ids;
  float *y;
  int64_t n_tokens, n_rows;
  int n_adapters, rank, splits;
  int row_tiles, chunks;  // tiles of 16 rows per wavefront, workgroups per token tile
};

// Four values from p[0..3], of which those before `n` exist.
template <bool VEC, class V4, class T> __device__ __forceinline__ V4 load4(const T *p, int64_t n) {
  if constexpr (VEC) {
    return n > 0 ? *reinterpret_cast<const V4 *>(p) : V4{};
  } else {
    V4 v{};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) v[i] = p[i];
    return v;
  }
}

// Y^T = B V^T: a lane holds four consecutive rows of token lane % 16. RQ: 16s
// of the rank; RV, YV: the rows of B and V, and of base and Y, allow 8- and
// 16-byte accesses.
template <int RQ, bool RV, bool YV>
__global__ __launch_bounds__(kThreads) void lora_up_kernel(UpArgs p) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, grp = lane >> 4;
  const int64_t tok = static_cast<int64_t>(blockIdx.x / p.chunks) * kTok + col;
  const bool live = tok < p.n_tokens;
  const int64_t token = live ? tok : p.n_tokens - 1;
  const int id = live ? p.ids[token] : -1;
  const bool valid = id >= 0 && id < p.n_adapters;

  float4_t v[RQ];
#pragma unroll
  for (int q = 0; q < RQ; ++q) v[q] = float4_t{};
  if (valid) {
    const float s = p.scales ? p.scales[id] : 1.f;
    for (int i = 0; i < p.splits; ++i) {
      const float *src = p.v + (i * p.n_tokens + token) * p.rank;
#pragma unroll
      for (int q = 0; q < RQ; ++q) {
        const int j = 16 * q + 4 * grp;
        v[q] += load4<RV, float4_t>(src + j, p.rank - j);
      }
    }
#pragma unroll
    for (int q = 0; q < RQ; ++q) v[q] *= s;
  }

  for (int i = 0; i < p.row_tiles; ++i) {
    const int64_t row0 = ((static_cast<int64_t>(blockIdx.x % p.chunks) * p.row_tiles + i) * 4 + wave) * 16;
    if (row0 >= p.n_rows) break;
    const int64_t r4 = row0 + 4 * grp;
    const int64_t left = live ? p.n_rows - r4 : 0;
    float4_t y{};
    if (p.base) y = load4<YV, float4_t>(p.base + token * p.n_rows + r4, left);
    float4_t d{};
    const int64_t brow = row0 + col < p.n_rows ? row0 + col : p.n_rows - 1;
    each_adapter(id, p.n_adapters, [&](int a, bool mine) {
      const _Float16 *b = p.b + (a * p.n_rows + brow) * p.rank;
      float4_t acc{};
#pragma unroll
      for (int q = 0; q < RQ; ++q) {
        const int j = 16 * q + 4 * grp;
        const half4_t w = load4<RV, half4_t>(b + j, p.rank - j);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc = __builtin_amdgcn_mfma_f32_16x16x4f32(static_cast<float>(w[e]), v[q][e], acc, 0, 0, 0);
      }
      if (mine) d = acc;
    });
    y += d;
    if (id != -1 && !valid) {
      const float nan = __builtin_bit_cast(float, 0x7FC00000u);
      y = float4_t{nan, nan, nan, nan};
    }
    float *o = p.y + token * p.n_rows + r4;
    if constexpr (YV) {
      if (left > 0) *reinterpret_cast<float4_t *>(o) = y;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) o[e] = y[e];
    }
  }
}

// Few tiles: short ranges of k, so that the adapters' rows are read by many
// workgroups at once. Many: longer ones, which leave fewer partial sums.
bool few_tiles(int64_t n_tokens, int64_t k, int64_t rank) {
  const int64_t groups = (n_tokens + kTok - 1) / kTok * ((rank + kRankGroup - 1) / kRankGroup);
  return groups * ((k + 4 * kSlab - 1) / (4 * kSlab)) < 256;
}
int lora_rounds(int64_t n_tokens, int64_t k, int64_t rank) {
  if (few_tiles(n_tokens, k, rank)) return 1;
  const int64_t groups = (n_tokens + kTok - 1) / kTok * ((rank + kRankGroup - 1) / kRankGroup);
  const int64_t most = (k + 4 * kSlab - 1) / (4 * kSlab);
  const int64_t want = std::min(most, std::max<int64_t>(1, (768 + groups - 1) / groups));
  return static_cast<int>((most + want - 1) / want);
}

}  // namespace

int lora_splits(int64_t n_tokens, int64_t k, int64_t rank) {
  const int64_t per = int64_t{4} * (few_tiles(n_tokens, k, rank) ? kSlabFew : kSlab) * lora_rounds(n_tokens, k, rank);
  return static_cast<int>((k + per - 1) / per);
}

hipError_t launch_lora(const void *X, bool x_f16, int64_t n_tokens, int64_t k, const void *A, const void *B,
                       int64_t n_adapters, int64_t rank, int64_t n_rows, const float *scales, const int32_t *ids,
                       const float *base, float *Y, float *partial, hipStream_t stream) {
  const bool few = few_tiles(n_tokens, k, rank);
  const int splits = lora_splits(n_tokens, k, rank);
  const int64_t tiles = (n_tokens + kTok - 1) / kTok;
  DownArgs d{X, static_cast<const _Float16 *>(A), ids, partial, n_tokens, k, static_cast<int>(n_adapters),
             static_cast<int>(rank), splits, lora_rounds(n_tokens, k, rank)};
  const dim3 grid(static_cast<unsigned>(tiles), splits, static_cast<unsigned>((rank + kRankGroup - 1) / kRankGroup));
  const dim3 block(kThreads);
  auto down = [&](auto xf16, auto rt) {
    constexpr bool X16 = decltype(xf16)::value;
    constexpr int RT = decltype(rt)::value;
    return few ? launch(lora_down_kernel<X16, RT, kSlabFew>, grid, block, 0, stream, d)
               : launch(lora_down_kernel<X16, RT, kSlab>, grid, block, 0, stream, d);
  };
  auto by_rank = [&](auto xf16) {
    if (rank <= 16) return down(xf16, std::integral_constant<int, 1>{});
    if (rank <= 32) return down(xf16, std::integral_constant<int, 2>{});
    return down(xf16, std::integral_constant<int, 4>{});
  };
  const hipError_t e = x_f16 ? by_rank(std::true_type{}) : by_rank(std::false_type{});
  if (e != hipSuccess) return e;

  // 64 rows per workgroup and step; several steps where there are workgroups
  // enough, since each one first adds up its tokens' V
  const int64_t steps = (n_rows + 63) / 64;
  const int64_t row_tiles = std::max({int64_t{1}, std::min<int64_t>(16, steps * tiles / 1024), (steps * tiles) >> 23});
  const int64_t chunks = (steps + row_tiles - 1) / row_tiles;
  UpArgs u{static_cast<const _Float16 *>(B), partial, scales, base, ids, Y, n_tokens, n_rows,
           static_cast<int>(n_adapters), static_cast<int>(rank), splits, static_cast<int>(row_tiles),
           static_cast<int>(chunks)};
  const dim3 ugrid(static_cast<unsigned>(chunks * tiles));
  const bool rv = rank % 4 == 0 && reinterpret_cast<uintptr_t>(B) % 8 == 0;
  const bool yv = n_rows % 4 == 0 && reinterpret_cast<uintptr_t>(Y) % 16 == 0 && reinterpret_cast<uintptr_t>(base) % 16 == 0;
  auto up = [&](auto rq) {
    constexpr int RQ = decltype(rq)::value;
    if (rv && yv) return launch(lora_up_kernel<RQ, true, true>, ugrid, block, 0, stream, u);
    if (rv) return launch(lora_up_kernel<RQ, true, false>, ugrid, block, 0, stream, u);
    if (yv) return launch(lora_up_kernel<RQ, false, true>, ugrid, block, 0, stream, u);
    return launch(lora_up_kernel<RQ, false, false>, ugrid, block, 0, stream, u);
  };
  if (rank <= 16) return up(std::integral_constant<int, 1>{});
  if (rank <= 32) return up(std::integral_constant<int, 2>{});
  if (rank <= 64) return up(std::integral_constant<int, 4>{});
  return up(std::integral_constant<int, 16>{});
}

}  // namespace qmm
