// kvo_attend_chunk: causal attention of prompt chunks over a paged cache.  With
// the columns c = (token, head) of a sequence and its positions p:
//     z_pc = scale * k_p . q_c,   out_c = sum_p exp(z_pc - lse_c) v_p,
//     lse_c = log sum_p exp(z_pc),  over the positions that c's token sees.
//
// Chunks with few columns go through the kernel of kvo_attend, which
// dequantises rows for 64 columns at a time.  With many, the rows are first
// unpacked to bf16 in the caller's scratch, once, and pairs of CTAs take 128
// columns and 256 positions at a time:
//     S^T [256 positions x 128 columns]      = K [256 x 576] Q^T
//     O^T [512 values x 128 columns]        += V^T [512 x 256] P^T
// as pair MMAs with M = 256: a CTA holds 128 of the positions for the first
// product and 256 of the values for the second, so that O^T takes 256 of its
// 512 columns of tensor memory and S^T, twice, the rest.  The columns' operand
// is halved between them: 64 columns of queries (72 KB) and of weights (32 KB
// for 256 positions) lie in each CTA's shared memory; the positions' operands
// stream through a ring of six pieces of 16 KB (128 positions of 64 values
// for the first product, 64 positions of 128 values for the second).
//
// Sixteen worker warps do the softmax: a lane of S^T is a position.  The
// weights of the other CTA's 64 columns go to it as one bulk copy (16 KB);
// stored there directly they took 3,700 clocks a tile, most of them in the
// fence before the MMAs.  Maxima and sums go the same way.
// The softmax's reference is the column's maximum in the first tile of
// positions and 2^32 above it.  Weights within 2^+-64 of it lose nothing in
// fp32 and bf16; where a later logit lies further above, or the first tile shows
// a column nothing and a later one does, the tile is done again at the end,
// with the true maximum from a pass over its logits.  So no tile waits for a
// maximum.
//
// Tiles of columns times tiles of positions, end to end, are shared out evenly
// over the pairs, or over rows of up to four pairs that take as many tiles of
// columns and go over the same positions at the same time.  Where a share begins
// or ends inside a tile of columns, the parts are joined by their log-sum-exps in
// a last launch.
//
// Measured: 512 tokens of 64 heads over 50,023 positions 2.07-2.14 ms (1.66-1.72
// PFLOP/s; 2.26 ms back to back, at the power limit), 2,048 of 128 heads over
// 16,384 5.35-5.54 ms, a prompt of 4,096 tokens and 16 heads alone 246 us (its tiles of
// columns meet 8.5 tiles of positions on average, and beginning and ending one
// takes the time of two), 16 sequences of 8,192 rows with 4,096 columns each 850
// us (1.37 PFLOP/s).  A tile of 256 positions is 68 MMAs of 64 clocks, 4,352,
// and keeps shared memory busy for 6,300 wavefronts of 128 bytes: 3,250 of the
// MMAs' operands, 2,180 of the copies, 900 of the workers.  That is the bound.
// Steps, ms for the first case: rows dequantised for 64 columns at a time 7.17,
// pairs 3.80, copies instead of stores to the other CTA 3.27, three loading warps
// and no order over the cluster in the workers' loop 2.45, a loop for each role
// 2.24; the last two with two pairs that shared a ring, each bringing half of
// every piece for both: a pair by itself takes 2.10, as all 152 SMs have work then
// (two such pairs leave 8 out) and no pair waits for another.
#include <algorithm>

#include "kvo_cache.cuh"
#include "kvo_chunk.cuh"
#include "kvo_rows.cuh"
#include "kvo_tc.cuh"

namespace kvo {

// The kernel for few columns (kvo_attend.cu).
int64_t few_columns_work(int64_t tokens, int64_t sequences, uint32_t heads, int64_t rows);
cudaError_t launch_few_columns(const kvo_cache& cache, const kvo_chunk_query& s, uint32_t* status, int64_t wait_clocks,
                               cudaStream_t stream);

namespace {

constexpr uint32_t kSpan = 256;                          // positions of a tile
constexpr uint32_t kTileColumns = 2 * kColumns;          // of a pair of CTAs
constexpr uint32_t kTileCost = 2;                        // of a tile of columns, in tiles of positions
constexpr uint32_t kWorkers = 16;
constexpr uint32_t kMma = kWorkers, kLoader = kWorkers + 1;
constexpr uint32_t kLoaders = 3;                         // warps: one takes 500 clocks a copy beside the workers
constexpr uint32_t kChunkThreads = (kLoader + kLoaders) * 32;
constexpr uint32_t kQueryBytes = 9 * kColumns * 128;
constexpr uint32_t kHalfBytes = kSpan / 2 * 128;         // a CTA's positions' weights of 64 columns
constexpr uint32_t kSlotBytes = 16384, kSlots = 6;
constexpr uint32_t kChunkSmem = 1024 + kQueryBytes + 3 * kHalfBytes + kSlots * kSlotBytes;
constexpr uint32_t kValueBytes = KVO_DEQUANT_VALUES * 2;
static_assert(9 % kLoaders == 0 && kSlots % kLoaders == 0, "even shares of the queries, and a warp its own slots");
constexpr uint32_t kMostAbreast = 4;
constexpr float kRoom = 32.0f;                           // of a reference above the first tile's maximum, in powers of two

// One tile of columns, as the plan lists it.  `abreast` tiles are a row of the
// plan, one for each of as many pairs next to each other.
struct __align__(16) PlanTile {
  uint64_t units;            // work of all rows before it: their longest's tiles of positions and kTileCost each
  int32_t seq;
  uint32_t index;            // of its sequence's tiles
  uint32_t first, tokens;    // its sequence's tokens
  int32_t before;            // token i sees the first before + i positions
  uint16_t spans, longest;   // its tiles of positions; the longest of its row
};

// A tile that ends of shares cut, as the join takes it: of share g - 1 the part
// that ends inside it, of g .. last those that begin there.
struct __align__(16) Cut {
  PlanTile tile;
  uint32_t last;             // 0: share g is not the first to begin inside a tile
  uint32_t pad[3];
};

struct ChunkArgs {
  CacheView cache;
  const int32_t* starts;
  const int32_t* lens;
  uint16_t* out;
  float* lse;
  uint8_t* values;           // [sequences][span][576] bf16, of the group in turn
  float* off;                // [sequences][span]: 0, or -inf where there is no row
  PlanTile* plan;            // [tiles + 1]: the last one's units are all of them
  Cut* cuts;                 // [pairs], `abreast` for a share, from share 1 on
  uint8_t* again;            // [most_tiles] whole tiles, [2 * pairs] parts that need another pass
  float* part;               // [2 * pairs][128][512]
  float* part_lse;           // [2 * pairs][128], base 2
  uint32_t* status;
  uint32_t rows, span, tokens, heads, most_tiles;
  uint32_t pairs, abreast;   // pairs: a multiple of abreast
  uint32_t unpack_blocks;    // of a sequence
  Divider by_heads;
  Columns columns;
  float scale;               // times log2(e)
  float far;                 // a logit this far above its reference wants another pass
  int64_t wait_clocks;
};

// ---------------------------------------------------------------- the shares
// The share of pairs g * abreast and those behind it: [from(g), from(g + 1)).
struct Shares {
  uint64_t units, each;
  uint32_t count, rest;              // the first `rest` shares have one more than `each`
  __device__ __forceinline__ Shares(const ChunkArgs& a) {
    units = __ldcg(&a.plan[a.most_tiles + 1].units);
    count = (uint32_t)min((uint64_t)(a.pairs / a.abreast), max(units / 2, (uint64_t)1));
    each = units / count;
    rest = (uint32_t)(units - each * count);
  }
  __device__ __forceinline__ uint64_t from(uint32_t g) const { return g < count ? g * each + min(g, rest) : units; }
};

// The first tile of the row that unit u lies in; a whole warp.
__device__ __forceinline__ uint32_t tile_of(const ChunkArgs& a, uint64_t u) {
  uint32_t lo = 0, hi = __ldcg(&a.plan[a.most_tiles + 1].index);   // in [lo, hi)
  const uint32_t lane = threadIdx.x & 31;
  while (hi - lo > 1) {
    const uint32_t step = (hi - lo + 31) / 32, at = lo + lane * step;
    const bool before = at < hi && __ldcg(&a.plan[at].units) <= u;
    const uint32_t n = __popc(__ballot_sync(0xffffffffu, before));   // lane 0's always is
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
  }
  return lo / a.abreast * a.abreast;
}

__device__ __forceinline__ PlanTile plan_tile(uint4 x, uint4 y) {
  return PlanTile{(uint64_t)x.y << 32 | x.x, (int32_t)x.z,           x.w, y.x, y.y, (int32_t)y.z,
                  (uint16_t)(y.w & 0xffffu), (uint16_t)(y.w >> 16)};
}
__device__ __forceinline__ PlanTile plan_tile(const ChunkArgs& a, uint32_t i) {
  const uint4* const from = reinterpret_cast<const uint4*>(a.plan + i);
  const uint4 x = __ldcg(from), y = __ldcg(from + 1);
  return plan_tile(x, y);
}

// ------------------------------------------------------------ rows and plan
constexpr uint32_t kUnpackThreads = 256, kUnpackRows = 64;   // of a CTA, 8 of a warp

__device__ __forceinline__ uint32_t visible(const ChunkArgs& a, int32_t before, uint32_t token) {
  return (uint32_t)min(max(before + (int32_t)token, 0), (int32_t)a.rows);
}

// The token of column `in_half` of half tile `half`; >= tokens where there is none.
__device__ __forceinline__ uint32_t column_at(const ChunkArgs& a, const PlanTile& t, uint32_t half, uint32_t in_half,
                                              uint32_t* at) {
  const Columns& c = a.columns;
  const uint32_t deep = divide(in_half, c.by_wide), wide = in_half - deep * c.wide;
  const uint32_t row = half / c.across * c.deep + deep, head = half % c.across * c.wide + wide;
  *at = c.flat ? row : row * a.heads + head;
  if (deep >= c.deep || (!c.flat && head >= a.heads)) return UINT32_MAX;
  return divide(*at, a.by_heads);
}

// The last token of a tile.
__device__ __forceinline__ uint32_t last_token(const ChunkArgs& a, uint32_t index, uint32_t tokens) {
  const Columns& c = a.columns;
  const uint32_t rows = (2 * index + 1) / c.across * c.deep + c.deep;   // up to the tile's end
  return min(c.flat ? divide(min(rows, tokens * a.heads) - 1, a.by_heads) : rows - 1, tokens - 1);
}

// One CTA lists the tiles: 256 sequences at a time, then their tiles.
__device__ void make_plan(const ChunkArgs& a) {
  __shared__ uint32_t upto[kUnpackThreads], first[kUnpackThreads], count[kUnpackThreads];
  __shared__ uint64_t sums[kUnpackThreads / 32];
  __shared__ uint32_t tile_sums[kUnpackThreads / 32];
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Columns& c = a.columns;
  uint32_t tiles = 0;
  uint64_t units = 0;
  for (uint32_t i = tid; i < a.most_tiles + 2 * a.pairs; i += kUnpackThreads) a.again[i] = 0;
  for (uint32_t s0 = 0; s0 < a.cache.sequences; s0 += kUnpackThreads) {
    const uint32_t s = s0 + tid;
    uint32_t mine = 0;
    if (s < a.cache.sequences) {
      const Tokens t = tokens_of(a.starts, s, a.tokens);
      if (t.bad) atomicOr(a.status, kFlagRange);
      first[tid] = t.first;
      count[tid] = t.count;
      const uint32_t rows = c.flat ? count[tid] * a.heads : count[tid];
      mine = ((rows + c.deep - 1) / c.deep * c.across + 1) / 2;
    }
    uint32_t incl = mine;
#pragma unroll
    for (uint32_t d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) tile_sums[warp] = incl;
    __syncthreads();
    for (uint32_t w = 0; w < warp; ++w) incl += tile_sums[w];
    upto[tid] = incl;
    __syncthreads();
    // (starts that go back could list more tiles than there is room for)
    const uint32_t real = min(upto[kUnpackThreads - 1], (a.most_tiles - tiles) / a.abreast * a.abreast);
    const uint32_t all = (real + a.abreast - 1) / a.abreast * a.abreast;   // the last row's rest: tiles of nothing
    for (uint32_t j0 = 0; j0 < all; j0 += kUnpackThreads) {
      const uint32_t j = j0 + tid;
      PlanTile t = {};
      if (j < real) {
        uint32_t lo = 0, hi = kUnpackThreads - 1;        // the first with upto > j
        while (lo < hi) {
          const uint32_t mid = (lo + hi) / 2;
          if (upto[mid] > j) hi = mid; else lo = mid + 1;
        }
        t.seq = (int32_t)(s0 + lo);
        t.index = j - (lo ? upto[lo - 1] : 0);
        t.first = first[lo];
        t.tokens = count[lo];
        t.before = min(max(a.lens[t.seq], 0), INT32_MAX - 1) - (int32_t)t.tokens + 1;
        t.spans = (uint16_t)max((visible(a, t.before, last_token(a, t.index, t.tokens)) + kSpan - 1) / kSpan, 1u);
      }
      uint32_t longest = t.spans;
      for (uint32_t d = 1; d < a.abreast; d <<= 1) longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, d));
      t.longest = (uint16_t)longest;
      const uint64_t n = j < all ? longest + kTileCost : 0;
      uint64_t sum = tid % a.abreast == 0 ? n : 0;
#pragma unroll
      for (uint32_t d = 1; d < 32; d <<= 1) {
        const uint64_t o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
      }
      if (lane == 31) sums[warp] = sum;
      __syncthreads();
      uint64_t total = 0;
      for (uint32_t w = 0; w < kUnpackThreads / 32; ++w) {
        if (w < warp) sum += sums[w];
        total += sums[w];
      }
      if (j < all) {
        t.units = units + sum - n;
        a.plan[tiles + j] = t;
      }
      units += total;
      __syncthreads();
    }
    tiles += all;
    __syncthreads();
  }
  if (tid == 0) {
    // the end's units, and the number of tiles in its index
    PlanTile end = {};
    end.units = units;
    a.plan[tiles] = end;
    PlanTile head = {};
    head.units = units;
    head.index = tiles;
    a.plan[a.most_tiles + 1] = head;
  }
  __threadfence_block();
  __syncthreads();
  const Shares shares(a);
  for (uint32_t i = a.abreast + warp; i < shares.count * a.abreast; i += kUnpackThreads / 32) {
    const uint32_t g = i / a.abreast;
    const uint64_t at = shares.from(g);
    Cut cut;
    cut.tile = plan_tile(a, tile_of(a, at) + i % a.abreast);
    const uint64_t from = cut.tile.units, end = from + cut.tile.spans;
    cut.last = 0;
    if (at > from && at < end && shares.from(g - 1) <= from) {
      cut.last = g;
      while (cut.last + 1 < shares.count && shares.from(cut.last + 1) < end) ++cut.last;
    }
    if (lane == 0) a.cuts[i] = cut;
  }
}

// The rows that a tile of positions may hold as bf16.  A row that reads as NaN
// somewhere gets zero latents and a NaN position part: its logits are NaN, as
// they would have been, and a weight of 0 keeps it out of the second product.
__global__ void __launch_bounds__(kUnpackThreads) unpack_kernel(const __grid_constant__ ChunkArgs a) {
  wait_previous_grid();
  allow_next_grid();
  if (blockIdx.x == 0) {
    make_plan(a);
    return;
  }
  const uint32_t s = (blockIdx.x - 1) / a.unpack_blocks, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t p0 = ((blockIdx.x - 1) % a.unpack_blocks) * kUnpackRows + warp * 8;
  const uint32_t len = (uint32_t)min(max(a.lens[s], 0), (int32_t)a.rows);
  if (p0 >= (max(len, 1u) + kSpan - 1) / kSpan * kSpan) return;
  // rows that no token looks at: they may be on pages that are not there
  if (tokens_of(a.starts, s, a.tokens).count == 0) return;
  int64_t row = -1;
  if (lane < 8) {
    const uint32_t p = p0 + lane;
    if (p < len) {
      row = cache_row(a.cache, s, p);
      if (row < 0) atomicOr(a.status, kFlagRange);
    }
    a.off[(int64_t)s * a.span + p] = row < 0 ? -INFINITY : 0.0f;
  }
  uint4 lat[8], eight[8], rope[8];
  const uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (uint32_t r = 0; r < 8; ++r) {
    const int64_t at = __shfl_sync(0xffffffffu, row, r);
    const uint4* from = reinterpret_cast<const uint4*>(a.cache.rows) + at * (KVO_ROW_BYTES / 16);
    lat[r] = at >= 0 ? __ldg(from + lane) : none;
    eight[r] = at >= 0 ? __ldg(from + KVO_LATENT_BYTES / 16) : none;
    rope[r] = at >= 0 && lane < 8 ? __ldg(from + KVO_LATENT_BYTES / 16 + 1 + lane) : none;
  }
#pragma unroll
  for (uint32_t r = 0; r < 8; ++r) {
    const bool bad = any_not_finite(eight[r]);
    const uint32_t g = lane >> 2;                        // the lane's group of 64 values
    const uint32_t two = g < 4 ? (g < 2 ? eight[r].x : eight[r].y) : (g < 6 ? eight[r].z : eight[r].w);
    const uint16_t scale = bad ? 0 : (uint16_t)(two >> (g & 1) * 16);
    const float bias = -1152.0f * __half2float(__ushort_as_half(scale));
    uint4 x, y;
    dequant4(lat[r].x, scale, bias, x.x, x.y);
    dequant4(lat[r].y, scale, bias, x.z, x.w);
    dequant4(lat[r].z, scale, bias, y.x, y.y);
    dequant4(lat[r].w, scale, bias, y.z, y.w);
    uint4* const to = reinterpret_cast<uint4*>(a.values + ((int64_t)s * a.span + p0 + r) * kValueBytes);
    to[2 * lane] = x;
    to[2 * lane + 1] = y;
    if (lane < 8) to[64 + lane] = bad ? make_uint4(~0u, ~0u, ~0u, ~0u) : rope[r];
  }
}

// ---------------------------------------------------------------- the segments
// A share's part of one tile of columns: tiles of positions [from, to).
struct Segment {
  PlanTile tile;
  uint32_t number, from, to;
  bool whole;
  // where a segment notes that it needs another pass, and its result if it is
  // part of a tile: a share has one that begins inside a tile and one that
  // ends inside one at most
  __device__ __forceinline__ uint32_t slot(uint32_t pair) const { return 2 * pair + (from == 0); }
  __device__ __forceinline__ uint32_t note(const ChunkArgs& a, uint32_t pair) const {
    return whole ? number : a.most_tiles + slot(pair);
  }
};

// f(segment) for every segment of a pair's share, in order, in every warp, from
// tile `tile` on.  tile_at(i): tile i of the plan.
template <typename T, typename F>
__device__ __forceinline__ void for_segments(const ChunkArgs& a, uint64_t begin, uint64_t end, uint32_t tile, T tile_at, F f) {
  for (uint64_t u = begin; u < end; tile += a.abreast) {
    Segment g;
    g.tile = tile_at(tile);
    const uint64_t past = g.tile.units + g.tile.longest + kTileCost;
    g.number = tile;
    g.from = min((uint32_t)(u - g.tile.units), (uint32_t)g.tile.spans);
    g.to = min((uint32_t)(min(past, end) - g.tile.units), (uint32_t)g.tile.spans);
    g.whole = g.to - g.from == g.tile.spans;
    u = past;
    if (g.from < g.to && !f(g)) return;
  }
}

// What a pair's CTAs send each other: weights of the other's columns, maxima of
// the columns, sums of their weights.
enum Letter : uint32_t { kGift, kTop, kSum, kLetters };

struct Sums {
  float of[4][4][32];                // per quarter of the columns and warp
  uint32_t again[kWorkers];          // per warp: this segment needs another pass
};

struct ChunkShared {
  uint64_t full[kSlots], empty[kSlots], q_full, q_empty, s_full[2], s_empty[2], p_full, p_empty, o_empty;
  uint64_t ready[kLetters], come[kLetters], drained;
  uint32_t tmem, gave_up;
  // per CTA and loading warp: copies of its own and before them that it has started, and queries
  uint32_t issued[2][kLoaders], q_issued[2][kLoaders];
  uint32_t sent[kLetters], armed[kLetters];   // letters that the other CTA has sent, and that this one has been ready for
  uint32_t redo;                     // some segment needs another pass
  alignas(16) float top[2][4][4][32];         // per CTA, quarter of the columns and warp: maxima
  alignas(16) Sums sums[2];
  // per column: the softmax's reference, and after a segment 1 / the sum of its
  // weights; the positions it sees.  The four warps of a quarter write the same
  // values, when all of them have done with the ones before.
  alignas(16) float ref[4][32];
  alignas(16) uint32_t seen[4][32];
  PlanTile upcoming[2];              // the workers' next tile, in turns
};

template <uint32_t kN, uint32_t kBit>
__device__ __forceinline__ void add_lanes(float* v, uint32_t lane) {
  // a step halves the columns that a lane keeps: v[0] is column lane's sum at last
  const bool up = lane & kBit;
#pragma unroll
  for (uint32_t c = 0; c < kN / 2; ++c) {
    const float stay = up ? v[c + kN / 2] : v[c], give = up ? v[c] : v[c + kN / 2];
    v[c] = stay + __shfl_xor_sync(0xffffffffu, give, kBit);
  }
  if constexpr (kBit > 1) add_lanes<kN / 2, kBit / 2>(v, lane);
}

__global__ void __launch_bounds__(kChunkThreads, 1)
    chunk_kernel(const __grid_constant__ ChunkArgs a, const __grid_constant__ CUtensorMap qmap,
                 const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ uint8_t raw[];
  __shared__ ChunkShared sh;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank(), other = rank ^ 1, pair = blockIdx.x >> 1;
  constexpr uint16_t kBoth = 3;
  const uint32_t queries = (smem_u32(raw) + 1023u) & ~1023u, probs = queries + kQueryBytes;
  const uint32_t gift = probs + 2 * kHalfBytes, ring = gift + kHalfBytes;

  if (tid == 0) {
    for (uint32_t i = 0; i < kSlots; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 1);
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_empty[i], 2 * kWorkers);
    }
    for (uint32_t i = 0; i < 2; ++i)
      for (uint32_t w = 0; w < kLoaders; ++w) sh.issued[i][w] = sh.q_issued[i][w] = 0;
    mbar_init(&sh.p_full, kWorkers + 1);                 // both CTAs' own columns, and that rank 1 has all of its
    for (uint32_t i = 0; i < kLetters; ++i) {
      mbar_init(&sh.ready[i], i == kGift ? kWorkers / 2 : kWorkers);
      mbar_init(&sh.come[i], 1);
      sh.sent[i] = sh.armed[i] = 0;
    }
    mbar_init(&sh.p_empty, 1);
    mbar_init(&sh.o_empty, 2 * kWorkers);
    mbar_init(&sh.drained, 1);
    sh.gave_up = a.wait_clocks == 0;
    sh.redo = 0;
  }
  if (warp == kMma) pair_tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  wait_previous_grid();
  allow_next_grid();

  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return wait_or_give_up(bar, parity, &sh.gave_up, a.wait_clocks);
  };
  const Shares shares(a);
  const uint32_t share = pair / a.abreast;
  const uint64_t begin = shares.from(share), end = share < shares.count ? shares.from(share + 1) : begin;
  const uint32_t tile0 = begin < end ? tile_of(a, begin) + pair % a.abreast : 0;
  const uint32_t box = a.columns.wide * a.columns.deep * 128;

  // The roles' counters run on over segments and passes.
  uint32_t n = 0, q_n = 0;                               // copies; segments' queries
  uint32_t it = 0, pv = 0;                               // tiles of S; second products
  uint32_t full_n = 0, met_n = 0;                        // whole passes; exchanges of maxima
  uint32_t sent[kLetters] = {};                          // by this thread
  uint32_t upcoming_number = UINT32_MAX;                 // the tile that the workers have asked for
  bool ok = true;

  // One segment's work for each role; max_only: only the columns' maxima.
  //
  // Loading warp w takes every kLoaders-th copy from copy w on, and as many of
  // the queries' nine.
  const uint32_t load_warp = warp - kLoader, full0 = dsmem_addr(&sh.full[0], 0);
  auto load = [&](const Segment& g, bool max_only) -> bool {
    const uint32_t tiles = g.to - g.from;
    if (lane == 0) {
      if (q_n > 0) ok = ok && wait(&sh.q_empty, (q_n - 1) & 1);
      if (ok) {
        const uint32_t half = 2 * g.tile.index + rank, row = half / a.columns.across, bar = dsmem_addr(&sh.q_full, 0);
        if (rank == 0 && load_warp == 0) mbar_arrive_expect_tx(&sh.q_full, 2 * 9 * box);
        for (uint32_t i = load_warp; i < 9; i += kLoaders)
          pair_load_box(queries + i * (kColumns * 128), &qmap, (int32_t)(i * 64),
                        (int32_t)(half % a.columns.across * a.columns.wide),
                        (int32_t)((a.columns.flat ? g.tile.first * a.heads : g.tile.first) + row * a.columns.deep), bar);
        ++q_n;
      }
      uint32_t at = n;                                   // the copy that a run of them begins with
      // the next `count` copies, the k-th from a map's (0, y(k), z(k)) on
      auto copies = [&](const CUtensorMap* map, uint32_t count, auto&& y, auto&& z) {
        for (uint32_t k = (load_warp + kLoaders - at % kLoaders) % kLoaders; k < count && ok; k += kLoaders) {
          const uint32_t m = at + k, slot = m % kSlots;
          if (m >= kSlots) ok = wait(&sh.empty[slot], (m / kSlots - 1) & 1);
          if (!ok) break;
          if (rank == 0) mbar_arrive_expect_tx(&sh.full[slot], 2 * kSlotBytes);
          pair_load_box(ring + slot * kSlotBytes, map, 0, (int32_t)y(k), (int32_t)z(k), full0 + slot * 8);
          n = m + 1;
        }
        at += count;
      };
      const uint32_t first = (uint32_t)g.tile.seq * a.span;
      for (uint32_t i = 0; i <= tiles && ok; ++i) {
        const uint32_t row = first + (g.from + i) * kSpan;
        if (i < tiles)
          copies(&kmap, 9, [&](uint32_t) { return row + rank * (kSpan / 2); }, [](uint32_t k) { return k; });
        if (i > 0 && !max_only)
          copies(&vmap, 8, [&](uint32_t k) { return row - kSpan + (k & 3) * 64; },
                 [&](uint32_t k) { return (k >> 2) * 4 + rank * 2; });
      }
      if (ok) n = at;
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    return ok;
  };

  // Letters go as bulk copies: what a warp stores to the other CTA's memory
  // itself, and the order over the cluster behind it, takes 2,000 to 4,000 clocks.
  // arm: one thread of the receiver, for the n-th letter of its kind; send: one
  // thread, after everyone who wrote it has passed a proxy fence and arrived.
  auto arm = [&](Letter kind, uint32_t n, uint32_t bytes) {
    mbar_arrive_expect_tx(&sh.come[kind], bytes);
    sh.armed[kind] = n + 1;
  };
  auto send = [&](Letter kind, uint32_t dst, uint32_t src, uint32_t bytes) {
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(dst), "r"(other));
    bulk_copy_s2peer(there, src, bytes, dsmem_addr(&sh.come[kind], other));
    ++sent[kind];
  };
  // the weights that the other CTA sends, the p-th of them; one thread
  auto come = [&](uint32_t p) -> bool {
    arm(kGift, p, kHalfBytes);
    return wait(&sh.come[kGift], p & 1);
  };
  // every worker warp has written its part of this CTA's letter, the n-th of its kind: both CTAs' are there afterwards
  auto trade = [&](Letter kind, uint32_t n, const void* mine, uint32_t bytes) -> bool {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.ready[kind]);
    bool there = wait(&sh.ready[kind], n & 1);
    if (tid == 0 && there) {
      arm(kind, n, bytes);
      send(kind, smem_u32(mine), smem_u32(mine), bytes);
    }
    __syncwarp();
    there = there && wait(&sh.come[kind], n & 1);
    return __all_sync(0xffffffffu, there);
  };

  // One thread issues all of a segment's MMAs: what it does between them has
  // to fit into the 256 clocks that four take, beside the workers' instructions.
  // (Waits of the whole warp, with a vote, a fence and an election for every
  // four: 430 clocks.)
  auto multiply = [&](const Segment& g, bool max_only) -> bool {
    constexpr uint32_t kQk = pair_desc(1, kTileColumns, false, false), kPv = pair_desc(1, kTileColumns, true, true);
    const uint32_t tiles = g.to - g.from;
    if (ok && elect_one()) {
      const uint64_t q_desc = tile_desc(queries, 16), k_desc = tile_desc(ring, 16);
      const uint64_t p_desc = tile_desc(probs, 16), v_desc = tile_desc(ring, kSlotBytes / 2);
      uint32_t slot = n % kSlots, turn = n / kSlots & 1;
      auto next = [&] {
        if (++slot == kSlots) {
          slot = 0;
          turn ^= 1;
        }
      };
      ok = wait(&sh.q_full, q_n & 1);
      for (uint32_t i = 0, t = it, p = pv; i <= tiles && ok; ++i) {
        if (i < tiles) {
          const uint32_t buf = t & 1, d = tmem + 256 + buf * kTileColumns;
          if (t >= 2) ok = wait(&sh.s_empty[buf], ((t >> 1) - 1) & 1);
          tc_fence_after();
#pragma unroll 3
          for (uint32_t k = 0; k < 9 && ok; ++k, next()) {
            ok = wait(&sh.full[slot], turn);
            if (!ok) break;
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e)
              pair_mma_bf16(d, k_desc + slot * (kSlotBytes >> 4) + 2 * e, q_desc + k * (kColumns * 128 >> 4) + 2 * e, kQk,
                            k + e > 0);
            pair_commit(&sh.empty[slot], kBoth);
          }
          if (!ok) break;
          pair_commit(&sh.s_full[buf], kBoth);
          if (i + 1 == tiles) pair_commit(&sh.q_empty, kBoth);
          ++t;
        }
        if (i > 0 && !max_only) {
          ok = come(p) && wait(&sh.p_full, p & 1);
          if (i == 1 && full_n > 0) ok = ok && wait(&sh.o_empty, (full_n - 1) & 1);
          tc_fence_after();
#pragma unroll 4
          for (uint32_t k = 0; k < 8 && ok; ++k, next()) {
            ok = wait(&sh.full[slot], turn);
            if (!ok) break;
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e)
              pair_mma_bf16(tmem + (k / 4) * kTileColumns, v_desc + slot * (kSlotBytes >> 4) + 128 * e,
                            p_desc + (k % 4) * 512 + 128 * e, kPv, i > 1 || k % 4 + e > 0);
            pair_commit(&sh.empty[slot], kBoth);
          }
          if (!ok) break;
          pair_commit(&sh.p_empty, kBoth);
          ++p;
        }
      }
    }
    ok = __all_sync(0xffffffffu, ok);
    ++q_n;
    n += tiles * (max_only ? 9 : 17);
    it += tiles;
    if (!max_only) {
      pv += tiles;
      ++full_n;
    }
    return ok;
  };

  // rank 1's warp without MMAs tells rank 0 when its weights have come
  auto pass_on = [&](const Segment& g, bool max_only) -> bool {
    for (uint32_t i = g.from; i < g.to && !max_only; ++i, ++pv) {
      if (lane == 0) {
        ok = come(pv);
        if (ok) cluster_mbar_arrive_own(dsmem_addr(&sh.p_full, 0));
      }
      if (!__all_sync(0xffffffffu, ok)) return false;
    }
    return true;
  };

  // A worker's position of a tile: rank * 128 + quad * 32 + lane; its columns: quarter * 32 + c.
  const uint32_t quad = warp & 3, quarter = (warp >> 2) & 3, mine = rank * 128 + quad * 32 + lane;
  const uint32_t lanes = tmem + (quad << 21);
  auto arrive0 = [&](uint64_t* bar) {                    // at rank 0's, for the warp's loads from tensor memory
    __syncwarp();
    if (lane == 0) cluster_mbar_arrive_relaxed(dsmem_addr(bar, 0));
  };
  // the maxima of this warp's columns (lane c: column c's) to both CTAs, and back the whole tile's
  auto meet = [&](float best) -> float {
    sh.top[rank][quarter][quad][lane] = best;
    ok = ok && trade(kTop, met_n, &sh.top[rank], sizeof(sh.top[0]));
    ++met_n;
    float m = -INFINITY;
    for (uint32_t r = 0; r < 2; ++r)
      for (uint32_t w = 0; w < 4; ++w) m = fmaxf(m, ((volatile float*)sh.top[r][quarter][w])[lane]);
    return m;
  };

  // first: the references are still to be found
  auto soften = [&](const Segment& g, bool max_only, bool first) -> bool {
    uint32_t at;
    const uint32_t token = column_at(a, g.tile, 2 * g.tile.index + quarter / 2, quarter % 2 * 32 + lane, &at);
    const bool real = token < g.tile.tokens;
    const uint32_t sees = real ? visible(a, g.tile.before, token) : UINT32_MAX;   // (others hold nothing up)
    const uint32_t least = __reduce_min_sync(0xffffffffu, sees);
    __syncwarp();
    sh.seen[quarter][lane] = sees;
    __syncwarp();
    // (what a column that is none multiplies may be anything: its weights are zeros, or NaN for itself alone)
    auto reference = [&](float best) { return !real ? INFINITY : fabsf(best) < INFINITY ? best : 0.0f; };
    float sum[32];                                       // or maxima
#pragma unroll
    for (uint32_t c = 0; c < 32; ++c) sum[c] = max_only ? -INFINITY : 0.0f;
    uint32_t flagged = 0;
    const float* const off = a.off + (int64_t)g.tile.seq * a.span;
    if (warp == 0 && !max_only) {                        // the next segment's tile, there once the sums have been traded
      if (lane < 2)
        copy16_async(smem_u32(&sh.upcoming[full_n & 1]) + 16 * lane, reinterpret_cast<const uint4*>(a.plan + g.number + a.abreast) + lane,
                     true);
      copy_async_commit();
    }
    for (uint32_t i = g.from; i < g.to; ++i, ++it) {
      const uint32_t p = i * kSpan + mine;
      const bool gone = __ldcg(off + p) != 0.0f;
      ok = ok && wait(&sh.s_full[it & 1], it >> 1 & 1);
      if (!__all_sync(0xffffffffu, ok)) return false;
      tc_fence_after();
      const uint32_t scores = lanes + 256 + (it & 1) * kTileColumns + quarter * 32;
      const bool edge = __any_sync(0xffffffffu, gone) || (i + 1) * kSpan > least;
      // sixteen columns at a time, `x` times `scale` their logits
      auto logits = [&](uint32_t h, float* x) -> float {
        tmem_ld16(scores + 16 * h, x);
        tmem_ld_wait();
        if (!edge) return a.scale;
#pragma unroll
        for (uint32_t c = 0; c < 16; c += 4) {
          const uint4 see = *reinterpret_cast<const uint4*>(&sh.seen[quarter][16 * h + c]);
          x[c] = p < see.x ? x[c] * a.scale : -INFINITY;
          x[c + 1] = p < see.y ? x[c + 1] * a.scale : -INFINITY;
          x[c + 2] = p < see.z ? x[c + 2] * a.scale : -INFINITY;
          x[c + 3] = p < see.w ? x[c + 3] * a.scale : -INFINITY;
        }
        if (gone) {
#pragma unroll
          for (uint32_t c = 0; c < 16; ++c) x[c] = -INFINITY;
        }
        return 1.0f;
      };
      if (max_only) {
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
          float x[16];
          const float scale = logits(h, x);
#pragma unroll
          for (uint32_t c = 0; c < 16; ++c) sum[16 * h + c] = fmaxf(sum[16 * h + c], x[c] * scale);
        }
        tc_fence_before();
        arrive0(&sh.s_empty[it & 1]);
        continue;
      }
      if (first && i == g.from) {
        float best = -INFINITY;
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
          float x[16];
          const float scale = logits(h, x);
#pragma unroll
          for (uint32_t c = 0; c < 16; ++c) {
            float m;
            asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x[c] * scale));
            if (lane == 16 * h + c) best = m;
          }
        }
        best = meet(best);
        if (!__all_sync(0xffffffffu, ok)) return false;
        const bool unset = !(fabsf(best) < INFINITY);
        sh.ref[quarter][lane] = reference(best) + kRoom;
        flagged = __any_sync(0xffffffffu, unset && real && sees > (i + 1) * kSpan);
        __syncwarp();
      }
      // The weights are rounded to bf16 for the second product (half a step is
      // 2^-8 of a weight); their sum takes them before that, in fp32.  Two
      // values an instruction: the MMAs' and the copies' threads have to find
      // room between the workers' instructions.
      uint32_t w[16];
      float most = -INFINITY;
#pragma unroll
      for (uint32_t h = 0; h < 2; ++h) {
        float x[16];
        const float scale = logits(h, x);
        if (h == 1) {
          tc_fence_before();
          arrive0(&sh.s_empty[it & 1]);
        }
#pragma unroll
        for (uint32_t c = 0; c < 16; c += 4) {
          const float4 ref = *reinterpret_cast<const float4*>(&sh.ref[quarter][16 * h + c]);
          fma_two(x[c], x[c + 1], scale, -ref.x, -ref.y);
          fma_two(x[c + 2], x[c + 3], scale, -ref.z, -ref.w);
          most = max_three(max_three(most, x[c], x[c + 1]), x[c + 2], x[c + 3]);
        }
#pragma unroll
        for (uint32_t c = 0; c < 16; c += 2) {
          const float u = exp2_approx(x[c]), v = exp2_approx(x[c + 1]);
          add_two(sum[16 * h + c], sum[16 * h + c + 1], u, v);
          w[8 * h + c / 2] = bf16_pair(u, v);
        }
      }
      flagged |= most > a.far;
      if (pv > 0) ok = ok && wait(&sh.p_empty, (pv - 1) & 1);
      if (!__all_sync(0xffffffffu, ok)) return false;
      const bool own = quarter >> 1 == rank;             // this CTA's columns, or the other's
      const uint32_t dst = own ? probs + rank * kHalfBytes : gift;
#pragma unroll
      for (uint32_t c = 0; c < 4; ++c)
        sts16(dst + swizzled(quad * 32 + lane, (quarter & 1) * 4 + c),
              make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]));
      fence_proxy_async_smem();
      __syncwarp();
      if (own) {
        if (lane == 0) cluster_mbar_arrive_own(dsmem_addr(&sh.p_full, 0));
      } else {
        if (lane == 0) mbar_arrive(&sh.ready[kGift]);
        if (warp % 8 == 0) {                             // the first of the eight warps with the other's columns
          ok = ok && wait(&sh.ready[kGift], pv & 1);
          if (!__all_sync(0xffffffffu, ok)) return false;
          if (lane == 0) send(kGift, probs + rank * kHalfBytes, gift, kHalfBytes);
        }
      }
      ++pv;
    }
    if (max_only) {
      float best = -INFINITY;
#pragma unroll
      for (uint32_t c = 0; c < 32; ++c) {
        float m;
        asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(sum[c]));
        if (lane == c) best = m;
      }
      best = meet(best);
      sh.ref[quarter][lane] = reference(best);
      __syncwarp();
      return __all_sync(0xffffffffu, ok);
    }

    // the sums of both CTAs' positions, and whether the segment stands
    add_lanes<32, 16>(sum, lane);
    flagged = first && __any_sync(0xffffffffu, flagged);
    sh.sums[rank].of[quarter][quad][lane] = sum[0];
    if (lane == 0) sh.sums[rank].again[warp] = flagged;
    const float ref = sh.ref[quarter][lane];
    if (warp == 0) copy_async_wait<0>();
    ok = ok && trade(kSum, full_n, &sh.sums[rank], sizeof(Sums));
    upcoming_number = g.number + a.abreast;
    ++full_n;
    if (!__all_sync(0xffffffffu, ok)) return false;
    const bool again = __any_sync(0xffffffffu, ((volatile uint32_t*)sh.sums[lane >> 4].again)[lane & 15] != 0);
    float total = 0.0f;
    for (uint32_t r = 0; r < 2; ++r)
      for (uint32_t q = 0; q < 4; ++q) total += ((volatile float*)sh.sums[r].of[quarter][q])[lane];
    const uint32_t slot = g.slot(pair);
    ok = ok && wait(&sh.p_empty, (pv - 1) & 1);
    if (!__all_sync(0xffffffffu, ok)) return false;
    tc_fence_after();
    if (again) {
      if (tid == 0) {
        a.again[g.note(a, pair)] = 1;                 // (both CTAs write it)
        sh.redo = 1;
      }
    } else {
      // (the room taken off the sum again before its logarithm)
      const float up = total < 1.0f ? kRoom : 0.0f;
      const float lse2 = total == 0.0f ? -INFINITY : ref - up + log2f(total * (up ? 0x1p32f : 1.0f));
      if (quad == 0 && rank == 0) {
        if (!g.whole)
          a.part_lse[slot * kTileColumns + quarter * 32 + lane] = lse2;
        else if (real && a.lse)
          a.lse[(int64_t)g.tile.first * a.heads + at] = lse2 * 0.6931471805599453f;
      }
      const float inv = total == 0.0f ? 0.0f : 1.0f / total;
      const uint32_t there = __ballot_sync(0xffffffffu, real), columns = __popc(there);
      const uint32_t first_at = __shfl_sync(0xffffffffu, at, 0);
      // sixteen columns of 128 values at a time (in one run the columns' results follow each other)
      const int64_t row0 = g.whole ? (int64_t)g.tile.first * a.heads + (a.columns.flat ? first_at : 0)
                                   : (int64_t)slot * kTileColumns + quarter * 32;
      sh.ref[quarter][lane] = inv;
      __syncwarp();
#pragma unroll 1
      for (uint32_t part = 0; part < 4; ++part) {
        const uint32_t c0 = part % 2 * 16, half = part / 2;
        float o[16];
        tmem_ld16(lanes + half * kTileColumns + quarter * 32 + c0, o);
        tmem_ld_wait();
#pragma unroll
        for (uint32_t c = 0; c < 16; c += 4) {
          const float4 by = *reinterpret_cast<const float4*>(&sh.ref[quarter][c0 + c]);
          o[c] *= by.x;
          o[c + 1] *= by.y;
          o[c + 2] *= by.z;
          o[c + 3] *= by.w;
        }
        const int64_t d = row0 * KVO_LATENT_BYTES + half * 256 + rank * 128 + quad * 32 + lane;
        if (!g.whole) {
          float* const out = a.part + d + c0 * KVO_LATENT_BYTES;
#pragma unroll
          for (uint32_t c = 0; c < 16; ++c) out[c * KVO_LATENT_BYTES] = o[c];
        } else if (a.columns.flat) {
          __nv_bfloat16* const out = reinterpret_cast<__nv_bfloat16*>(a.out) + d + c0 * KVO_LATENT_BYTES;
          if (columns == 32) {
#pragma unroll
            for (uint32_t c = 0; c < 16; ++c) out[c * KVO_LATENT_BYTES] = __float2bfloat16_rn(o[c]);
          } else {
#pragma unroll
            for (uint32_t c = 0; c < 16; ++c)
              if (c0 + c < columns) out[c * KVO_LATENT_BYTES] = __float2bfloat16_rn(o[c]);
          }
        } else {
#pragma unroll
          for (uint32_t c = 0; c < 16; ++c) {
            const uint32_t to = __shfl_sync(0xffffffffu, at, c0 + c);
            if (there >> (c0 + c) & 1)
              reinterpret_cast<__nv_bfloat16*>(a.out)[d + (int64_t)to * KVO_LATENT_BYTES] = __float2bfloat16_rn(o[c]);
          }
        }
      }
    }
    tc_fence_before();
    arrive0(&sh.o_empty);
    return true;
  };

  // All segments, then those that need another pass: their columns' maxima,
  // and the whole of it with them.  (A loop for each role, so that none keeps
  // the others' values.)
  auto rounds = [&](auto&& tile_at, auto&& work) {
    for (uint32_t round = 0; round < 2; ++round) {
      for_segments(a, begin, end, tile0, tile_at, [&](const Segment& g) -> bool {
        if (round && !__ldcg(a.again + g.note(a, pair))) return true;
        for (uint32_t pass = round ? 0 : 1; pass < 2; ++pass)
          if (!work(g, pass == 0, !round)) return false;
        return true;
      });
      ok = __all_sync(0xffffffffu, ok);
      __threadfence();
      __syncthreads();
      cluster_sync();
      // the same answer in both CTAs: nothing changes between the barriers
      uint32_t redo = 0, gave_up = 0;
      for (uint32_t r = 0; r < 2; ++r) {
        redo |= dsmem_ld_u32(dsmem_addr(&sh.redo, r));
        gave_up |= dsmem_ld_u32(dsmem_addr(&sh.gave_up, r));
      }
      __syncthreads();
      cluster_sync();
      if (!redo || gave_up) break;
    }
  };
  // most warps ask for a tile of the plan while they work on the one before
  PlanTile next;
  uint32_t next_number = UINT32_MAX;
  auto ahead = [&](uint32_t i) {
    const PlanTile t = i == next_number ? next : plan_tile(a, i);
    next = plan_tile(a, i + a.abreast);
    next_number = i + a.abreast;
    return t;
  };
  if (warp < kWorkers) {
    rounds([&](uint32_t i) { return i == upcoming_number ? sh.upcoming[(full_n - 1) & 1] : plan_tile(a, i); }, soften);
    copy_async_wait<0>();
    if (lane == 0) {
      if (warp % 8 == 0 && (warp >> 3) != rank) dsmem_st_u32(dsmem_addr(&sh.sent[kGift], other), sent[kGift]);
      if (warp == 0) {
        dsmem_st_u32(dsmem_addr(&sh.sent[kTop], other), sent[kTop]);
        dsmem_st_u32(dsmem_addr(&sh.sent[kSum], other), sent[kSum]);
      }
    }
  } else if (warp >= kLoader) {
    rounds(ahead, [&](const Segment& g, bool max_only, bool) { return load(g, max_only); });
    if (lane == 0) {
      // no slot's release may still be on its way when the CTA ends
      for (uint32_t m = n > kSlots ? n - kSlots : 0; ok && m < n; ++m) ok = wait(&sh.empty[m % kSlots], m / kSlots & 1);
      if (ok && q_n) wait(&sh.q_empty, (q_n - 1) & 1);
      dsmem_st_u32(dsmem_addr(&sh.issued[rank][load_warp], 0), n);
      dsmem_st_u32(dsmem_addr(&sh.q_issued[rank][load_warp], 0), q_n);
    }
  } else if (rank == 0) {
    rounds(ahead, [&](const Segment& g, bool max_only, bool) { return multiply(g, max_only); });
  } else {
    rounds(ahead, [&](const Segment& g, bool max_only, bool) { return pass_on(g, max_only); });
  }
  // Both CTAs end together.  Where a wait gave up in either, what is in flight
  // finishes first: the MMAs, then the copies; those that a CTA has not started
  // count as come.
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  const uint32_t other_gave_up = dsmem_ld_u32(dsmem_addr(&sh.gave_up, other));
  if (sh.gave_up | other_gave_up) {
    if (tid == 0) atomicOr(a.status, kFlagTimeout);
    if (rank == 0 && warp == kMma && elect_one()) {
      pair_commit(&sh.drained, 1);
      if (!landed(&sh.drained, 0)) atomicOr(a.status, kFlagInflight);
    }
    if (tid == 0) {
      const uint32_t bytes[kLetters] = {kHalfBytes, sizeof(sh.top[0]), sizeof(Sums)};
      for (uint32_t i = 0; i < kLetters; ++i) {
        if (sh.armed[i] < sh.sent[i]) mbar_arrive_expect_tx(&sh.come[i], bytes[i]);   // one at most
        if (sh.sent[i] && !landed(&sh.come[i], (sh.sent[i] - 1) & 1)) atomicOr(a.status, kFlagInflight);
      }
    }
    if (rank == 0 && warp == kLoader && lane == 0) {
      uint32_t most = 0, least = UINT32_MAX, queried = 0;
      for (uint32_t r = 0; r < 2; ++r)
        for (uint32_t w = 0; w < kLoaders; ++w) {
          most = max(most, sh.issued[r][w]);
          least = min(least, sh.issued[r][w]);
          queried = max(queried, sh.q_issued[r][w]);
        }
      // (whoever starts a copy has seen the one before it in its slot used up)
      auto started = [&](uint32_t m) { return m < sh.issued[0][m % kLoaders] || m < sh.issued[1][m % kLoaders]; };
      for (uint32_t m = least; m < most; ++m) {
        uint64_t* const bar = &sh.full[m % kSlots];
        if (!started(m)) continue;
        if (m >= sh.issued[0][m % kLoaders]) mbar_arrive_expect_tx(bar, 2 * kSlotBytes);
        for (uint32_t r = 0; r < 2; ++r)
          if (m >= sh.issued[r][m % kLoaders]) mbar_complete_tx(bar, kSlotBytes);
      }
      for (uint32_t m = most > kSlots ? most - kSlots : 0; m < most; ++m)
        if (started(m) && !landed(&sh.full[m % kSlots], m / kSlots & 1)) atomicOr(a.status, kFlagInflight);
      if (queried) {
        if (sh.q_issued[0][0] < queried) mbar_arrive_expect_tx(&sh.q_full, 2 * 9 * box);
        for (uint32_t r = 0; r < 2; ++r)
          for (uint32_t w = 0; w < kLoaders; ++w)
            if (sh.q_issued[r][w] < queried) mbar_complete_tx(&sh.q_full, 9 / kLoaders * box);
        if (!landed(&sh.q_full, (queried - 1) & 1)) atomicOr(a.status, kFlagInflight);
      }
    }
    __syncthreads();
  }
  cluster_sync();
  if (warp == kMma) pair_tmem_free(tmem, 512);
}

// Joins the parts of a cut tile by their log-sum-exps: blocks ((g - 1) * abreast
// + k, ..) those of the k-th tile that share g is the first to cut, four columns of
// 128 threads each.
constexpr uint32_t kJoinColumns = 4, kMostParts = 96;

__global__ void __launch_bounds__(128 * kJoinColumns) join_parts_kernel(const __grid_constant__ ChunkArgs a) {
  const uint32_t g = blockIdx.x / a.abreast + 1, beside = blockIdx.x % a.abreast, d = threadIdx.x & 127, lane = threadIdx.x & 31;
  const uint32_t column = blockIdx.y * kJoinColumns + (threadIdx.x >> 7);
  wait_previous_grid();
  if (g >= Shares(a).count) return;
  const uint32_t last = __ldcg(&a.cuts[g * a.abreast + beside].last);
  if (last == 0) return;
  const uint4 *const cut = reinterpret_cast<const uint4*>(a.cuts + g * a.abreast + beside), x = __ldcg(cut), y = __ldcg(cut + 1);
  const PlanTile t = plan_tile(x, y);
  uint32_t where;
  const uint32_t token = column_at(a, t, 2 * t.index + column / kColumns, column % kColumns, &where);
  if (token >= t.tokens) return;                         // (the same for a column's warps)
  const uint32_t parts = last - g + 2;
  auto row_of = [&](uint32_t i) { return (2 * ((g - 1 + i) * a.abreast + beside) + (i == 0)) * kTileColumns + column; };
  // lane l has the weights of parts l, l + 32 and l + 64
  float l[kMostParts / 32], top = -INFINITY;
#pragma unroll
  for (uint32_t k = 0; k < kMostParts / 32; ++k) {
    l[k] = lane + 32 * k < parts ? __ldcg(a.part_lse + row_of(lane + 32 * k)) : -INFINITY;
    top = fmaxf(top, l[k]);
  }
#pragma unroll
  for (uint32_t e = 16; e; e >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, e));
  const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
  for (uint32_t k = 0; k < kMostParts / 32; ++k) l[k] = exp2f(l[k] - base);
  float total = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (uint32_t i = 0; i < parts; ++i) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part + (int64_t)row_of(i) * KVO_LATENT_BYTES) + d);
    const float w = __shfl_sync(0xffffffffu, i < 32 ? l[0] : i < 64 ? l[1] : l[2], i & 31);
    if (!(w > 0.0f) && !isnan(w)) continue;
    total += w;
    o.x = fmaf(w, v.x, o.x);
    o.y = fmaf(w, v.y, o.y);
    o.z = fmaf(w, v.z, o.z);
    o.w = fmaf(w, v.w, o.w);
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  const int64_t row = (int64_t)t.first * a.heads + where;
  reinterpret_cast<uint2*>(a.out + row * KVO_LATENT_BYTES)[d] =
      make_uint2(bf16_pair(o.x * inv, o.y * inv), bf16_pair(o.z * inv, o.w * inv));
  if (a.lse && d == 0) a.lse[row] = total == 0.0f ? -INFINITY : (base + log2f(total)) * 0.6931471805599453f;
}

// ------------------------------------------------------------------ the host
// Sequences are taken in groups whose unpacked rows fit into 4 GiB of scratch,
// one group after the other, however many there are and however long `rows`
// says they may be.  No group: a single one's do not fit.
constexpr int64_t kMostValueBytes = (int64_t)4 << 30;
static_assert(kMostValueBytes / kValueBytes / kSpan < 1 << 16, "PlanTile counts tiles of positions in 16 bits");

struct Groups {
  int64_t span, count, each;         // positions of a sequence; groups; sequences of a group
  Groups(int64_t sequences, int64_t rows) {
    span = ((rows > 0 ? rows : 1) + kSpan - 1) / kSpan * kSpan;
    const int64_t most = kMostValueBytes / (span * kValueBytes);
    count = most ? (sequences + most - 1) / most : 0;
    each = count ? (sequences + count - 1) / count : 0;
  }
};

// Whether unpacking the rows pays.  Per 1,000 rows of a sequence the kernel for
// few columns takes about 0.29 us for every 64 columns, this one 0.20 us for
// every 128 and 0.45 us to unpack them, and about 21 us more a group.  Both
// ways, us: 16 sequences of 8,192 rows with 128 columns each 91 and 114, with
// 256 168 and 141; 64 of 4,096 with 128 164 and 195, with 256 324 and 255; one of
// 50,000 rows with 256 66 and 73, with 384 89 and 78, with 1,024 221 and 116; 1,024
// columns over 4,000 rows 32 and 43; 2,048 over 4,000 51 and 48; 4,096 over 2,000 52
// and 49, over 1,000 34 and 45; 16,384 over 500 52 and 57.
bool many_columns(int64_t tokens, int64_t sequences, uint32_t heads, int64_t rows) {
  const int64_t busy = sequences < tokens ? sequences : tokens;
  const Groups groups(sequences, rows);
  if (!groups.count) return false;
  const int64_t columns = (tokens * heads + busy - 1) / busy, each = (tokens + busy - 1) / busy;
  const int64_t seen = rows - std::min(each, rows) / 2;  // of the middle token
  const int64_t gain = 29 * ((columns + 63) / 64) - 20 * ((columns + 127) / 128) - 45;
  return gain > 0 && (double)busy * (double)seen * (double)gain > 2.1e6 * (double)groups.count;
}

// Pairs that go over the same positions side by side, as the tiles of columns of
// a sequence allow: the first to take a piece brings it into L2 for all of them.
// One, two and four, us: 8 sequences of 131,072 rows with 1,024 columns each 2,255,
// 1,944 and 1,870; 64 of 8,192 with 1,024 1,188, 1,032 and 986; 32 of 65,536 with 256
// 1,673, 1,510 and 1,514; one of 100,000 with 32,768 4,666, 4,629 and 4,560; a prompt's
// 4,096 tokens of 16 heads 248, 248 and 247.  A row's pairs wait for the longest of
// its tiles, so no more than a sequence of average size fills.
uint32_t abreast_of(int64_t tokens, int64_t sequences, uint32_t heads) {
  const int64_t busy = sequences < tokens ? sequences : tokens, tiles = tokens * heads / (busy * kTileColumns);
  return tiles >= 4 ? 4 : tiles >= 2 ? 2 : 1;
}
static_assert(kMostAbreast >= 4 && kUnpackThreads % kMostAbreast == 0);

struct Layout {              // of the scratch
  int64_t tiles, pairs;
  int64_t values, off, plan, cuts, again, part, part_lse, bytes;
};

Layout layout_of(int64_t tokens, int64_t sequences, uint32_t heads, int64_t rows) {
  Layout l;
  const Groups groups(sequences, rows);
  l.pairs = std::min(device_sms() / 2, (int)kMostParts);
  // Tiles of either way to fill them: at worst 33 heads of one token a half.
  const int64_t busy = sequences < tokens ? sequences : tokens;
  const int64_t deep = heads < kColumns ? kColumns / heads : 1, across = heads > kColumns ? 2 : 1;
  const int64_t halves = (tokens + busy * (deep - 1)) / deep * across;
  const int64_t flat = (tokens * heads + busy * (kColumns - 1)) / kColumns;
  l.tiles = ((halves > flat ? halves : flat) + busy + 1) / 2 + (sequences + kUnpackThreads - 1) / kUnpackThreads * (kMostAbreast - 1);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t from = at;
    at += (bytes + 255) / 256 * 256;
    return from;
  };
  l.values = take(groups.each * groups.span * kValueBytes);
  l.off = take(groups.each * groups.span * 4);
  l.plan = take((l.tiles + 2) * (int64_t)sizeof(PlanTile));
  l.cuts = take(l.pairs * (int64_t)sizeof(Cut));
  l.again = take(l.tiles + 2 * l.pairs);
  l.part = take(2 * l.pairs * kTileColumns * KVO_LATENT_BYTES * 4);
  l.part_lse = take(2 * l.pairs * kTileColumns * 4);
  l.bytes = at;
  return l;
}

cudaError_t launch_chunk(ChunkArgs a, const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                         cudaStream_t stream) {
  static int room[64] = {};                              // pairs that run at the same time
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  lc.gridDim = dim3(2);
  lc.blockDim = dim3(kChunkThreads);
  lc.dynamicSmemBytes = kChunkSmem;
  lc.stream = stream;
  lc.attrs = attr;
  lc.numAttrs = 1;
  if (!room[dev & 63]) {
    e = cudaFuncSetAttribute(chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kChunkSmem);
    if (e != cudaSuccess) return e;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, chunk_kernel, &lc);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    room[dev & 63] = n;
  }
  if (a.pairs > (uint32_t)room[dev & 63]) a.pairs = (uint32_t)room[dev & 63];
  if (a.pairs < a.abreast) a.abreast = 1;
  a.pairs -= a.pairs % a.abreast;
  e = launch_early(unpack_kernel, dim3(1 + a.unpack_blocks * a.cache.sequences), kUnpackThreads, 0, stream, a);
  if (e != cudaSuccess) return e;
  lc.gridDim = dim3(2 * a.pairs);
  lc.numAttrs = 2;
  e = cudaLaunchKernelEx(&lc, chunk_kernel, a, qmap, kmap, vmap);
  if (e != cudaSuccess || a.pairs <= a.abreast) return e;
  return launch_early(join_parts_kernel, dim3(a.pairs - a.abreast, kTileColumns / kJoinColumns), 128 * kJoinColumns, 0,
                      stream, a);
}

}  // namespace
}  // namespace kvo

extern "C" int64_t kvo_attend_chunk_work_bytes(int64_t tokens, int32_t sequences, int32_t heads, int64_t rows) {
  using namespace kvo;
  if (tokens < 0 || tokens > KVO_MAX_QUERIES || sequences < 1 || sequences > KVO_MAX_QUERIES) return -1;
  if (heads < 1 || heads > KVO_MAX_HEADS || rows < 0 || rows > INT32_MAX - 255) return -1;
  if (tokens == 0) return 0;
  return many_columns(tokens, sequences, (uint32_t)heads, rows) ? layout_of(tokens, sequences, (uint32_t)heads, rows).bytes
                                                                : few_columns_work(tokens, sequences, (uint32_t)heads, rows);
}

extern "C" kvo_status kvo_attend_chunk(kvo_ctx* ctx, const kvo_cache* cache, const kvo_chunk_query* s, void* stream) {
  using namespace kvo;
  uint32_t* status = nullptr;
  if (!ctx || !cache_ok(cache) || !s || !cache_rows_ok(cache)) return KVO_EINVAL;
  const int64_t need = kvo_attend_chunk_work_bytes(s->tokens, cache->sequences, s->heads, s->rows);
  if (need < 0 || !s->starts || !s->lens || !std::isfinite(s->scale)) return KVO_EINVAL;
  if (!aligned(s->starts, 4) || !aligned(s->lens, 4)) return KVO_EINVAL;
  if (s->tokens > 0) {
    if (!s->q || !s->out || s->work_bytes < need || (need && !s->work)) return KVO_EINVAL;
    if (!query_ok(s->q, s->q_ld, s->q_head_ld, s->tokens, s->heads) || !aligned(s->out, 16)) return KVO_EINVAL;
    if (!aligned(s->lse, 4) || !aligned(s->work, 16)) return KVO_EINVAL;
  }
  int64_t wait_clocks = 0;
  const kvo_status st = usable_status(ctx, &status, &wait_clocks);
  if (st != KVO_OK) return st;
  if (s->tokens == 0) return KVO_OK;
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  if (!many_columns(s->tokens, cache->sequences, (uint32_t)s->heads, s->rows))
    return launch_few_columns(*cache, *s, status, wait_clocks, on) == cudaSuccess ? KVO_OK : KVO_ECUDA;

  const Groups groups(cache->sequences, s->rows);
  const Layout l = layout_of(s->tokens, cache->sequences, (uint32_t)s->heads, s->rows);
  uint8_t* const work = static_cast<uint8_t*>(s->work);
  ChunkArgs a = {};
  a.out = s->out;
  a.lse = s->lse;
  a.values = work + l.values;
  a.off = reinterpret_cast<float*>(work + l.off);
  a.plan = reinterpret_cast<PlanTile*>(work + l.plan);
  a.cuts = reinterpret_cast<Cut*>(work + l.cuts);
  a.again = work + l.again;
  a.part = reinterpret_cast<float*>(work + l.part);
  a.part_lse = reinterpret_cast<float*>(work + l.part_lse);
  a.status = status;
  a.rows = (uint32_t)s->rows;
  a.span = (uint32_t)groups.span;
  a.tokens = (uint32_t)s->tokens;
  a.heads = (uint32_t)s->heads;
  a.most_tiles = (uint32_t)l.tiles;
  a.pairs = (uint32_t)l.pairs;
  a.abreast = abreast_of(s->tokens, cache->sequences, (uint32_t)s->heads);
  a.unpack_blocks = (uint32_t)(groups.span / kUnpackRows);
  a.by_heads = divider(a.heads);
  a.scale = s->scale * kLog2e;
  // sums of weights up to 2^far over all rows, times latents below 2^23, stay below 2^126
  a.far = 103.0f - std::ceil(std::log2((float)(s->rows > 1 ? s->rows : 1)));
  a.wait_clocks = wait_clocks;
  // a dimension of one has no next element: its stride says nothing
  const int64_t head_ld = a.heads > 1 ? s->q_head_ld : KVO_DEQUANT_VALUES;
  const int64_t q_ld = s->tokens > 1 ? s->q_ld : a.heads * head_ld;
  a.columns = columns_of(a.heads, q_ld, head_ld, s->tokens);
  CUtensorMap qmap, kmap, vmap;
  if (!query_map(&qmap, s->q, a.heads, s->tokens, q_ld * 2, head_ld * 2, a.columns) ||
      !value_map(&kmap, a.values, groups.each * groups.span, kSpan / 2, 1) ||
      !value_map(&vmap, a.values, groups.each * groups.span, 64, 2))
    return KVO_ECUDA;
  for (int64_t first = 0; first < cache->sequences; first += groups.each) {
    kvo_cache part = *cache;
    part.sequences = (int32_t)std::min(groups.each, cache->sequences - first);
    if (part.table) {
      part.table += first * part.table_ld;
    } else {                                             // sequence s is block s
      part.rows = static_cast<uint8_t*>(part.rows) + first * part.block_rows * KVO_ROW_BYTES;
      part.blocks -= first;
    }
    a.cache = cache_view(part);
    a.starts = s->starts + first;
    a.lens = s->lens + first;
    if (launch_chunk(a, qmap, kmap, vmap, on) != cudaSuccess) return KVO_ECUDA;
  }
  return KVO_OK;
}
