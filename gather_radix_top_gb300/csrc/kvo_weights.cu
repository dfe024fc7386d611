// kvo_attention_weights: the attention weight that a chunk's tokens give to
// every cached position, summed over tokens and heads:
//     w_p = keep * carry_p + sum_c exp(scale * k_p . q_c - lse_c)
// over the (token, head) columns c whose token sees position p.
//
// Two CTAs of a cluster hold 128 positions each, dequantised once, and walk
// over the columns in tiles of 128: S [256 positions x 128 columns] = K Q^T as
// pair MMAs, for which each CTA brings half of a tile's queries.  A position is
// a lane of S, so its sum over the columns stays in one thread's register.
// Shared memory holds the positions (144 KB) and a ring of nine pieces of 64
// columns by 64 values; tensor memory four tiles of S.
//
// A thread's sum over a tile is added to its running sum with the rounding
// error carried along, so that many tokens lose nothing.
//
// Where a call's positions do not fill the GPU, the columns are split over
// several pairs, whose sums a second launch adds in their order.
#include "kvo_cache.cuh"
#include "kvo_chunk.cuh"
#include "kvo_rows.cuh"
#include "kvo_tc.cuh"

namespace kvo {
namespace {

constexpr uint32_t kTile = 128;                          // positions of a CTA
constexpr uint32_t kTileColumns = 2 * kColumns;          // of a pair
constexpr uint32_t kWorkers = 16;                        // warps: four for each quarter of the columns
constexpr uint32_t kMma = kWorkers, kLoader = kWorkers + 1;
constexpr uint32_t kWeightThreads = (kLoader + 1) * 32;
constexpr uint32_t kPieceBytes = kTile * 128;            // 64 values of every position
constexpr uint32_t kSlotBytes = kColumns * 128;          // 64 values of a CTA's columns
constexpr uint32_t kSlots = 9, kAhead = 4;               // ring of slots, tiles of S
constexpr uint32_t kWeightSmem = 1024 + 9 * kPieceBytes + kSlots * kSlotBytes;
constexpr uint32_t kPairGrid = 2 * kTile;                // positions of a pair

struct WeightArgs {
  CacheView cache;
  const int32_t* starts;
  const int32_t* lens;
  const float* lse;
  const float* carry;        // or NULL
  float* out;
  float* part;               // [splits][sequences][rows], with several splits
  uint32_t* status;
  int64_t carry_ld, out_ld;
  uint32_t rows, tokens, heads, window, splits;
  Divider by_heads;
  Columns columns;
  float scale;               // times log2(e)
  float keep;
  int64_t wait_clocks;
};

struct WeightShared {
  uint64_t k_full, full[kSlots], empty[kSlots], s_full[kAhead], s_empty[kAhead], drained;
  uint32_t tmem, gave_up;
  uint32_t issued[2];                // slots that each CTA's loader has filled
  float lse[kWorkers][32];           // per warp and column, base 2
  int32_t seen[kWorkers][32];        // and the positions it sees
  float sums[4][kTile];
};

// The columns of one sequence and the tiles of them that a CTA pair takes.
struct Run {
  uint32_t first, tokens;            // of the sequence
  int32_t before;                    // token i sees the first before + i positions
  uint32_t from;                     // the first token that counts
  uint32_t begin, end;               // tiles of 128 columns
};

__device__ __forceinline__ void run_of(const WeightArgs& a, uint32_t s, uint32_t p0, uint32_t split, Run* r) {
  const int32_t b = a.starts[s], e = a.starts[s + 1], T = (int32_t)a.tokens;
  if (b < 0 || b > T || e < b || e > T) atomicOr(a.status, kFlagRange);
  r->first = (uint32_t)min(max(b, 0), T);
  r->tokens = (uint32_t)min(max(e, (int32_t)r->first), T) - r->first;
  const int32_t n = (int32_t)r->tokens;
  r->before = min(max(a.lens[s], 0), INT32_MAX - 1) - n + 1;
  const int32_t sees = max((int32_t)p0 - r->before + 1, 0);   // the first token that sees position p0
  r->from = (uint32_t)max(a.window && a.window < r->tokens ? n - (int32_t)a.window : 0, sees);
  const Columns& c = a.columns;
  const uint32_t units = c.flat ? r->tokens * a.heads : r->tokens, skip = c.flat ? r->from * a.heads : r->from;
  const uint32_t halves = (units + c.deep - 1) / c.deep * c.across;
  const uint32_t t0 = r->from < r->tokens ? skip / c.deep * c.across / 2 : 0;
  const uint32_t t1 = r->from < r->tokens ? (halves + 1) / 2 : 0;
  const uint32_t share = (t1 - t0 + a.splits - 1) / a.splits;
  r->begin = min(t0 + split * share, t1);
  r->end = min(r->begin + share, t1);
}

__global__ void __launch_bounds__(kWeightThreads, 1)
    weights_kernel(const __grid_constant__ WeightArgs a, const __grid_constant__ CUtensorMap qmap) {
  extern __shared__ uint8_t raw[];
  __shared__ WeightShared sh;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = cluster_rank();
  const uint32_t s = blockIdx.y, split = (blockIdx.x >> 1) % a.splits;
  const uint32_t pair0 = (blockIdx.x >> 1) / a.splits * kPairGrid, p0 = pair0 + rank * kTile;
  const uint32_t keys = (smem_u32(raw) + 1023u) & ~1023u, ring = keys + 9 * kPieceBytes;

  wait_previous_grid();
  allow_next_grid();
  const uint32_t len = (uint32_t)min(max(a.lens[s], 0), (int32_t)a.rows);
  float* const part = a.part + ((int64_t)split * a.cache.sequences + s) * a.rows;
  Run run;
  run_of(a, s, pair0, split, &run);
  if (pair0 >= len || run.begin == run.end) {            // the same in both CTAs
    const uint32_t p = p0 + tid;
    if (tid < kTile && p < a.rows) {
      if (a.splits > 1)
        part[p] = 0.0f;
      else
        a.out[s * a.out_ld + p] = p < len && a.carry ? a.keep * a.carry[s * a.carry_ld + p] : 0.0f;
    }
    return;
  }

  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return wait_or_give_up(bar, parity, &sh.gave_up, a.wait_clocks);
  };
  if (tid == 0) {
    mbar_init(&sh.k_full, 2 * kWorkers);
    for (uint32_t i = 0; i < kSlots; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (uint32_t i = 0; i < kAhead; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_empty[i], 2 * kWorkers);
    }
    mbar_init(&sh.drained, 1);
    sh.gave_up = a.wait_clocks == 0;
    sh.issued[0] = sh.issued[1] = 0;
  }
  if (warp == kMma) pair_tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const Columns& cols = a.columns;
  const uint32_t box = cols.wide * cols.deep * 128;      // bytes of a slot that a copy fills

  // Piece k of tile t's queries to their slot: the n-th of this CTA's copies.
  auto bring = [&](uint32_t n) {
    const uint32_t tile = run.begin + n / 9, piece = n % 9, slot = n % kSlots, half = 2 * tile + rank;
    if (rank == 0) mbar_arrive_expect_tx(&sh.full[slot], 2 * box);
    const uint32_t row = half / cols.across, head = half % cols.across * cols.wide;
    pair_load_box(ring + slot * kSlotBytes, &qmap, (int32_t)(piece * 64), (int32_t)head,
                  (int32_t)((cols.flat ? run.first * a.heads : run.first) + row * cols.deep), dsmem_addr(&sh.full[slot], 0));
  };

  if (warp == kLoader) {
    if (lane == 0) {
      const uint32_t all = (run.end - run.begin) * 9;
      uint32_t n = 0;
      for (; n < all; ++n) {
        if (n >= kSlots && !wait(&sh.empty[n % kSlots], (n / kSlots - 1) & 1)) break;
        bring(n);
      }
      // no slot's release may still be on its way when the CTA ends
      for (uint32_t m = all > kSlots ? all - kSlots : 0; n == all && m < all; ++m)
        if (!wait(&sh.empty[m % kSlots], m / kSlots & 1)) break;
      dsmem_st_u32(dsmem_addr(&sh.issued[rank], 0), n);  // both counts are looked at by both CTAs
      dsmem_st_u32(dsmem_addr(&sh.issued[rank], 1), n);
    }
  } else if (warp == kMma) {
    if (rank == 0) {
      constexpr uint32_t kDesc = pair_desc(1, kTileColumns, false, false);
      const uint64_t k_tile = tile_desc(keys, 16), q_ring = tile_desc(ring, 16);
      bool ok = cluster_wait_or_give_up(&sh.k_full, 0, &sh.gave_up, a.wait_clocks);
      uint32_t n = 0;
      for (uint32_t t = 0; t < run.end - run.begin && __all_sync(0xffffffffu, ok); ++t) {
        const uint32_t buf = t % kAhead;
        if (t >= kAhead) ok = wait(&sh.s_empty[buf], (t / kAhead - 1) & 1);
        tc_fence_after();
        for (uint32_t piece = 0; piece < 9; ++piece, ++n) {
          const uint32_t slot = n % kSlots;
          ok = ok && wait(&sh.full[slot], n / kSlots & 1);
          if (!__all_sync(0xffffffffu, ok)) break;
          if (elect_one()) {
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k)
              pair_mma_bf16(tmem + buf * kTileColumns, k_tile + piece * (kPieceBytes >> 4) + 2 * k,
                            q_ring + slot * (kSlotBytes >> 4) + 2 * k, kDesc, piece + k > 0);
            pair_commit(&sh.empty[slot], 3);
            if (piece == 8) pair_commit(&sh.s_full[buf], 3);
          }
          __syncwarp();
        }
      }
    }
  } else {
    // positions: piece `piece` of each 128 latent bytes of rows slot and slot + 64
    const uint32_t piece = ((lane >> 3) & 1) * 4 + (lane & 3);
    const uint32_t slot = warp * 4 + (lane >> 4) * 2 + ((lane >> 2) & 1);
    const uint32_t to_lo = keys + (piece >> 2) * kPieceBytes + swizzled(slot, 2 * (piece & 3));
    const uint32_t to_hi = keys + (piece >> 2) * kPieceBytes + swizzled(slot, 2 * (piece & 3) + 1);
    const uint32_t to_rope = keys + 8 * kPieceBytes + swizzled(slot, piece);
    uint4 lat[2][4], rope[2], eight[2];
#pragma unroll
    for (uint32_t u = 0; u < 2; ++u) {
      const uint32_t p = p0 + slot + 64 * u;
      const int64_t row = p < len ? cache_row(a.cache, s, p) : -1;
      const uint4* from = reinterpret_cast<const uint4*>(a.cache.rows) + row * (KVO_ROW_BYTES / 16);
      const uint4 none = make_uint4(0, 0, 0, 0);
      for (uint32_t k = 0; k < 4; ++k) lat[u][k] = row >= 0 ? __ldg(from + 8 * k + piece) : none;
      eight[u] = row >= 0 ? __ldg(from + KVO_LATENT_BYTES / 16) : none;
      rope[u] = row >= 0 ? __ldg(from + KVO_LATENT_BYTES / 16 + 1 + piece) : none;
    }
#pragma unroll
    for (uint32_t u = 0; u < 2; ++u) {
      const uint32_t pick = piece >= 4 ? 0x7632u : 0x5410u;
      const uint32_t scales[2] = {__byte_perm(eight[u].x, eight[u].y, pick), __byte_perm(eight[u].z, eight[u].w, pick)};
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k) {
        const uint16_t scale = (uint16_t)(scales[k >> 1] >> (k & 1) * 16);
        const float bias = -1152.0f * __half2float(__ushort_as_half(scale));
        uint4 x, y;
        dequant4(lat[u][k].x, scale, bias, x.x, x.y);
        dequant4(lat[u][k].y, scale, bias, x.z, x.w);
        dequant4(lat[u][k].z, scale, bias, y.x, y.y);
        dequant4(lat[u][k].w, scale, bias, y.z, y.w);
        sts16(to_lo + 2 * k * kPieceBytes + u * 8192, x);
        sts16(to_hi + 2 * k * kPieceBytes + u * 8192, y);
      }
      sts16(to_rope + u * 8192, rope[u]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) cluster_mbar_arrive(dsmem_addr(&sh.k_full, 0));

    // this thread: position p0 + quad * 32 + lane against 32 columns of a tile
    const uint32_t quad = warp & 3, quarter = warp >> 2, mine = p0 + quad * 32 + lane;
    const bool there = mine < len && cache_row(a.cache, s, mine) >= 0;
    if (quarter == 0 && mine < len && !there) atomicOr(a.status, kFlagRange);
    // lane l looks up column 32 * quarter + l: its half of a tile, and where it lies in it
    const uint32_t in_half = quarter % 2 * 32 + lane, deep = divide(in_half, cols.by_wide);
    const uint32_t wide = in_half - deep * cols.wide;
    auto column = [&](uint32_t t, float* lse, int32_t* seen) {
      *lse = 0.0f;
      *seen = 0;
      if (t >= run.end || deep >= cols.deep) return;
      const uint32_t half = 2 * t + quarter / 2, row = half / cols.across * cols.deep + deep;
      const uint32_t head = half % cols.across * cols.wide + wide;
      const uint32_t at = cols.flat ? row : row * a.heads + head, token = divide(at, a.by_heads);
      if (token < run.from || token >= run.tokens || (!cols.flat && head >= a.heads)) return;
      const float l = __ldg(a.lse + (int64_t)run.first * a.heads + at);
      if (l == -INFINITY) return;
      *lse = l * kLog2e;
      *seen = min(run.before + (int32_t)token, (int32_t)len);
    };
    float total = 0.0f, lost = 0.0f, next_lse;
    int32_t next_seen;
    column(run.begin, &next_lse, &next_seen);
    const uint32_t lanes = tmem + (quad << 21) + quarter * 32, s_empty = dsmem_addr(&sh.s_empty[0], 0);
    for (uint32_t t = 0; t < run.end - run.begin; ++t) {
      const uint32_t buf = t % kAhead;
      sh.lse[warp][lane] = next_lse;
      sh.seen[warp][lane] = next_seen;
      const bool edge = __any_sync(0xffffffffu, next_seen < (int32_t)(p0 + kTile));
      column(run.begin + t + 1, &next_lse, &next_seen);
      const bool ok = wait(&sh.s_full[buf], t / kAhead & 1);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      float x[32];
      tmem_ld32(lanes + buf * kTileColumns, x);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) cluster_mbar_arrive_relaxed(s_empty + buf * 8);
      float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (uint32_t c = 0; c < 32; ++c) {
        float e = exp2_approx(fmaf(x[c], a.scale, -sh.lse[warp][c]));
        if (edge && (int32_t)mine >= sh.seen[warp][c]) e = 0.0f;
        sum[c & 3] += e;
      }
      const float add = (sum[0] + sum[1]) + (sum[2] + sum[3]) - lost, now = total + add;
      lost = (now - total) - add;
      total = now;
      __syncwarp();
    }
    sh.sums[quarter][quad * 32 + lane] = total;
    named_sync(1, kWorkers * 32);
    if (quarter == 0 && mine < a.rows) {
      total = (sh.sums[0][mine - p0] + sh.sums[1][mine - p0]) + (sh.sums[2][mine - p0] + sh.sums[3][mine - p0]);
      if (!there) total = 0.0f;
      if (a.splits > 1)
        part[mine] = total;
      else
        a.out[s * a.out_ld + mine] =
            mine < len ? (a.carry ? fmaf(a.keep, a.carry[s * a.carry_ld + mine], total) : total) : 0.0f;
    }
  }

  // Both CTAs end together: the MMAs read the other's memory, and arrivals and
  // copies go to rank 0's barriers.  Where a wait gave up in either, what is in
  // flight finishes first: the MMAs, then the copies, of which the CTA that has
  // fewer out issues the missing ones, so that every phase can end.
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  const uint32_t other_gave_up = dsmem_ld_u32(dsmem_addr(&sh.gave_up, rank ^ 1));
  if (sh.gave_up | other_gave_up) {
    if (tid == 0) atomicOr(a.status, kFlagTimeout);
    if (warp == kMma && rank == 0) {
      if (elect_one()) {
        pair_commit(&sh.drained, 1);
        if (!landed(&sh.drained, 0)) atomicOr(a.status, kFlagInflight);
      }
    }
    __syncthreads();
    cluster_sync();
    if (warp == kLoader && lane == 0) {
      const uint32_t most = max(sh.issued[0], sh.issued[1]);
      for (uint32_t n = sh.issued[rank]; n < most; ++n) bring(n);
      if (rank == 0)
        for (uint32_t n = most > kSlots ? most - kSlots : 0; n < most; ++n)
          if (!landed(&sh.full[n % kSlots], n / kSlots & 1)) atomicOr(a.status, kFlagInflight);
    }
    __syncthreads();
  }
  cluster_sync();
  if (warp == kMma) pair_tmem_free(tmem, 512);
}

__global__ void __launch_bounds__(256) add_weights_kernel(const __grid_constant__ WeightArgs a) {
  wait_previous_grid();
  allow_next_grid();
  const uint32_t p = blockIdx.x * 256 + threadIdx.x, s = blockIdx.y;
  if (p >= a.rows) return;
  float total = 0.0f;
  if ((int32_t)p < a.lens[s]) {
    for (uint32_t i = 0; i < a.splits; ++i) total += __ldcg(a.part + ((int64_t)i * a.cache.sequences + s) * a.rows + p);
    if (a.carry) total = fmaf(a.keep, a.carry[s * a.carry_ld + p], total);
  }
  a.out[s * a.out_ld + p] = total;
}

// Pairs that the columns of a sequence's positions are split over: as many as
// the GPU has room for.
uint32_t weight_splits(int64_t tokens, int64_t sequences, uint32_t heads, int64_t rows, int64_t window) {
  const int64_t pairs = (rows + kPairGrid - 1) / kPairGrid * sequences, room = device_sms() / 2;
  int64_t n = tokens / sequences + (tokens % sequences != 0);
  if (window && window < n) n = window;
  const int64_t tiles = (n * heads + kTileColumns - 1) / kTileColumns;
  int64_t splits = pairs < 1 || pairs >= room ? 1 : room / pairs;
  if (splits > tiles) splits = tiles;
  return (uint32_t)(splits < 1 ? 1 : splits);
}

cudaError_t launch_weights(const WeightArgs& a, const CUtensorMap& map, cudaStream_t stream) {
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!ready[dev & 63]) {
    e = cudaFuncSetAttribute(weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kWeightSmem);
    if (e != cudaSuccess) return e;
    ready[dev & 63] = true;
  }
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  lc.gridDim = dim3(2 * ((a.rows + kPairGrid - 1) / kPairGrid) * a.splits, a.cache.sequences);
  lc.blockDim = dim3(kWeightThreads);
  lc.dynamicSmemBytes = kWeightSmem;
  lc.stream = stream;
  lc.attrs = attr;
  lc.numAttrs = 2;
  return cudaLaunchKernelEx(&lc, weights_kernel, a, map);
}

}  // namespace
}  // namespace kvo

extern "C" int64_t kvo_attention_weights_work_bytes(int64_t tokens, int32_t sequences, int32_t heads, int64_t rows,
                                                    int64_t window) {
  if (tokens < 0 || tokens > KVO_MAX_QUERIES || sequences < 1 || sequences > KVO_MAX_QUERIES) return -1;
  if (heads < 1 || heads > KVO_MAX_HEADS || rows < 0 || rows > INT32_MAX - 255 || window < 0) return -1;
  const uint32_t splits = kvo::weight_splits(tokens, sequences, (uint32_t)heads, rows, window);
  return splits == 1 ? 0 : (int64_t)splits * sequences * rows * 4;
}

extern "C" kvo_status kvo_attention_weights(kvo_ctx* ctx, const kvo_cache* cache, const kvo_weight_query* s,
                                            void* stream) {
  using namespace kvo;
  uint32_t* status = nullptr;
  if (!ctx || !cache_ok(cache) || !s || !cache_rows_ok(cache)) return KVO_EINVAL;
  const int64_t need = kvo_attention_weights_work_bytes(s->tokens, cache->sequences, s->heads, s->rows, s->window);
  if (need < 0 || !s->starts || !s->lens || !std::isfinite(s->scale) || !std::isfinite(s->keep)) return KVO_EINVAL;
  if (!aligned(s->starts, 4) || !aligned(s->lens, 4) || !aligned(s->lse, 4)) return KVO_EINVAL;
  if (s->tokens > 0) {
    if (!s->lse || !query_ok(s->q, s->q_ld, s->q_head_ld, s->tokens, s->heads)) return KVO_EINVAL;
  }
  if (s->rows > 0) {
    if (!s->out || !aligned(s->out, 4) || !aligned(s->carry, 4)) return KVO_EINVAL;
    if (cache->sequences > 1 && (s->out_ld < s->rows || (s->carry && s->carry_ld < s->rows))) return KVO_EINVAL;
    if (s->work_bytes < need || (need && !s->work) || !aligned(s->work, 4)) return KVO_EINVAL;
  }
  int64_t wait_clocks = 0;
  const kvo_status st = usable_status(ctx, &status, &wait_clocks);
  if (st != KVO_OK) return st;
  if (s->rows == 0) return KVO_OK;

  WeightArgs a = {};
  a.cache = cache_view(*cache);
  a.starts = s->starts;
  a.lens = s->lens;
  a.lse = s->lse;
  a.carry = s->carry;
  a.out = s->out;
  a.part = static_cast<float*>(s->work);
  a.status = status;
  a.carry_ld = s->carry_ld;
  a.out_ld = s->out_ld;
  a.rows = (uint32_t)s->rows;
  a.tokens = (uint32_t)s->tokens;
  a.heads = (uint32_t)s->heads;
  a.window = s->window > KVO_MAX_QUERIES ? 0 : (uint32_t)s->window;
  a.splits = weight_splits(s->tokens, cache->sequences, a.heads, s->rows, s->window);
  a.by_heads = divider(a.heads);
  a.scale = s->scale * kLog2e;
  a.keep = s->keep;
  a.wait_clocks = wait_clocks;
  // a dimension of one has no next element: its stride says nothing
  const int64_t head_ld = a.heads > 1 ? s->q_head_ld : KVO_DEQUANT_VALUES;
  const int64_t q_ld = s->tokens > 1 ? s->q_ld : a.heads * head_ld;
  a.columns = columns_of(a.heads, q_ld, head_ld, s->tokens);
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  CUtensorMap map = {};
  // without tokens no CTA gets as far as a copy
  if (s->tokens > 0 && !query_map(&map, s->q, a.heads, s->tokens, q_ld * 2, head_ld * 2, a.columns)) return KVO_ECUDA;
  cudaError_t e = launch_weights(a, map, on);
  if (e == cudaSuccess && a.splits > 1)
    e = launch_early(add_weights_kernel, dim3((a.rows + 255) / 256, a.cache.sequences), 256, 0, on, a);
  return e == cudaSuccess ? KVO_OK : KVO_ECUDA;
}
