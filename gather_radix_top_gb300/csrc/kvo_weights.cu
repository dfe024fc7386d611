// kvo_attention_weights: the attention weight that a chunk's tokens give to
// every cached position, summed over tokens and heads:
//     w_p = keep * carry_p + sum_c exp(scale * k_p . q_c - lse_c)
// over the (token, head) columns c whose token sees position p.
//
// Two CTAs of a cluster hold 128 positions each, dequantised once, and walk
// over the columns in tiles of 64 or 128: S [256 positions x columns] = K Q^T as
// pair MMAs, for which each CTA brings half of a tile's queries.  A position is
// a lane of S, so its sum over the columns stays in one thread's register; no
// maximum is needed, as lse_c is given.  Shared memory holds the positions (144
// KB), a ring for the queries' pieces (64 values of a CTA's columns), and raw
// rows, which come by bulk copies in groups of 16, each with its own four warps:
// they take them to registers, let the next ones come, and store the
// dequantised ones when the MMAs of the positions before have ended.  Tensor
// memory holds four tiles of S.
//
// A thread's sum over a tile is added to its running sum with the rounding
// error carried along, so that many tokens lose nothing.
//
// Tiles of positions times tiles of columns, end to end, are shared out evenly
// over the pairs.  Where a share begins or ends inside a tile of positions, a
// second launch adds the parts in their order.
//
// Measured: 32 tokens of 64 heads over 50,023 positions 84 us (1.41 PFLOP/s; 90
// us in a row of eager calls): a tile of 128 columns takes 2,650 clocks, of which
// its 36 MMAs need 2,304, and between two tiles of positions the tensor core
// waits 7,500 (the second half of the rows is converted behind the last MMA).
// The ring of queries matters most: with four slots, and room for four groups
// of rows, it takes 92 us.  301 uneven tokens of 20 heads in 7 sequences 77 us.
// A token of 64 heads in each of 64 sequences of 16,384 positions 215 us (3.3
// TB/s).  There a tile's rows are one chain: 42 KB of raw rows are all that fits
// beside the dequantised ones, so that memory is idle while they are converted,
// the tensor core while they are stored, and the workers while its MMAs run.
// Steps for that case, us: rows one copy each 585, even shares 347, groups of 16
// rows as one copy 264, four groups at once 221 (242 with the rows' release made
// sound), release before the conversion 231, kept queries and blocks looked up
// ahead 222, rows read without bank conflicts 215.
#include "kvo_cache.cuh"
#include "kvo_chunk.cuh"
#include "kvo_rows.cuh"
#include "kvo_tc.cuh"

namespace kvo {
namespace {

constexpr uint32_t kTile = 128;                          // positions of a CTA
constexpr uint32_t kSpan = 2 * kTile;                    // of a pair
constexpr uint32_t kHalf = 64;                           // rows that come together
constexpr uint32_t kWorkers = 16;                        // warps: four for each quarter of the columns
constexpr uint32_t kMma = kWorkers, kRows = kWorkers + 1, kQuery = kWorkers + 2, kQueries = 2;
constexpr uint32_t kWeightThreads = (kQuery + kQueries) * 32;
constexpr uint32_t kPieceBytes = kTile * 128;            // 64 values of every position
constexpr uint32_t kAhead = 4;                           // tiles of S
constexpr uint32_t kTileCost = 3;                        // of a tile of positions, in tiles of columns

// kC: a CTA's columns of a tile.  What the positions leave of shared memory goes
// to the raw rows where a tile of positions meets few columns (room for four
// groups of 16, and one tile's nine pieces of 32 columns, which stay for as long
// as the next tile of positions meets the same ones), else to the queries (six
// pieces of 64 columns, two groups).
template <uint32_t kC>
struct WeightShape {
  static constexpr uint32_t kSlotBytes = kC * 128, kSlots = kC == 32 ? 9 : 6;
  static constexpr bool kKeep = kSlots == 9;
  static constexpr uint32_t kRegions = kC == 32 ? 4 : 2;           // group g's rows go to region g % kRegions
  static constexpr uint32_t kRegionBytes = 16 * KVO_ROW_BYTES;
  static constexpr uint32_t kSmem = 1024 + 9 * kPieceBytes + kSlots * kSlotBytes + kRegions * kRegionBytes;
};

struct WeightArgs {
  CacheView cache;
  const int32_t* starts;
  const int32_t* lens;
  const float* lse;
  const float* carry;        // or NULL
  float* out;
  float* part;               // [2 * pairs][256]: of shares that begin, or end, inside a tile of positions
  uint32_t* status;
  int64_t carry_ld, out_ld;
  uint32_t rows, tokens, heads, window, pairs;
  Divider by_heads;
  Columns columns;           // of a CTA's half of a tile
  float scale, keep;
  int64_t wait_clocks;
};

template <uint32_t kSlots, uint32_t kRegions>
struct WeightShared {
  uint64_t k_full, k_empty, full[kSlots], empty[kSlots], s_full[kAhead], s_empty[kAhead], raw_full[4], raw_empty[kRegions];
  uint64_t summed[2], drained;       // summed: per job in turns, as a quarter may be a job ahead of another
  uint32_t tmem, gave_up;
  uint32_t issued[2][kQueries];      // per CTA and query warp: pieces of its own and before them that it has asked for
  uint32_t brought[4];               // halves that each group's rows have come for
  uint32_t there[4][4];              // per job in turns: rows that are not masked, row r is bit r % 32 of word r / 32
  float sums[2][3][kTile];           // per job in turns: of the quarters 1 to 3
};

// A worker warp's columns, where they are too many to pass from lane to lane.
template <uint32_t kMine>
struct ColumnShared {
  alignas(16) float lse[kWorkers][kMine];
  alignas(16) int32_t seen[kWorkers][kMine]; // the positions it sees
};
template <>
struct ColumnShared<16> {};

// A sequence's columns.
struct Run {
  uint32_t first, tokens;            // of the sequence
  int32_t before;                    // token i sees the first before + i positions
  uint32_t from;                     // the first token that counts
  uint32_t len;                      // positions held
  uint32_t begin, end;               // tiles of columns that count, for position 0

  __device__ __forceinline__ Run(const WeightArgs& a, uint32_t s) {
    const int32_t b = a.starts[s], e = a.starts[s + 1], T = (int32_t)a.tokens, held = max(a.lens[s], 0);
    if (b < 0 || b > T || e < b || e > T) atomicOr(a.status, kFlagRange);
    first = (uint32_t)min(max(b, 0), T);
    tokens = (uint32_t)min(max(e, (int32_t)first), T) - first;
    len = (uint32_t)min(held, (int32_t)a.rows);
    before = min(held, INT32_MAX - 1) - (int32_t)tokens + 1;
    from = max(a.window && a.window < tokens ? tokens - a.window : 0, sees(0));
    const Columns& c = a.columns;
    const uint32_t units = c.flat ? tokens * a.heads : tokens;
    begin = tile_of(a, from);
    end = len && from < tokens ? ((units + c.deep - 1) / c.deep * c.across + 1) / 2 : begin;
  }
  // The first token that sees position p.
  __device__ __forceinline__ uint32_t sees(uint32_t p) const { return (uint32_t)max((int32_t)p - before + 1, 0); }
  __device__ __forceinline__ uint32_t tile_of(const WeightArgs& a, uint32_t token) const {
    const Columns& c = a.columns;
    return (c.flat ? token * a.heads : token) / c.deep * c.across / 2;
  }
  __device__ __forceinline__ uint32_t tiles() const { return end - begin; }
  __device__ __forceinline__ uint32_t spans() const { return tiles() ? (len + kSpan - 1) / kSpan : 0; }
  __device__ __forceinline__ uint64_t work() const { return (uint64_t)spans() * (tiles() + kTileCost); }
};

// Part of the columns of one tile of positions.
struct Job {
  uint32_t seq, p0;                  // the pair's first position
  uint32_t begin, end;               // tiles of columns
  uint32_t slot;                     // of part, or UINT32_MAX: all of its columns
};

// The queries of one tile, as the roles that bring and use them count jobs: a
// job whose first tile is the last one's before it finds them in place.
struct Kept {
  uint32_t seq = UINT32_MAX, tile = 0;
  __device__ __forceinline__ bool has(const Job& job) const { return seq == job.seq && tile == job.begin; }
  __device__ __forceinline__ void set(const Job& job) {
    seq = job.seq;
    tile = job.end - 1;
  }
};

// All sequences' work, 32 of them at a time: f(first sequence, work before it and the lanes' after it).
template <typename F>
__device__ __forceinline__ uint64_t for_work(const WeightArgs& a, F f) {
  const uint32_t lane = threadIdx.x & 31;
  uint64_t before = 0;
  for (uint32_t s0 = 0; s0 < a.cache.sequences; s0 += 32) {
    uint64_t upto = s0 + lane < a.cache.sequences ? Run(a, s0 + lane).work() : 0;
#pragma unroll
    for (uint32_t d = 1; d < 32; d <<= 1) {
      const uint64_t o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    if (!f(s0, before, upto)) break;
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return before;
}

struct Shares {
  uint64_t work, each;
  uint32_t pairs, rest;              // the first `rest` shares have one more than `each`
  __device__ __forceinline__ Shares(const WeightArgs& a) {
    work = for_work(a, [](uint32_t, uint64_t, uint64_t) { return true; });
    pairs = (uint32_t)min((uint64_t)a.pairs, max(work / (kTileCost + 1), (uint64_t)1));
    each = work / pairs;
    rest = (uint32_t)(work - each * pairs);
  }
  __device__ __forceinline__ uint64_t from(uint32_t g) const { return g < pairs ? g * each + min(g, rest) : work; }
};

// f(job, run) for every job of the pair's share [lo, hi), in order, in every warp.
template <typename F>
__device__ __forceinline__ void for_jobs(const WeightArgs& a, uint32_t pair, uint64_t lo, uint64_t hi, F f) {
  if (lo >= hi) return;
  bool go = true;
  for_work(a, [&](uint32_t s0, uint64_t before, uint64_t upto) {
    for (uint32_t i = 0; i < 32 && s0 + i < a.cache.sequences && go; ++i) {
      const uint64_t end = before + __shfl_sync(0xffffffffu, upto, i);
      const uint64_t from = i ? before + __shfl_sync(0xffffffffu, upto, i - 1) : before;
      if (end <= lo || from == end) continue;
      if (from >= hi) return false;
      const Run run(a, s0 + i);
      const uint32_t tiles = run.tiles();
      const uint64_t cost = tiles + kTileCost, stop = min(hi, end) - from;
      uint64_t u = lo > from ? lo - from : 0;
      for (uint32_t j = (uint32_t)(u / cost); u < stop && go; ++j) {
        const uint64_t start = j * cost;
        const uint32_t x = (uint32_t)min(u - start, (uint64_t)tiles), y = (uint32_t)min(stop - start, (uint64_t)tiles);
        u = start + cost;
        if (x == y) continue;
        Job job{s0 + i, j * kSpan, run.begin + x, run.begin + y, UINT32_MAX};
        if (y - x < tiles) job.slot = 2 * pair + (x == 0);
        if (run.sees(job.p0) > run.from) job.begin = max(job.begin, run.tile_of(a, run.sees(job.p0)));   // others see none of them
        go = f(job, run);
      }
    }
    return go;
  });
}

// kC: a CTA's columns of a tile, 32 or 64.
template <uint32_t kC>
__global__ void __launch_bounds__(kWeightThreads, 1)
    weights_kernel(const __grid_constant__ WeightArgs a, const __grid_constant__ CUtensorMap qmap) {
  using S = WeightShape<kC>;
  constexpr uint32_t kSlotBytes = S::kSlotBytes, kSlots = S::kSlots, kRegions = S::kRegions;
  constexpr uint32_t kMine = kC / 2;                     // columns of a worker warp
  extern __shared__ uint8_t raw[];
  __shared__ WeightShared<kSlots, kRegions> sh;
  __shared__ ColumnShared<kMine> sc;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = cluster_rank(), pair = blockIdx.x >> 1;
  const uint32_t keys = (smem_u32(raw) + 1023u) & ~1023u, ring = keys + 9 * kPieceBytes, stage = ring + kSlots * kSlotBytes;

  if (tid == 0) {
    mbar_init(&sh.k_full, 2 * kWorkers);
    mbar_init(&sh.k_empty, 1);
    for (uint32_t i = 0; i < kSlots; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (uint32_t i = 0; i < kAhead; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_empty[i], 2 * kWorkers);
    }
    for (uint32_t i = 0; i < 4; ++i) {
      mbar_init(&sh.raw_full[i], 1);
      sh.brought[i] = 0;
    }
    for (uint32_t i = 0; i < kRegions; ++i) mbar_init(&sh.raw_empty[i], 4);
    for (uint32_t i = 0; i < 2; ++i) mbar_init(&sh.summed[i], kWorkers);
    mbar_init(&sh.drained, 1);
    sh.gave_up = a.wait_clocks == 0;
    for (uint32_t i = 0; i < 2; ++i)
      for (uint32_t w = 0; w < kQueries; ++w) sh.issued[i][w] = 0;
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
  const uint64_t lo = shares.from(pair), hi = pair < shares.pairs ? shares.from(pair + 1) : lo;
  const Columns& cols = a.columns;
  const uint32_t box = cols.wide * cols.deep * 128;      // bytes of a slot that a copy fills
  uint32_t n = 0, t = 0, jobs = 0;                       // pieces, tiles of S, jobs so far
  bool ok = true;

  if (warp == kRows) {
    // Lane l looks up rows l and l + 32 of each half, a job ahead: their blocks are
    // asked for before the rows of the job before come.  Sixteen rows
    // are a group: one copy where they lie one behind the other, as those of a
    // block do (a copy for every row takes 66 clocks each to issue).
    uint32_t halves = 0, p0 = 0;
    int32_t block[2][2];                                 // of the job whose rows come next: [half][l, l + 32]
    uint32_t held = 0;
    auto bring = [&]() -> bool {
#pragma unroll
      for (uint32_t h = 0; h < 2; ++h, ++halves) {
        uint32_t there[2], run[2];
        int64_t row[2], first[2];
#pragma unroll
        for (uint32_t u = 0; u < 2; ++u) {
          row[u] = cache_row_in(a.cache, block[h][u], p0 + h * kHalf + u * 32 + lane);
          there[u] = __ballot_sync(0xffffffffu, row[u] >= 0);
          first[u] = __shfl_sync(0xffffffffu, row[u], lane & 16);
          run[u] = __ballot_sync(0xffffffffu, row[u] >= 0 && row[u] == first[u] + (lane & 15));
        }
        if (lane < 2) sh.there[jobs & 3][2 * h + lane] = lane ? there[1] : there[0];   // (a slow warp may be three jobs behind)
        // The regions' uses so far: group g of this half is use `uses + g / kRegions` of its region.
        const uint32_t uses = halves * (4 / kRegions);
        const bool quick = (run[0] & run[1]) == ~0u;     // all four groups are runs
        if (quick) {
#pragma unroll
          for (uint32_t turn = 0; turn < 4 / kRegions; ++turn) {   // kRegions groups at a time, a lane for each
            // lane 16 e + u: group 2 u + e
            const uint32_t u = lane & 1, group = 2 * u + (lane >> 4), region = group % kRegions;
            if ((lane & 14) == 0 && group / kRegions == turn) {
              if (uses + turn) ok = wait(&sh.raw_empty[region], (uses + turn - 1) & 1);
              if (ok) {
                mbar_arrive_expect_tx(&sh.raw_full[group], 16 * KVO_ROW_BYTES);
                sh.brought[group] = halves + 1;
                bulk_copy_g2s(raw + (stage - smem_u32(raw)) + region * S::kRegionBytes,
                              a.cache.rows + (u ? first[1] : first[0]) * KVO_ROW_BYTES, 16 * KVO_ROW_BYTES,
                              &sh.raw_full[group]);
              }
            }
            if (!__all_sync(0xffffffffu, ok)) return false;
          }
          continue;
        }
#pragma unroll
        for (uint32_t u = 0; u < 2; ++u) {
          const uint32_t p = p0 + h * kHalf + u * 32 + lane;
          if (p < held && row[u] < 0) atomicOr(a.status, kFlagRange);
#pragma unroll 1
          for (uint32_t e = 0; e < 2; ++e) {             // lanes 16 e ..
            const uint32_t group = 2 * u + e, region = group % kRegions, use = uses + group / kRegions;
            const uint32_t mask = there[u] >> 16 * e & 0xffffu;
            const uint32_t dst = stage + region * S::kRegionBytes + lane % 16 * KVO_ROW_BYTES;
            const bool together = (run[u] >> 16 * e & 0xffffu) == 0xffffu, mine = lane / 16 == e;
            if (use) ok = wait(&sh.raw_empty[region], (use - 1) & 1);
            if (!__all_sync(0xffffffffu, ok)) return false;
            if (mine && row[u] < 0) {
              for (uint32_t c = 0; c < KVO_ROW_BYTES / 16; ++c) sts16(dst + 16 * c, make_uint4(0, 0, 0, 0));
              fence_proxy_async_smem();                  // before a later copy to the same place
            }
            __syncwarp();
            if (lane == 0) {
              mbar_arrive_expect_tx(&sh.raw_full[group], __popc(mask) * KVO_ROW_BYTES);
              sh.brought[group] = halves + 1;
            }
            __syncwarp();
            if (mine && row[u] >= 0 && (!together || lane % 16 == 0))
              bulk_copy_g2s(raw + (dst - smem_u32(raw)), a.cache.rows + row[u] * KVO_ROW_BYTES,
                            (together ? 16 : 1) * KVO_ROW_BYTES, &sh.raw_full[group]);
          }
        }
      }
      ++jobs;
      return true;
    };
    bool some = false;
    for_jobs(a, pair, lo, hi, [&](const Job& job, const Run& run) {
      int32_t next[2][2];
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        const uint32_t p = job.p0 + rank * kTile + i * 32 + lane;
        next[i / 2][i % 2] = p < run.len ? cache_block(a.cache, job.seq, p) : -1;
      }
      if (some && !bring()) return false;
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) block[i / 2][i % 2] = next[i / 2][i % 2];
      p0 = job.p0 + rank * kTile;
      held = run.len;
      some = true;
      return true;
    });
    if (some && __all_sync(0xffffffffu, ok)) bring();
  } else if (warp >= kQuery) {
    // the queries' pieces: warp w takes those of slots w, w + kQueries, ..  (A
    // slot stays with its warp: a wait for a phase is only sound for whoever has
    // seen the one before it.)
    const uint32_t w = warp - kQuery, full0 = dsmem_addr(&sh.full[0], 0);
    uint32_t at = 0;                                     // the tile's first piece
    uint32_t mine = w, slot = w, lap = 0;                // the warp's next one, its slot, and how often that was used
    Kept kept;
    for_jobs(a, pair, lo, hi, [&](const Job& job, const Run& run) {
      if (job.end <= job.begin) return true;
      const uint32_t begin = job.begin + (S::kKeep && kept.has(job));
      kept.set(job);
      if (lane == 0) {
        for (uint32_t tile = begin; tile < job.end && ok; ++tile, at += 9) {
          const uint32_t half = 2 * tile + rank, row = half / cols.across;
          const int32_t y = (int32_t)((half - row * cols.across) * cols.wide);
          const int32_t z = (int32_t)((cols.flat ? run.first * a.heads : run.first) + row * cols.deep);
          while (mine < at + 9) {
            if (lap) ok = wait(&sh.empty[slot], (lap - 1) & 1);
            if (!ok) break;
            if (rank == 0) mbar_arrive_expect_tx(&sh.full[slot], 2 * box);
            pair_load_box(ring + slot * kSlotBytes, &qmap, (int32_t)((mine - at) * 64), y, z, full0 + slot * 8);
            n = mine + 1;
            mine += kQueries;
            slot += kQueries;
            if (slot >= kSlots) {
              slot = w;
              mine = ++lap * kSlots + w;
            }
          }
        }
      }
      return (bool)__shfl_sync(0xffffffffu, ok, 0);
    });
    if (lane == 0) {
      if (ok) n = at;
      // no slot's release may still be on its way when the CTA ends
      for (uint32_t m = n > kSlots ? n - kSlots : 0; ok && m < n; ++m)
        if (m % kSlots % kQueries == w) ok = wait(&sh.empty[m % kSlots], m / kSlots & 1);
      dsmem_st_u32(dsmem_addr(&sh.issued[rank][w], 0), n);
    }
  } else if (warp == kMma) {
    if (rank == 0) {
      Kept kept;
      for_jobs(a, pair, lo, hi, [&](const Job& job, const Run&) {
        constexpr uint32_t kDesc = pair_desc(1, 2 * kC, false, false);
        const uint64_t k_tile = tile_desc(keys, 16), q_ring = tile_desc(ring, 16);
        const uint32_t tiles = job.end > job.begin ? job.end - job.begin : 0;
        const bool again = S::kKeep && tiles && kept.has(job), other = S::kKeep && tiles && !again && kept.seq != UINT32_MAX;
        if (tiles) kept.set(job);
        if (elect_one()) {
          if (other)                                       // the kept queries are done with
            for (uint32_t i = 0; i < kSlots; ++i) pair_commit(&sh.empty[i], 3);
          ok = wait(&sh.k_full, jobs & 1);
          uint32_t slot = n % kSlots, turn = n / kSlots & 1;
          for (uint32_t i = 0, at = t; i < tiles && ok; ++i, ++at) {
            const uint32_t buf = at % kAhead;
            const bool here = again && i == 0, keep = S::kKeep && i + 1 == tiles;
            if (at >= kAhead) ok = wait(&sh.s_empty[buf], (at / kAhead - 1) & 1);
            tc_fence_after();
#pragma unroll 3
            for (uint32_t piece = 0; piece < 9 && ok; ++piece) {
              if (!here) ok = wait(&sh.full[slot], turn);
              if (!ok) break;
#pragma unroll
              for (uint32_t k = 0; k < 4; ++k)
                pair_mma_bf16(tmem + buf * (2 * kC), k_tile + piece * (kPieceBytes >> 4) + 2 * k,
                              q_ring + slot * (kSlotBytes >> 4) + 2 * k, kDesc, piece + k > 0);
              if (!keep) pair_commit(&sh.empty[slot], 3);
              if (++slot == kSlots) {
                slot = 0;
                turn ^= !here;
              }
            }
            if (ok) pair_commit(&sh.s_full[buf], 3);
          }
          if (ok) pair_commit(&sh.k_empty, 3);
        }
        ok = __all_sync(0xffffffffu, ok);
        n += 9 * (tiles - again);
        t += tiles;
        ++jobs;
        return ok;
      });
      if (S::kKeep && kept.seq != UINT32_MAX && ok && elect_one())
        for (uint32_t i = 0; i < kSlots; ++i) pair_commit(&sh.empty[i], 3);
    }
  } else {
    // positions: piece `piece` of each 128 latent bytes of rows slot and slot + 64.
    // Eight lanes take a row's eight pieces (all banks once), and the upper four
    // store their second 16 bytes first: those of the lower four and of the upper
    // four go to the same banks, whose even 16 bytes then meet odd ones.
    const uint32_t piece = lane & 7, group = warp / 4;
    const uint32_t slot = warp * 4 + (lane >> 3), region = group % kRegions;
    const bool upper = piece >= 4;
    const uint32_t from = stage + region * S::kRegionBytes + slot % 16 * KVO_ROW_BYTES;
    const uint32_t to_lo = keys + (piece >> 2) * kPieceBytes + swizzled(slot, 2 * (piece & 3) + upper);
    const uint32_t to_hi = keys + (piece >> 2) * kPieceBytes + swizzled(slot, 2 * (piece & 3) + !upper);
    const uint32_t to_rope = keys + 8 * kPieceBytes + swizzled(slot, piece);
    // scores: position quad * 32 + lane against the columns quarter * kMine + c of a tile
    const uint32_t quad = warp & 3, quarter = warp >> 2;
    const uint32_t in_half = quarter % 2 * kMine + lane % kMine, deep = divide(in_half, cols.by_wide);
    const uint32_t wide = in_half - deep * cols.wide;
    const uint32_t lanes = tmem + (quad << 21) + quarter * kMine, s_empty = dsmem_addr(&sh.s_empty[0], 0);
    const uint32_t k_full = dsmem_addr(&sh.k_full, 0);
    // A job's last tile is taken after the next job's rows are in place, so that
    // its MMAs and this overlap.
    Job last{UINT32_MAX, 0, 0, 0, 0};
    uint32_t last_len = 0;
    float total = 0.0f, lost = 0.0f, lse = 0.0f, carried = 0.0f;   // of that job; lane l: column l of its last tile
    int32_t seen = 0;
    // one tile's weights to the sum; lane l has looked up column l
    auto add_tile = [&](uint32_t mine) -> bool {
      const uint32_t buf = t % kAhead;
      if (lse == -INFINITY) seen = 0;                      // a column that weighs nothing
      const float mine_lse = seen ? lse : 0.0f;
      if constexpr (kMine > 16) {
        if (lane < kMine) {
          sc.lse[warp][lane] = mine_lse;
          sc.seen[warp][lane] = seen;
        }
      }
      // four columns' values, from c on
      auto lses = [&](uint32_t c) -> float4 {
        if constexpr (kMine > 16)
          return *reinterpret_cast<const float4*>(&sc.lse[warp][c]);
        else
          return make_float4(__shfl_sync(~0u, mine_lse, c), __shfl_sync(~0u, mine_lse, c + 1), __shfl_sync(~0u, mine_lse, c + 2),
                             __shfl_sync(~0u, mine_lse, c + 3));
      };
      auto sees = [&](uint32_t c) -> int4 {
        if constexpr (kMine > 16)
          return *reinterpret_cast<const int4*>(&sc.seen[warp][c]);
        else
          return make_int4(__shfl_sync(~0u, seen, c), __shfl_sync(~0u, seen, c + 1), __shfl_sync(~0u, seen, c + 2),
                           __shfl_sync(~0u, seen, c + 3));
      };
      const bool edge = __any_sync(0xffffffffu, seen <= (int32_t)(mine | 31));
      __syncwarp();
      ok = wait(&sh.s_full[buf], t / kAhead & 1);
      if (!__all_sync(0xffffffffu, ok)) return false;
      tc_fence_after();
      float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (uint32_t c0 = 0; c0 < kMine; c0 += 16) {
        float x[16];
        tmem_ld16(lanes + buf * (2 * kC) + c0, x);
        tmem_ld_wait();
        if (c0 + 16 == kMine) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) cluster_mbar_arrive_relaxed(s_empty + buf * 8);
        }
#pragma unroll
        for (uint32_t c = 0; c < 16; c += 4) {
          const float4 l = lses(c0 + c);
          // The difference first, rounded once, then its power: with logits and
          // log-sum-exps that come times log2(e) already, each of the two is rounded
          // at their size, not at the difference's.  (Two more products for four.)
          fma_two(x[c], x[c + 1], a.scale, -l.x, -l.y);
          fma_two(x[c + 2], x[c + 3], a.scale, -l.z, -l.w);
          mul_two(x[c], x[c + 1], kLog2e);
          mul_two(x[c + 2], x[c + 3], kLog2e);
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) x[c + e] = exp2_approx(x[c + e]);
          if (edge) {
            const int4 see = sees(c0 + c);
            x[c] = (int32_t)mine < see.x ? x[c] : 0.0f;
            x[c + 1] = (int32_t)mine < see.y ? x[c + 1] : 0.0f;
            x[c + 2] = (int32_t)mine < see.z ? x[c + 2] : 0.0f;
            x[c + 3] = (int32_t)mine < see.w ? x[c + 3] : 0.0f;
          }
          add_two(sum[0], sum[1], x[c], x[c + 1]);
          add_two(sum[2], sum[3], x[c + 2], x[c + 3]);
        }
      }
      const float add = (sum[0] + sum[1]) + (sum[2] + sum[3]) - lost, now = total + add;
      lost = fabsf(now) < INFINITY ? (now - total) - add : 0.0f;   // (an infinite sum stays one)
      total = now;
      ++t;
      __syncwarp();
      return true;
    };
    // the last job's last tile, and its result
    auto finish = [&]() -> bool {
      const uint32_t mine = last.p0 + rank * kTile + quad * 32 + lane;
      if (last.begin < last.end && !add_tile(mine)) return false;
      const uint32_t job = jobs - 1;
      const bool there = sh.there[job & 3][quad] >> lane & 1;
      float* const sums = &sh.sums[job & 1][0][quad * 32 + lane];
      if (quarter) sums[(quarter - 1) * kTile] = total;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.summed[job & 1]);
      if (quarter == 0) {
        ok = wait(&sh.summed[job & 1], job >> 1 & 1);
        if (!__all_sync(0xffffffffu, ok)) return false;
        total = there ? (total + sums[0]) + (sums[kTile] + sums[2 * kTile]) : 0.0f;
        if (last.slot != UINT32_MAX)
          a.part[last.slot * kSpan + rank * kTile + quad * 32 + lane] = total;
        else if (mine < last_len)
          a.out[last.seq * a.out_ld + mine] = a.carry ? fmaf(a.keep, carried, total) : total;
      }
      return true;
    };
    for_jobs(a, pair, lo, hi, [&](const Job& job, const Run& run) {
      const uint32_t mine = job.p0 + rank * kTile + quad * 32 + lane;
      // lane l looks up column l of the warp's: its log-sum-exp, and the positions it sees
      auto column = [&](uint32_t tile, float* to_lse, int32_t* to_seen) {
        *to_lse = 0.0f;
        *to_seen = 0;
        if (tile >= job.end || deep >= cols.deep) return;
        const uint32_t half = 2 * tile + quarter / 2;
        uint32_t at = half * cols.deep + deep;
        if (!cols.flat) {
          const uint32_t row = half / cols.across, head = (half - row * cols.across) * cols.wide + wide;
          if (head >= a.heads) return;
          at = (row * cols.deep + deep) * a.heads + head;
        }
        const uint32_t token = divide(at, a.by_heads);
        if (token < run.from || token >= run.tokens) return;
        *to_lse = __ldg(a.lse + (int64_t)run.first * a.heads + at);   // (looked at when its tile is)
        *to_seen = min(run.before + (int32_t)token, (int32_t)run.len);
      };
      float next_lse, next_carried = 0.0f;
      int32_t next_seen;
      if (last.seq == job.seq && last.begin < last.end && last.end - 1 == job.begin) {
        next_lse = lse;                                    // the same columns again
        next_seen = seen;
      } else {
        column(job.begin, &next_lse, &next_seen);
      }
      if (quarter == 0 && a.carry && mine < run.len) next_carried = a.carry[job.seq * a.carry_ld + mine];

#pragma unroll
      for (uint32_t h = 0; h < 2; ++h) {
        ok = ok && wait(&sh.raw_full[group], h);         // (two halves a job)
        uint4 lat[4], lo[4], up[4];
        for (uint32_t k = 0; k < 4; ++k) lat[k] = lds16(from + 128 * k + 16 * piece);
        const uint4 eight = lds16(from + KVO_LATENT_BYTES), rope = lds16(from + KVO_LATENT_BYTES + 16 + 16 * piece);
        uint32_t all = mixed(eight) ^ mixed(rope);       // the rows are in registers before the next ones may come
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) all ^= mixed(lat[k]);
        loads_are_in(all);
        if (!__all_sync(0xffffffffu, ok)) return false;  // (then the next rows must not come)
        if (lane == 0) mbar_arrive(&sh.raw_empty[region]);
        const uint32_t pick = upper ? 0x7632u : 0x5410u;
        const uint32_t scales[2] = {__byte_perm(eight.x, eight.y, pick), __byte_perm(eight.z, eight.w, pick)};
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) {
          const uint16_t scale = (uint16_t)(scales[k >> 1] >> (k & 1) * 16);
          const float bias = -1152.0f * __half2float(__ushort_as_half(scale));
          dequant4(upper ? lat[k].z : lat[k].x, scale, bias, lo[k].x, lo[k].y);
          dequant4(upper ? lat[k].w : lat[k].y, scale, bias, lo[k].z, lo[k].w);
          dequant4(upper ? lat[k].x : lat[k].z, scale, bias, up[k].x, up[k].y);
          dequant4(upper ? lat[k].y : lat[k].w, scale, bias, up[k].z, up[k].w);
        }
        if (h == 0 && jobs) ok = wait(&sh.k_empty, (jobs - 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) return false;
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) {
          sts16(to_lo + 2 * k * kPieceBytes + h * 8192, lo[k]);
          sts16(to_hi + 2 * k * kPieceBytes + h * 8192, up[k]);
        }
        sts16(to_rope + h * 8192, rope);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) cluster_mbar_arrive_own(k_full);
      if (jobs && !finish()) return false;
      ++jobs;
      last = job;
      last_len = run.len;
      total = lost = 0.0f;
      lse = next_lse;
      seen = next_seen;
      carried = next_carried;
      for (uint32_t tile = job.begin; tile + 1 < job.end; ++tile) {
        column(tile + 1, &next_lse, &next_seen);
        if (!add_tile(mine)) return false;
        lse = next_lse;
        seen = next_seen;
      }
      return true;
    });
    // The last release too has to come before the CTA ends: what came later
    // would find another CTA's shared memory there.  And it says that every warp
    // has ended the job before the last but one, whose barrier and sums are next.
    if (jobs && __all_sync(0xffffffffu, ok)) {
      ok = wait(&sh.k_empty, (jobs - 1) & 1);
      if (__all_sync(0xffffffffu, ok)) finish();
    }
  }

  // Both CTAs end together: the MMAs read the other's memory, and arrivals and
  // copies go to rank 0's barriers.  Where a wait gave up in either, what is in
  // flight finishes first: the MMAs, then the copies, of which one that a CTA has
  // not asked for counts as come.
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
    if (warp == kRows && lane < 4 && sh.brought[lane] && !landed(&sh.raw_full[lane], (sh.brought[lane] - 1) & 1))
      atomicOr(a.status, kFlagInflight);
    if (warp == kQuery && lane == 0 && rank == 0) {
      uint32_t most = 0, least = UINT32_MAX;
      for (uint32_t i = 0; i < 2 * kQueries; ++i) {
        most = max(most, sh.issued[i / kQueries][i % kQueries]);
        least = min(least, sh.issued[i / kQueries][i % kQueries]);
      }
      for (uint32_t m = least; m < most; ++m) {
        const uint32_t owner = m % kSlots % kQueries;
        const bool here = m < sh.issued[0][owner], there = m < sh.issued[1][owner];
        if (here == there) continue;
        if (!here) mbar_arrive_expect_tx(&sh.full[m % kSlots], 2 * box);
        mbar_complete_tx(&sh.full[m % kSlots], box);
      }
      for (uint32_t m = most > kSlots ? most - kSlots : 0; m < most; ++m) {
        const uint32_t owner = m % kSlots % kQueries;
        if (m >= sh.issued[0][owner] && m >= sh.issued[1][owner]) continue;
        if (!landed(&sh.full[m % kSlots], m / kSlots & 1)) atomicOr(a.status, kFlagInflight);
      }
    }
    __syncthreads();
  }
  // Positions that no column sees, or none is held at.
  const uint32_t per = max(gridDim.x / a.cache.sequences, 1u), groups = gridDim.x / per;   // CTAs a sequence
  for (uint32_t s = blockIdx.x / per; s < a.cache.sequences && blockIdx.x / per < groups; s += groups) {
    const Run run(a, s);
    for (uint32_t p = (run.spans() ? run.len : 0) + blockIdx.x % per * kWeightThreads + tid; p < a.rows; p += per * kWeightThreads)
      a.out[s * a.out_ld + p] = p < run.len && a.carry ? a.keep * a.carry[s * a.carry_ld + p] : 0.0f;
  }
  cluster_sync();
  if (warp == kMma) pair_tmem_free(tmem, 512);
}

// Block g - 1: the tile of positions that share g is the first to cut.
__global__ void __launch_bounds__(kSpan) add_parts_kernel(const __grid_constant__ WeightArgs a) {
  const uint32_t g = blockIdx.x + 1;
  wait_previous_grid();
  allow_next_grid();
  const Shares shares(a);
  if (g >= shares.pairs) return;
  const uint64_t at = shares.from(g);
  uint32_t seq = 0;
  uint64_t base = 0;                                     // work before sequence seq
  for_work(a, [&](uint32_t s0, uint64_t before, uint64_t upto) {
    const uint32_t past = __ballot_sync(0xffffffffu, before + upto > at);
    if (!past) return true;
    const int i = __ffs((int)past) - 1;
    seq = s0 + i;
    const uint64_t prior = __shfl_sync(0xffffffffu, upto, i > 0 ? i - 1 : 0);
    base = before + (i > 0 ? prior : 0);
    return false;
  });
  const Run run(a, seq);
  const uint64_t cost = run.tiles() + kTileCost, j = (at - base) / cost, from = base + j * cost, end = from + run.tiles();
  if (at == from || at >= end || shares.from(g - 1) > from) return;
  float total = 0.0f;
  for (uint32_t p = g - 1; p < shares.pairs && shares.from(p) < end; ++p)
    total += __ldcg(a.part + (2 * p + (p == g - 1)) * kSpan + threadIdx.x);
  const uint32_t mine = (uint32_t)j * kSpan + threadIdx.x;
  if (mine < run.len)
    a.out[seq * a.out_ld + mine] = a.carry ? fmaf(a.keep, a.carry[seq * a.carry_ld + mine], total) : total;
}

template <uint32_t kC>
cudaError_t launch_weights(const WeightArgs& a, const CUtensorMap& map, cudaStream_t stream) {
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!ready[dev & 63]) {
    e = cudaFuncSetAttribute(weights_kernel<kC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)WeightShape<kC>::kSmem);
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
  lc.gridDim = dim3(2 * a.pairs);
  lc.blockDim = dim3(kWeightThreads);
  lc.dynamicSmemBytes = WeightShape<kC>::kSmem;
  lc.stream = stream;
  lc.attrs = attr;
  lc.numAttrs = 2;
  e = cudaLaunchKernelEx(&lc, weights_kernel<kC>, a, map);
  // no share ends inside a tile of positions that meets one tile of columns
  const Columns& c = a.columns;
  const uint32_t units = c.flat ? a.tokens * a.heads : a.tokens, most = ((units + c.deep - 1) / c.deep * c.across + 1) / 2;
  if (e != cudaSuccess || a.pairs < 2 || most < 2) return e;
  return launch_early(add_parts_kernel, dim3(a.pairs - 1), kSpan, 0, stream, a);
}

}  // namespace
}  // namespace kvo

extern "C" int64_t kvo_attention_weights_work_bytes(int64_t tokens, int32_t sequences, int32_t heads, int64_t rows,
                                                    int64_t window) {
  if (tokens < 0 || tokens > KVO_MAX_QUERIES || sequences < 1 || sequences > KVO_MAX_QUERIES) return -1;
  if (heads < 1 || heads > KVO_MAX_HEADS || rows < 0 || rows > INT32_MAX - 255 || window < 0) return -1;
  return tokens > 0 && rows > 0 ? (int64_t)(kvo::device_sms() / 2) * 2 * kvo::kSpan * 4 : 0;
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
  a.pairs = (uint32_t)device_sms() / 2;
  a.by_heads = divider(a.heads);
  a.scale = s->scale;
  a.keep = s->keep;
  a.wait_clocks = wait_clocks;
  // a dimension of one has no next element: its stride says nothing
  const int64_t head_ld = a.heads > 1 ? s->q_head_ld : KVO_DEQUANT_VALUES;
  const int64_t q_ld = s->tokens > 1 ? s->q_ld : a.heads * head_ld;
  int64_t each = (s->tokens + cache->sequences - 1) / cache->sequences;
  if (a.window && a.window < each) each = a.window;
  // Tiles of 64 or of 128 columns, by the columns of a sequence when all have the
  // same.  Both ways, us: 64 columns, 64 sequences of 16,384 positions 212 and
  // 347, one of 50,000 24 and 29 (with the second launch); 16 columns, 64 of 2,048
  // 51 and 66; 128 columns, 64 of 2,048 62 and 66, 16 of 4,096 37 and 34, one of
  // 50,000 30 and 28; 256 columns, 8 of 8,192 44 and 42.
  const bool few = each * a.heads <= 64;
  a.columns = columns_of(a.heads, q_ld, head_ld, s->tokens, few ? 32 : 64);
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  CUtensorMap map = {};
  // without tokens no CTA gets as far as a copy
  if (s->tokens > 0 && !query_map(&map, s->q, a.heads, s->tokens, q_ld * 2, head_ld * 2, a.columns)) return KVO_ECUDA;
  return (few ? launch_weights<32>(a, map, on) : launch_weights<64>(a, map, on)) == cudaSuccess ? KVO_OK : KVO_ECUDA;
}
