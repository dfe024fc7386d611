// kvo_index_scores: score[t][j] = s_j * sum_h w[t][h] * max(0, q[t][h] . key_j).
//
// Keys times queries is a matrix product with a reduction over its columns:
// a tile of 128 keys is the A operand (M = 128), the heads of up to 8 query
// tokens of one sequence are B (N = 32 .. 256 columns).  With the keys along M, a
// thread of the epilogue holds one key's products with every head, so the
// weighted sum over heads needs no exchange between threads, and the keys
// are read once for all query tokens of their sequence.
//
// One CTA per SM: a warp brings key tiles into a ring in shared memory
// (a TMA box per run of keys of one block, looked up in the table), another
// issues the MMAs into accumulators in tensor memory, and four
// teams of four warps reduce them in turn.  Nothing but the queries and the
// scores passes through global memory twice.  A sequence's query tokens (a
// task) have a row of the grid, whose CTAs take their tiles in turn; of many
// tasks, whose lengths may differ, the tiles are shared out end to end, and a
// CTA goes from one task to the next while its ring fills on.
//
// What bounds it: up to 128 columns, reading the keys (132 bytes a key as e4m3,
// 256 as bf16) after about 4 us of launch, queries and first keys: a million
// keys take 25.4 us as one run of e4m3 (5.5 TB/s), 26.7 in shuffled blocks of
// 16 and 42.2 as bf16 (6.4 TB/s), whether for 16 or 64 heads.  For 256
// columns (four tokens of 64 heads), the epilogue: 262,144 keys take 16.0 us
// against 8.6 for one token.  Not its two operations per product, though: they
// are under half of its 5 warp instructions per 32 products, the issue slots are
// 54 % busy, and a copy without them took 14.7 us where all took 18.5.  The rest
// is what goes with a tile (both teams of an accumulator look its rows up) and
// waiting; the two have not been told apart.  Slower ones, for
// the million in blocks: a barrier of all warps before the first keys instead of
// one for the queries alone 27.5 us, MMAs from one thread of a diverged warp 30.3
// (28.4 by then), one loading warp alone 45.2 (it issues a box every 60 clocks),
// table entries that are used as soon as they are asked for 48.2.
#include <algorithm>
#include <cstddef>
#include <type_traits>

#include <cuda.h>

#include "kvo_cache.cuh"
#include "kvo_tc.cuh"

namespace kvo {
namespace {

constexpr uint32_t kScoreTeams = 4;                             // of four warps each: the epilogue
constexpr uint32_t kScoreEpilogue = kScoreTeams * 128;
constexpr uint32_t kLoadWarps = 3;                              // they take key tiles in turn
constexpr uint32_t kLoadWarp = kScoreEpilogue / 32, kMmaWarp = kLoadWarp + kLoadWarps;
constexpr uint32_t kScoreThreads = (kMmaWarp + 1) * 32;
constexpr uint32_t kKeyTile = 128;
constexpr uint32_t kScoreMaxCols = 256;
constexpr uint32_t kScoreMaxTokens = kScoreMaxCols / 32;
constexpr uint32_t kMostTasks = 512;                            // of a grid's row
constexpr uint32_t kTaskCost = 4;                               // of going to another task, in tiles

struct ScoreArgs {
  CacheView cache;
  const uint8_t* q;
  const float* w;
  const int32_t* lens;
  float* scores;
  uint32_t* status;
  int64_t q_ld, q_head_ld;   // bytes
  int64_t w_ld, ld;          // elements
  uint32_t n;
  uint32_t per_seq, heads;
  uint32_t block_shift;      // positions per column, as a power of two
  uint32_t head_cols;        // columns of a query token: heads rounded up to 32
  uint32_t group;            // query tokens of a CTA
  uint32_t groups;           // groups of a sequence
  Divider by_groups;
  uint32_t tasks, slice;     // groups of all sequences, and how many of them a row of the grid shares out
  uint32_t accs;             // accumulators in tensor memory: 4, or 2 of more than 128 columns
  uint32_t tmem_cols;
  int64_t wait_clocks;       // after which a wait gives up
  uint32_t run;              // consecutive keys that never leave their block (>= 4), or 1
};

template <bool kF8>
struct ScoreShape {
  static constexpr uint32_t kKeyBytes = kF8 ? 128 : 256;
  static constexpr uint32_t kTileBytes = kKeyTile * kKeyBytes;
  // tiles in the ring: 112 or 128 KB, about twice what covers the memory latency at an SM's share of the
  // bandwidth
  static constexpr uint32_t kStages = kF8 ? 7 : 4;
  static constexpr uint32_t kPieces = kKeyBytes / 16;           // 16-byte pieces of a query head
};

struct ScoreShared {
  uint64_t full[8], empty[8], acc_full[4], acc_empty[4], q_full, task_done, drained;
  uint32_t tmem;
  uint32_t gave_up;
  uint32_t brought[kLoadWarps];                                 // per loading warp: its first tile that it has not brought
  uint32_t first, last, first_task;                             // this CTA's tiles
  uint32_t warp_tiles[kScoreThreads / 32], warp_cost[kScoreThreads / 32];
  uint32_t start[kMostTasks + 1];                               // tiles before each task's
  uint32_t most[kMostTasks];                                    // positions that any of a task's tokens sees
  int32_t len[2][kScoreMaxTokens];                              // of the task at hand and the next
  alignas(16) float w[2][kScoreMaxCols];                        // read four at a time
  float best[kScoreTeams][4];
};
static_assert(alignof(ScoreShared) >= 16 && offsetof(ScoreShared, w) % 16 == 0);

// kShared: the CTAs of a row of the grid share the tiles of many tasks out;
// else a row is one task, whose tiles go to its CTAs in turn.  kPadded: there
// are fewer heads than columns of a token.
template <bool kF8, bool kShared, bool kPadded>
__global__ void __launch_bounds__(kScoreThreads, 1) index_scores_kernel(const __grid_constant__ ScoreArgs a,
                                                                        const __grid_constant__ CUtensorMap map) {
  using S = ScoreShape<kF8>;
  extern __shared__ uint8_t raw[];
  __shared__ ScoreShared sh;
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t cols = a.group * a.head_cols;
  const uint32_t ring = smem_u32(smem), queries = ring + S::kStages * S::kTileBytes;

  // a task is a group of query tokens of one sequence: here task0 .. task0 + tasks - 1
  const uint32_t task0 = kShared ? blockIdx.y * a.slice : blockIdx.y;
  const uint32_t tasks = kShared ? min(a.slice, a.tasks - task0) : 1;
  auto seq_of = [&](uint32_t r) -> uint32_t { return divide(task0 + r, a.by_groups); };
  auto token_of = [&](uint32_t r) -> uint32_t {                 // the first token of task r
    const uint32_t s = seq_of(r);
    return s * a.per_seq + (task0 + r - s * a.groups) * a.group;
  };
  auto tokens_of = [&](uint32_t r) -> uint32_t {
    return min(a.group, a.per_seq - (task0 + r - seq_of(r) * a.groups) * a.group);
  };
  auto longest = [&](uint32_t r) -> uint32_t {                  // positions that any of its tokens sees
    const uint32_t t0 = token_of(r), tokens = tokens_of(r);
    int32_t most = 0;
    for (uint32_t g = 0; g < tokens; ++g) most = max(most, min(a.lens[t0 + g], (int32_t)a.n));
    return (uint32_t)most;
  };

  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return wait_or_give_up(bar, parity, &sh.gave_up, a.wait_clocks);
  };

  wait_previous_grid();
  allow_next_grid();
  if (tid == 0) {
    for (uint32_t i = 0; i < S::kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (uint32_t i = 0; i < a.accs; ++i) {
      mbar_init(&sh.acc_full[i], 1);
      mbar_init(&sh.acc_empty[i], kScoreEpilogue / a.accs);
    }
    mbar_init(&sh.q_full, kLoadWarp);
    mbar_init(&sh.task_done, 1);
    mbar_init(&sh.drained, 1);
    sh.gave_up = a.wait_clocks == 0;
    sh.first = sh.last = sh.first_task = 0;
  }
  if (warp == kMmaWarp) tmem_alloc(&sh.tmem, a.tmem_cols);
  // this CTA's tiles are number first, first + step, .. below last of all tasks' tiles end to end
  uint32_t first, last, first_task = 0, only = 0;
  const uint32_t step = kShared ? 1 : gridDim.x;
  if constexpr (kShared) {
    // a part of about the same cost for every CTA, from running sums over the tasks
    const uint32_t most = tid < tasks ? longest(tid) : 0;
    const uint32_t here = (most + kKeyTile - 1) / kKeyTile, cost = here ? here + kTaskCost : 0;
    uint32_t tiles_to = here, cost_to = cost;                   // up to and with task tid
#pragma unroll
    for (uint32_t d = 1; d < 32; d *= 2) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, tiles_to, d), c = __shfl_up_sync(0xffffffffu, cost_to, d);
      if (lane >= d) tiles_to += t, cost_to += c;
    }
    if (lane == 31) sh.warp_tiles[warp] = tiles_to, sh.warp_cost[warp] = cost_to;
    __syncthreads();
    const uint32_t wt = lane < kScoreThreads / 32 ? sh.warp_tiles[lane] : 0;
    const uint32_t wc = lane < kScoreThreads / 32 ? sh.warp_cost[lane] : 0;
    const uint32_t all = __reduce_add_sync(0xffffffffu, wc);
    tiles_to += __reduce_add_sync(0xffffffffu, lane < warp ? wt : 0);
    cost_to += __reduce_add_sync(0xffffffffu, lane < warp ? wc : 0);
    if (tid < tasks) {
      const uint32_t from = cost_to - cost, tiles_from = tiles_to - here;
      sh.most[tid] = most;
      sh.start[tid] = tiles_from;
      if (tid == tasks - 1) sh.start[tasks] = tiles_to;
      const uint32_t lo = (uint32_t)((uint64_t)all * blockIdx.x / gridDim.x);
      const uint32_t hi = (uint32_t)((uint64_t)all * (blockIdx.x + 1) / gridDim.x);
      auto tile_at = [&](uint32_t x) { return tiles_from + (x - from > kTaskCost ? x - from - kTaskCost : 0); };
      if (lo >= from && lo < cost_to) sh.first = tile_at(lo), sh.first_task = tid;
      if (hi > from && hi <= cost_to) sh.last = tile_at(hi);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    first = sh.first, last = sh.last, first_task = sh.first_task;
  } else {
    only = longest(0);
    first = blockIdx.x, last = (only + kKeyTile - 1) / kKeyTile;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  const uint32_t mine = last > first ? (last - first + step - 1) / step : 0;
  const uint32_t tmem = sh.tmem;

  if (mine) {
    // whether tile i is behind task r, the task of tile i from one before, and
    // its first position there
    auto behind = [&](uint32_t i, uint32_t r) -> bool { return kShared && first + i >= sh.start[r + 1]; };
    auto walk = [&](uint32_t i, uint32_t& r) {
      while (behind(i, r)) ++r;
    };
    auto position = [&](uint32_t i, uint32_t r) -> uint32_t {
      return (kShared ? first + i - sh.start[r] : first + i * step) * kKeyTile;
    };
    const uint32_t only_seq = kShared ? 0 : seq_of(0);
    auto task_seq = [&](uint32_t r) -> uint32_t { return kShared ? seq_of(r) : only_seq; };
    auto most_of = [&](uint32_t r) -> uint32_t { return kShared ? sh.most[r] : only; };

    // Lane l of the loading warp brings the l-th run of a.run keys of a tile
    // (all in one block), or keys 4l .. 4l+3 where a block holds no such run;
    // one that is not there is replaced by the cache's first and masked later.
    // Table entries are asked for kLookup tiles before the keys: they take as
    // long to come.
    constexpr uint32_t kLookup = 2;
    const bool loads = warp >= kLoadWarp && warp < kMmaWarp;
    const uint32_t turn0 = warp - kLoadWarp;                    // a loading warp's first tile
    const bool runs = a.run > 1;
    const uint32_t width = runs ? a.run : 4;
    int4 block[kLookup];
    uint32_t ahead_task = first_task, bring_task = ahead_task;
    auto look_ahead = [&](uint32_t i) -> int4 {
      int32_t b[4] = {0, 0, 0, 0};
      if (i < mine) walk(i, ahead_task);
      if (i < mine && width * lane < kKeyTile) {
        const uint32_t p = position(i, ahead_task) + width * lane, seq = task_seq(ahead_task), most = most_of(ahead_task);
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k)
          if ((k == 0 || !runs) && p + k < most) b[k] = cache_block(a.cache, seq, p + k);
      }
      return make_int4(b[0], b[1], b[2], b[3]);
    };
    auto bring = [&](uint32_t j) {
      const uint32_t slot = j % S::kStages, dst = ring + slot * S::kTileBytes + lane * width * 128;
      walk(j, bring_task);
      const uint32_t p = position(j, bring_task) + width * lane, most = most_of(bring_task);
      auto row = [&](int32_t id, uint32_t k) -> int32_t {
        return p + k < most ? max(0, (int32_t)cache_row_in(a.cache, id, p + k)) : 0;
      };
      if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot], S::kTileBytes);
      __syncwarp();
      if (width * lane < kKeyTile) {
        const int32_t r0 = row(block[0].x, 0);
        if (runs) {
#pragma unroll
          for (uint32_t c = 0; c < S::kKeyBytes / 128; ++c)
            load_box(dst + c * (kKeyTile * 128), &map, (int32_t)(c * 64), r0, &sh.full[slot]);
        } else {
          const int32_t r1 = row(block[0].y, 1), r2 = row(block[0].z, 2), r3 = row(block[0].w, 3);
#pragma unroll
          for (uint32_t c = 0; c < S::kKeyBytes / 128; ++c)
            gather_rows(dst + c * (kKeyTile * 128), &map, (int32_t)(c * 64), r0, r1, r2, r3, &sh.full[slot]);
        }
      }
#pragma unroll
      for (uint32_t k = 0; k + 1 < kLookup; ++k) block[k] = block[k + 1];
      block[kLookup - 1] = look_ahead(j + kLookup * kLoadWarps);
    };
    if (loads) {
#pragma unroll
      for (uint32_t i = 0; i < kLookup; ++i) block[i] = look_ahead(turn0 + i * kLoadWarps);
    }
    if (warp < kLoadWarp) {
      // team w takes the tiles of accumulator w % accs, and of their query
      // tokens every parts-th
      const uint32_t team = warp >> 2, acc = team % a.accs, part = team / a.accs, parts = kScoreTeams / a.accs;
      const uint32_t lane_base = (warp & 3) * 32, key = lane_base + lane;
      const uint32_t from = tmem + (lane_base << 16) + acc * cols;
      // The queries of a task, their weights and lengths.  The workers bring
      // those of the next one when the last product of this one is done.
      uint32_t task = first_task, nth = 0, tokens = 0, t0 = 0;
      auto bring_queries = [&] {
        tokens = tokens_of(task), t0 = token_of(task);
        for (uint32_t i = tid; i < cols * S::kPieces; i += kScoreEpilogue) {
          const uint32_t r = i / S::kPieces, c = i % S::kPieces, g = r / a.head_cols, h = r - g * a.head_cols;
          const bool real = g < tokens && h < a.heads;
          copy16_async(queries + (c >> 3) * (cols * 128) + swizzled(r, c & 7),
                       real ? a.q + (t0 + g) * a.q_ld + h * a.q_head_ld + c * 16 : a.q, real);
        }
        copy_async_commit();
        for (uint32_t i = tid; i < cols; i += kScoreEpilogue) {
          const uint32_t g = i / a.head_cols, h = i - g * a.head_cols;
          sh.w[nth & 1][i] = g < tokens && h < a.heads ? a.w[(t0 + g) * a.w_ld + h] : 0.0f;
        }
        if (tid < tokens) sh.len[nth & 1][tid] = min(a.lens[t0 + tid], (int32_t)a.n);
        copy_async_wait<0>();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_full);
      };
      auto next_task = [&] {
        wait(&sh.task_done, nth & 1);
        __syncwarp();
        do ++task;
        while (sh.start[task + 1] == sh.start[task]);
        ++nth;
        bring_queries();
      };
      bring_queries();
      wait(&sh.q_full, 0);

      // table entries are asked for two of this team's tiles ahead, the keys'
      // factors one
      uint32_t block_task = task, row_task = task;
      auto look_up = [&](uint32_t i) -> int32_t {
        if (i >= mine) return -1;
        walk(i, block_task);
        const uint32_t p = position(i, block_task) + key;
        return p < most_of(block_task) ? cache_block(a.cache, task_seq(block_task), p) : -1;
      };
      auto row_in = [&](uint32_t i, int32_t id) -> int64_t {
        if (i >= mine) return -1;
        walk(i, row_task);
        return cache_row_in(a.cache, id, position(i, row_task) + key);
      };
      auto factor_of = [&](int64_t r) -> float { return kF8 && r >= 0 ? a.cache.key_scales[r] : 1.0f; };
      bool next_there;
      float next_factor;
      {
        const int64_t r = row_in(acc, look_up(acc));
        next_there = r >= 0;
        next_factor = factor_of(r);
      }
      int32_t block_after = look_up(acc + a.accs);
      for (uint32_t i = acc, turn = 0; i < mine; i += a.accs, turn ^= 1) {
        if (behind(i, task)) {
          while (behind(i, task)) next_task();
          wait(&sh.q_full, nth & 1);
        }
        const float* weights = sh.w[nth & 1];
        const int32_t* lens = sh.len[nth & 1];
        const uint32_t p = position(i, task) + key;
        const bool there = next_there;
        const float factor = next_factor;
        if (!there && p < most_of(task)) atomicOr(a.status, kFlagRange);
        const int64_t r = row_in(i + a.accs, block_after);
        next_there = r >= 0;
        next_factor = factor_of(r);
        block_after = look_up(i + 2 * a.accs);
        // after a wait that gave up the team goes on through what it finds
        // (its warps meet at barriers below); the status says so
        wait(&sh.acc_full[acc], turn);
        __syncwarp();
        tc_fence_after();
        for (uint32_t g = part; g < tokens; g += parts) {
          float s0 = 0.0f, s1 = 0.0f;
          for (uint32_t c = 0; c < a.head_cols; c += 32) {
            float v[32];
            tmem_ld32(from + g * a.head_cols + c, v);
            const float4* w4 = reinterpret_cast<const float4*>(&weights[g * a.head_cols + c]);
            tmem_ld_wait();
#pragma unroll
            for (uint32_t e = 0; e < 8; ++e) {
              const float4 w = w4[e];
              s0 = fmaf(w.x, max_nan(v[4 * e], 0.0f), s0);
              s1 = fmaf(w.y, max_nan(v[4 * e + 1], 0.0f), s1);
              s0 = fmaf(w.z, max_nan(v[4 * e + 2], 0.0f), s0);
              s1 = fmaf(w.w, max_nan(v[4 * e + 3], 0.0f), s1);
            }
          }
          // Columns past the last head are no part of the sum, but an infinite
          // key's products with their zeros are NaN, and so is the sum then:
          // it is formed again without them.  Asked of the sum, as that is
          // rare: 13 contexts of 24 heads take 9.2 us, with a bound or a choice
          // at the last columns' products 9.8 to 10.1, with neither 8.9.
          if (kPadded && __any_sync(0xffffffffu, isnan(s0 + s1))) {
            s0 = s1 = 0.0f;
#pragma unroll 1
            for (uint32_t c = 0; c < a.heads; c += 4) {
              float v[4];
              tmem_ld4(from + g * a.head_cols + c, v);
              tmem_ld_wait();
#pragma unroll
              for (uint32_t e = 0; e < 4; ++e)
                if (c + e < a.heads) s0 = fmaf(weights[g * a.head_cols + c + e], max_nan(v[e], 0.0f), s0);
            }
          }
          float score = there && (int32_t)p < lens[g] ? (s0 + s1) * factor : -INFINITY;
          float* out = a.scores + (t0 + g) * a.ld;
          if (a.block_shift == 0) {
            if (p < a.n) out[p] = score;
            continue;
          }
          score = isnan(score) ? -INFINITY : score;
#pragma unroll
          for (uint32_t d = 0; d < 5; ++d)
            if (d < a.block_shift) score = fmaxf(score, __shfl_xor_sync(0xffffffffu, score, 1u << d));
          if (a.block_shift > 5) {
            const uint32_t warps = 1u << (a.block_shift - 5), w0 = (warp & 3) & ~(warps - 1);
            if (lane == 0) sh.best[team][warp & 3] = score;
            named_sync(1 + team, 128);
            for (uint32_t k = 0; k < warps; ++k) score = fmaxf(score, sh.best[team][w0 + k]);
            named_sync(1 + team, 128);
          }
          if ((key & ((1u << a.block_shift) - 1)) == 0 && p < a.n) out[p >> a.block_shift] = score;
        }
        tc_fence_before();
        mbar_arrive(&sh.acc_empty[acc]);                        // the accumulator has been read
      }
      while (kShared && sh.start[task + 1] < last) next_task();  // those that other teams have tiles of
    } else if (warp < kMmaWarp) {
      uint32_t next = turn0;                                    // this warp's next tile
      for (; next < S::kStages && next < mine; next += kLoadWarps) bring(next);
      for (; next < mine; next += kLoadWarps) {                 // the slot held tile next - kStages
        const bool ok = wait(&sh.empty[next % S::kStages], (next / S::kStages - 1) & 1);
        if (__any_sync(0xffffffffu, !ok)) break;
        bring(next);
      }
      if (lane == 0) sh.brought[turn0] = next;
    } else {
      // the whole warp walks along, one elected lane issues: what a converged
      // warp computes stays in the uniform registers that the MMAs read
      const uint32_t idesc = mma_desc(kF8 ? 0u : 1u, cols, false, false);
      const uint64_t keys = tile_desc(ring, 16), heads = tile_desc(queries, 16);
      const uint64_t next_half = (cols * 128) >> 4;
      uint32_t task = first_task, nth = 0;
      bool ok = wait(&sh.q_full, 0);
      for (uint32_t i = 0, slot = 0, slot_turn = 0, acc = 0, acc_turn = 0; i < mine; ++i) {
        if (behind(i, task)) {                                  // the next task: its queries replace these
          if (elect_one()) mma_commit(&sh.task_done);
          __syncwarp();
          walk(i, task);
          ok = ok && wait(&sh.q_full, ++nth & 1);
        }
        ok = ok && wait(&sh.full[slot], slot_turn & 1) &&
             (acc_turn == 0 || wait(&sh.acc_empty[acc], (acc_turn - 1) & 1));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint64_t tile = keys + slot * (S::kTileBytes >> 4);
        const uint32_t d = tmem + acc * cols;
        if (elect_one()) {
#pragma unroll
          for (uint32_t k = 0; k < S::kKeyBytes / 32; ++k) {    // 32 bytes of K per MMA
            const uint64_t da = tile + (k >> 2) * (kKeyTile * 128 >> 4) + (k & 3) * 2;
            const uint64_t db = heads + (k >> 2) * next_half + (k & 3) * 2;
            if (kF8)
              mma_f8(d, da, db, idesc, k > 0);
            else
              mma_bf16(d, da, db, idesc, k > 0);
          }
          mma_commit(&sh.empty[slot]);
          mma_commit(&sh.acc_full[acc]);
        }
        __syncwarp();
        if (++slot == S::kStages) slot = 0, ++slot_turn;
        if (++acc == a.accs) acc = 0, ++acc_turn;
      }
    }
    tc_fence_before();
    __syncthreads();
    // Where any wait gave up, whoever it was, what is in flight finishes before
    // the CTA ends and its memory is given back: the MMAs (the lane that issued
    // them commits), and the last tile that was brought to each slot.  (One
    // before it has landed: its product released the slot.)
    if (sh.gave_up) {
      if (tid == 0) atomicOr(a.status, kFlagTimeout);
      if (warp == kMmaWarp) {
        if (elect_one()) {
          mma_commit(&sh.drained);
          if (!landed(&sh.drained, 0)) atomicOr(a.status, kFlagInflight);
        }
      } else if (warp == kLoadWarp && lane < S::kStages) {
        uint32_t to = 0;                                        // past the last tile that was brought
        for (uint32_t w = 0; w < kLoadWarps; ++w) to = max(to, sh.brought[w]);
        for (uint32_t i = to; i-- > 0;)
          if (i % S::kStages == lane && i < sh.brought[i % kLoadWarps]) {
            if (!landed(&sh.full[lane], (i / S::kStages) & 1)) atomicOr(a.status, kFlagInflight);
            break;
          }
      }
      __syncthreads();
    }
  }
  __syncwarp();
  if (warp == kMmaWarp) tmem_free(tmem, a.tmem_cols);

  // columns that no token sees, in pieces of 64 tiles of a task, or of one tile, to the CTAs in turn
  constexpr uint32_t kPiece = kShared ? 64 : 1;
  const uint32_t per_tile = kKeyTile >> a.block_shift, tiles = (a.n + kKeyTile - 1) / kKeyTile;
  const uint32_t pieces = (tiles + kPiece - 1) / kPiece;
  for (uint64_t i = kShared ? blockIdx.x : first + mine * step; i < (uint64_t)tasks * pieces; i += gridDim.x) {
    const uint32_t r = kShared ? (uint32_t)(i / pieces) : 0, piece = (uint32_t)(i - (uint64_t)r * pieces);
    const uint32_t from = max(piece * kPiece, kShared ? sh.start[r + 1] - sh.start[r] : 0), to = min(tiles, (piece + 1) * kPiece);
    if (from >= to) continue;
    const uint32_t t0 = token_of(r), tokens = tokens_of(r);
    for (uint32_t g = 0; g < tokens; ++g)
      for (uint32_t c = from * per_tile + tid; c < to * per_tile; c += kScoreThreads)
        if ((uint64_t)c << a.block_shift < a.n) a.scores[(t0 + g) * a.ld + c] = -INFINITY;
  }
}

// The keys as a matrix of rows, in boxes of `run` rows of 128 bytes.
bool key_map(CUtensorMap* map, const void* keys, int64_t rows, uint32_t run, bool f8) {
  static const auto encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(f);
  }();
  if (!encode) return false;
  const cuuint64_t size[2] = {KVO_KEY_VALUES, (cuuint64_t)rows}, pitch[1] = {f8 ? 128u : 256u};
  const cuuint32_t box[2] = {f8 ? 128u : 64u, run}, every[2] = {1, 1};
  return encode(map, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                const_cast<void*>(keys), size, pitch, box, every, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kF8, bool kShared, bool kPadded>
cudaError_t launch_scores(const ScoreArgs& a, int64_t cache_rows, cudaStream_t stream) {
  using S = ScoreShape<kF8>;
  CUtensorMap map;
  if (!key_map(&map, a.cache.keys, cache_rows, a.run, kF8)) return cudaErrorInvalidValue;
  const size_t smem = 1024 + (size_t)S::kStages * S::kTileBytes + (size_t)kScoreMaxCols * S::kKeyBytes;
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!ready[dev & 63]) {
    e = cudaFuncSetAttribute(index_scores_kernel<kF8, kShared, kPadded>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    ready[dev & 63] = true;
  }
  // one CTA per SM; where shared tasks are cut into several rows of the grid,
  // two waves, for these may differ
  const uint32_t sms = (uint32_t)device_sms(), tiles = (a.n + kKeyTile - 1) / kKeyTile;
  const uint32_t rows = kShared ? (a.tasks + a.slice - 1) / a.slice : a.tasks;
  const uint64_t most = kShared ? (uint64_t)std::min(a.slice, a.tasks) * tiles : tiles;
  uint32_t x = kShared && rows > 1 ? (2 * sms + rows - 1) / rows : rows <= sms ? sms / rows : 1;
  if (x > most) x = (uint32_t)most;
  return launch_early(index_scores_kernel<kF8, kShared, kPadded>, dim3(x, rows), kScoreThreads, smem, stream, a, map);
}

}  // namespace
}  // namespace kvo

extern "C" kvo_status kvo_index_scores(kvo_ctx* ctx, const kvo_cache* cache, const kvo_score_query* s, void* stream) {
  using namespace kvo;
  uint32_t* status = nullptr;
  if (!ctx || !cache_ok(cache) || !s || !cache_keys_ok(cache)) return KVO_EINVAL;
  if (!s->q || !s->weights || !s->lens || !s->scores) return KVO_EINVAL;
  if (s->heads < 1 || s->heads > KVO_MAX_HEADS || s->per_seq < 1 || s->n < 1 || s->n > INT32_MAX - 255) return KVO_EINVAL;
  if (s->block < 1 || s->block > KVO_MAX_SCORE_BLOCK || (s->block & (s->block - 1))) return KVO_EINVAL;
  const int64_t nq = (int64_t)cache->sequences * s->per_seq;
  const int64_t size = cache->key_type == KVO_BF16 ? 2 : 1, rows = cache->blocks * cache->block_rows;
  if (rows > INT32_MAX) return KVO_EINVAL;
  if (nq > KVO_MAX_QUERIES || s->ld < (s->n + s->block - 1) / s->block) return KVO_EINVAL;
  if (!aligned(s->q, 16) || (s->q_ld * size) % 16 || (s->q_head_ld * size) % 16) return KVO_EINVAL;
  if (!aligned(s->weights, 4) || !aligned(s->lens, 4) || !aligned(s->scores, 4)) return KVO_EINVAL;
  int64_t wait_clocks = 0;
  const kvo_status st = usable_status(ctx, &status, &wait_clocks);
  if (st != KVO_OK) return st;

  ScoreArgs a = {};
  a.wait_clocks = wait_clocks;
  a.cache = cache_view(*cache);
  if (cache->key_type == KVO_BF16) a.cache.key_scales = nullptr;
  a.q = static_cast<const uint8_t*>(s->q);
  a.w = s->weights;
  a.lens = s->lens;
  a.scores = s->scores;
  a.status = status;
  a.q_ld = s->q_ld * size;
  a.q_head_ld = s->q_head_ld * size;
  a.w_ld = s->weights_ld;
  a.ld = s->ld;
  a.n = (uint32_t)s->n;
  a.per_seq = (uint32_t)s->per_seq;
  a.heads = (uint32_t)s->heads;
  while ((1 << a.block_shift) < s->block) ++a.block_shift;
  a.head_cols = (a.heads + 31u) & ~31u;
  a.group = kScoreMaxCols / a.head_cols;
  if (a.group > a.per_seq) a.group = a.per_seq;
  a.groups = (a.per_seq + a.group - 1) / a.group;
  a.by_groups = divider(a.groups);
  a.tasks = (uint32_t)cache->sequences * a.groups;
  // a row of the grid counts its tiles in 31 bits
  a.slice = (uint32_t)std::min<uint64_t>(kMostTasks, 0x7fffffffu / ((uint64_t)(a.n + kKeyTile - 1) / kKeyTile + kTaskCost));
  a.accs = a.group * a.head_cols > 128 ? 2 : 4;
  a.tmem_cols = 128;
  while (a.tmem_cols < a.accs * a.group * a.head_cols) a.tmem_cols *= 2;
  // the largest power of two that divides both a tile and a block; without a
  // table a sequence is one block.  A million e4m3 keys take 26.7 us in runs of
  // 16, 39.7 as gathered rows (blocks of 5).
  a.run = kKeyTile;
  while (cache->table && a.run > 1 && cache->block_rows % a.run) a.run /= 2;
  if (a.run < 4) a.run = 1;
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  // With one task to a row of the grid uneven lengths leave SMs idle, and more
  // than half as many tasks as SMs one CTA a task; tiles shared out cost a
  // lookup of their task at every step.  e4m3 keys of 64 heads, 8,192 a
  // sequence, a row each against shared, us: 48 sequences of uneven length 11.3,
  // 11.6, of equal length 11.6, 13.6; 100 uneven 25.7, 18.2, equal 26.6, 25.1;
  // 128 26.3, 22.5 and 28.8, 31.5; 200 47.5, 35.3 and 54.2, 46.5; 700 116, 114
  // and 142, 155.  2,000 of up to 300 keys 52.8, 41.8 and 57.5, 46.5.
  const uint32_t sms = (uint32_t)device_sms();
  const bool shared = 2 * a.tasks > sms && (a.tasks <= 2 * sms || a.n <= 16 * kKeyTile);
  const auto choose = [&](auto f8, auto is_shared) {
    return a.heads == a.head_cols ? launch_scores<f8.value, is_shared.value, false> : launch_scores<f8.value, is_shared.value, true>;
  };
  using No = std::false_type;
  using Yes = std::true_type;
  const auto launch = cache->key_type == KVO_BF16 ? shared ? choose(No{}, Yes{}) : choose(No{}, No{})
                                                  : shared ? choose(Yes{}, Yes{}) : choose(Yes{}, No{});
  const cudaError_t e = launch(a, rows, on);
  return e == cudaSuccess ? KVO_OK : KVO_ECUDA;
}
