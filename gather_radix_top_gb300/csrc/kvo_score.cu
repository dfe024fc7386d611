// kvo_index_scores: score[t][j] = s_j * sum_h w[t][h] * max(0, q[t][h] . key_j).
//
// Keys times queries is a matrix product with a reduction over its columns:
// a tile of 128 keys is the A operand (M = 128), the heads of up to 8 query
// tokens of one sequence are B (N = 32 .. 256 columns).  With the keys along M, a
// thread of the epilogue holds one key's products with every head, so the
// weighted sum over heads needs no exchange between threads, and the keys
// are read once for all query tokens of their sequence.
//
// One CTA per SM, each over every gridDim.x-th key tile of one group of
// query tokens: a warp brings key tiles into a ring in shared memory
// (a TMA box per run of keys of one block, looked up in the table), another
// issues the MMAs into accumulators in tensor memory, and four
// teams of four warps reduce them in turn.  Nothing but the queries and the
// scores passes through global memory twice.
//
// What bounds it: up to 128 columns, reading the keys (132 bytes a key as e4m3,
// 256 as bf16) after about 4 us of launch, queries and first keys: a million
// keys take 25.5 us as one run of e4m3 (5.4 TB/s), 27.5 in shuffled blocks of
// 16 and 42.1 as bf16 (6.4 TB/s), whether for 16 or 64 heads.  For 256
// columns (four tokens of 64 heads), the epilogue's two operations per
// product: 262,144 keys take 18.3 us against 9.3 for one token.  Slower ones, for
// the million in blocks: MMAs from one thread of a diverged warp 30.3 us (28.4
// by then), one loading warp alone 45.2 (it issues a box every 60 clocks), table
// entries that are used as soon as they are asked for 48.2.
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
  uint32_t accs;             // accumulators in tensor memory: 4, or 2 of more than 128 columns
  uint32_t tmem_cols;
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
  uint64_t full[8], empty[8], acc_full[4], acc_empty[4], drained;
  uint32_t tmem;
  uint32_t gave_up;
  int32_t len[kScoreMaxTokens];
  float best[kScoreTeams][4];
  float w[kScoreMaxCols];
};

template <bool kF8>
__global__ void __launch_bounds__(kScoreThreads, 1) index_scores_kernel(const __grid_constant__ ScoreArgs a,
                                                                        const __grid_constant__ CUtensorMap map) {
  using S = ScoreShape<kF8>;
  extern __shared__ uint8_t raw[];
  __shared__ ScoreShared sh;
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t seq = blockIdx.y / a.groups, g0 = (blockIdx.y % a.groups) * a.group;
  const uint32_t tokens = min(a.group, a.per_seq - g0);         // of this CTA
  const uint32_t t0 = seq * a.per_seq + g0;
  const uint32_t cols = a.group * a.head_cols;
  const uint32_t ring = smem_u32(smem), queries = ring + S::kStages * S::kTileBytes;

  wait_previous_grid();
  allow_next_grid();
  int32_t most = 0;                                             // positions that any of the tokens sees
  for (uint32_t g = 0; g < tokens; ++g) most = max(most, min(a.lens[t0 + g], (int32_t)a.n));
  const uint32_t tiles = ((uint32_t)most + kKeyTile - 1) / kKeyTile;
  const uint32_t step = gridDim.x, first = blockIdx.x;
  const uint32_t mine = tiles > first ? (tiles - first + step - 1) / step : 0;

  if (mine) {
    if (tid == 0) {
      for (uint32_t i = 0; i < S::kStages; ++i) {
        mbar_init(&sh.full[i], 1);
        mbar_init(&sh.empty[i], 1);
      }
      for (uint32_t i = 0; i < a.accs; ++i) {
        mbar_init(&sh.acc_full[i], 1);
        mbar_init(&sh.acc_empty[i], kScoreEpilogue / a.accs);
      }
      mbar_init(&sh.drained, 1);
      sh.gave_up = 0;
    }
    if (warp == kMmaWarp) tmem_alloc(&sh.tmem, a.tmem_cols);

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
    auto look_ahead = [&](uint32_t i) -> int4 {
      const uint32_t p = (first + i * step) * kKeyTile + width * lane;
      int32_t b[4] = {0, 0, 0, 0};
      if (i < mine && width * lane < kKeyTile) {
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k)
          if ((k == 0 || !runs) && p + k < (uint32_t)most) b[k] = cache_block(a.cache, seq, p + k);
      }
      return make_int4(b[0], b[1], b[2], b[3]);
    };
    auto bring = [&](uint32_t j) {
      const uint32_t slot = j % S::kStages, dst = ring + slot * S::kTileBytes + lane * width * 128;
      const uint32_t p = (first + j * step) * kKeyTile + width * lane;
      auto row = [&](int32_t id, uint32_t k) -> int32_t {
        return p + k < (uint32_t)most ? max(0, (int32_t)cache_row_in(a.cache, id, p + k)) : 0;
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
    // the barriers are ready, and so are the first tiles' places
    __syncthreads();
    uint32_t next = turn0;                                      // a loading warp's next tile
    if (loads) {
      for (; next < S::kStages && next < mine; next += kLoadWarps) bring(next);
    } else {
      const uint32_t at = warp < kLoadWarp ? tid : tid - 32 * kLoadWarps;
      for (uint32_t i = at; i < cols * S::kPieces; i += kScoreThreads - 32 * kLoadWarps) {
        const uint32_t r = i / S::kPieces, c = i % S::kPieces, g = r / a.head_cols, h = r - g * a.head_cols;
        const bool real = g < tokens && h < a.heads;
        copy16_async(queries + (c >> 3) * (cols * 128) + swizzled(r, c & 7),
                     real ? a.q + (t0 + g) * a.q_ld + h * a.q_head_ld + c * 16 : a.q, real);
      }
      copy_async_commit();
      for (uint32_t i = at; i < cols; i += kScoreThreads - 32 * kLoadWarps) {
        const uint32_t g = i / a.head_cols, h = i - g * a.head_cols;
        sh.w[i] = g < tokens && h < a.heads ? a.w[(t0 + g) * a.w_ld + h] : 0.0f;
      }
      if (at < tokens) sh.len[at] = min(a.lens[t0 + at], (int32_t)a.n);
      copy_async_wait<0>();
      fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    if (warp < kLoadWarp) {
      // team w takes the tiles of accumulator w % accs, and of their query
      // tokens every parts-th
      const uint32_t team = warp >> 2, acc = team % a.accs, part = team / a.accs, parts = kScoreTeams / a.accs;
      const uint32_t lane_base = (warp & 3) * 32, key = lane_base + lane;
      const uint32_t from = tmem + (lane_base << 16) + acc * cols;
      // table entries are asked for two of this team's tiles ahead, the keys'
      // factors one
      auto look_up = [&](uint32_t i) -> int32_t {
        const uint32_t p = (first + i * step) * kKeyTile + key;
        return i < mine && p < (uint32_t)most ? cache_block(a.cache, seq, p) : -1;
      };
      auto row_in = [&](uint32_t i, int32_t id) -> int64_t {
        return cache_row_in(a.cache, id, (first + i * step) * kKeyTile + key);
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
        const uint32_t p = (first + i * step) * kKeyTile + key;
        const bool there = next_there;
        const float factor = next_factor;
        if (!there && p < (uint32_t)most) atomicOr(a.status, kFlagRange);
        const int64_t r = row_in(i + a.accs, block_after);
        next_there = r >= 0;
        next_factor = factor_of(r);
        block_after = look_up(i + 2 * a.accs);
        // after a wait that gave up the team goes on through what it finds
        // (its warps meet at barriers below); the status says so
        wait_or_give_up(&sh.acc_full[acc], turn, &sh.gave_up);
        __syncwarp();
        tc_fence_after();
        for (uint32_t g = part; g < tokens; g += parts) {
          float s0 = 0.0f, s1 = 0.0f;
          for (uint32_t c = 0; c < a.head_cols; c += 32) {
            float v[32];
            tmem_ld32(from + g * a.head_cols + c, v);
            const float4* w4 = reinterpret_cast<const float4*>(&sh.w[g * a.head_cols + c]);
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
          float score = there && (int32_t)p < sh.len[g] ? (s0 + s1) * factor : -INFINITY;
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
    } else if (warp < kMmaWarp) {
      for (; next < mine; next += kLoadWarps) {                 // the slot held tile next - kStages
        const bool ok = wait_or_give_up(&sh.empty[next % S::kStages], (next / S::kStages - 1) & 1, &sh.gave_up);
        if (__any_sync(0xffffffffu, !ok)) break;
        bring(next);
      }
      // where the CTA gives up, the copies in flight finish before it ends
      // (the last tile of each slot that this warp has brought)
      if (next < mine)
        for (uint32_t i = next < S::kStages + kLoadWarps ? turn0 : next - S::kStages; i < next; ++i)
          if ((i - turn0) % kLoadWarps == 0 && !landed(&sh.full[i % S::kStages], (i / S::kStages) & 1))
            atomicOr(a.status, kFlagInflight);
    } else {
      // the whole warp walks along, one elected lane issues: what a converged
      // warp computes stays in the uniform registers that the MMAs read
      const uint32_t idesc = mma_desc(kF8 ? 0u : 1u, cols, false, false);
      const uint64_t keys = tile_desc(ring, 16), heads = tile_desc(queries, 16);
      const uint64_t next_half = (cols * 128) >> 4;
      bool ok = true;
      for (uint32_t i = 0, slot = 0, slot_turn = 0, acc = 0, acc_turn = 0; i < mine; ++i) {
        ok = wait_or_give_up(&sh.full[slot], slot_turn & 1, &sh.gave_up) &&
             (acc_turn == 0 || wait_or_give_up(&sh.acc_empty[acc], (acc_turn - 1) & 1, &sh.gave_up));
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
      if (!ok && elect_one()) {
        // let the MMAs in flight finish before their memory is given back
        mma_commit(&sh.drained);
        atomicOr(a.status, kFlagTimeout);
        if (!landed(&sh.drained, 0)) atomicOr(a.status, kFlagInflight);
      }
      __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && sh.gave_up) atomicOr(a.status, kFlagTimeout);
    __syncwarp();
    if (warp == kMmaWarp) tmem_free(tmem, a.tmem_cols);
  }

  // columns that no token sees
  const uint32_t per_tile = kKeyTile >> a.block_shift;
  for (uint32_t t = first + mine * step; (uint64_t)t * kKeyTile < a.n; t += step)
    for (uint32_t i = tid; i < per_tile * tokens; i += kScoreThreads) {
      const uint32_t g = i / per_tile, c = t * per_tile + i % per_tile;
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

template <bool kF8>
cudaError_t launch_scores(const ScoreArgs& a, int64_t cache_rows, uint32_t sequences, cudaStream_t stream) {
  using S = ScoreShape<kF8>;
  CUtensorMap map;
  if (!key_map(&map, a.cache.keys, cache_rows, a.run, kF8)) return cudaErrorInvalidValue;
  const size_t smem = 1024 + (size_t)S::kStages * S::kTileBytes + (size_t)kScoreMaxCols * S::kKeyBytes;
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!ready[dev & 63]) {
    e = cudaFuncSetAttribute(index_scores_kernel<kF8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    ready[dev & 63] = true;
  }
  // one CTA per SM where the groups allow it in one wave, else several waves
  // of shorter ones, so that uneven lengths even out
  const uint32_t rows = sequences * a.groups, sms = (uint32_t)device_sms(), tiles = (a.n + kKeyTile - 1) / kKeyTile;
  uint32_t x = rows <= sms ? sms / rows : (4 * sms + rows - 1) / rows;
  if (x > tiles) x = tiles;
  return launch_early(index_scores_kernel<kF8>, dim3(x, rows), kScoreThreads, smem, stream, a, map);
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
  const kvo_status st = usable_status(ctx, &status);
  if (st != KVO_OK) return st;

  ScoreArgs a = {};
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
  a.accs = a.group * a.head_cols > 128 ? 2 : 4;
  a.tmem_cols = 128;
  while (a.tmem_cols < a.accs * a.group * a.head_cols) a.tmem_cols *= 2;
  // the largest power of two that divides both a tile and a block; without a
  // table a sequence is one block.  A million e4m3 keys take 27.5 us in runs of
  // 16, 41.3 as gathered rows (blocks of 5).
  a.run = kKeyTile;
  while (cache->table && a.run > 1 && cache->block_rows % a.run) a.run /= 2;
  if (a.run < 4) a.run = 1;
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->key_type == KVO_BF16 ? launch_scores<false>(a, rows, (uint32_t)cache->sequences, on)
                                                    : launch_scores<true>(a, rows, (uint32_t)cache->sequences, on);
  return e == cudaSuccess ? KVO_OK : KVO_ECUDA;
}
