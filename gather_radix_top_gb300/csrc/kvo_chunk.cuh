// What the calls on chunks of new tokens share: which columns a CTA has.
//
// The tokens of all sequences lie one after the other, sequence s's at
// [starts[s], starts[s + 1]).  A chunk's (token, head) pairs, the heads of a
// token next to each other, are cut into tiles of columns; a tile holds
// columns of one sequence only.
#pragma once

#include <cuda.h>

#include "kvo_cache.cuh"

namespace kvo {

struct ChunkTile {
  int32_t seq;               // -1: there is no such tile
  uint32_t index;            // of its sequence's tiles
  uint32_t first, tokens;    // the sequence's tokens
};

// Sequence s's tokens; starts outside the tokens, or that go back, count as the
// nearest ones that do not (`bad`).
struct Tokens {
  uint32_t first, count;
  bool bad;
};
__device__ __forceinline__ Tokens tokens_of(const int32_t* starts, uint32_t s, uint32_t tokens) {
  const int32_t b = starts[s], e = starts[s + 1], all = (int32_t)tokens, first = min(max(b, 0), all);
  return Tokens{(uint32_t)first, (uint32_t)(min(max(e, first), all) - first), b < 0 || b > all || e < b || e > all};
}

// Tiles that a call's sequences can have at most: their last ones may be part.
inline uint32_t chunk_tiles(int64_t tokens, int64_t sequences, int64_t heads, int64_t columns) {
  const int64_t busy = sequences < tokens ? sequences : tokens;
  return (uint32_t)((tokens * heads + busy * (columns - 1)) / columns);
}

// Tile `at` of the call, found by every warp for itself, 32 sequences at a
// time.  Starts outside the tokens, or that go back, count as the nearest ones
// that do not, and latch KVO_ERANGE.
__device__ __forceinline__ ChunkTile chunk_tile(const int32_t* starts, uint32_t sequences, uint32_t tokens, uint32_t heads,
                                                uint32_t columns, uint32_t at, uint32_t* status) {
  const uint32_t lane = threadIdx.x & 31;
  uint32_t before = 0;                                   // tiles of the sequences before these 32
  for (uint32_t s0 = 0; s0 < sequences; s0 += 32) {
    const uint32_t s = s0 + lane;
    const int32_t b = s < sequences ? starts[s] : 0, e = s < sequences ? starts[s + 1] : 0;
    const uint32_t first = (uint32_t)min(max(b, 0), (int32_t)tokens);
    const uint32_t end = (uint32_t)min(max(e, (int32_t)first), (int32_t)tokens);
    if (b < 0 || b > (int32_t)tokens || e < b || e > (int32_t)tokens) atomicOr(status, kFlagRange);
    const uint32_t tiles = ((end - first) * heads + columns - 1) / columns;
    uint32_t upto = tiles;
#pragma unroll
    for (uint32_t d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + upto > at);
    if (past) {
      const int from = __ffs((int)past) - 1;
      ChunkTile t;
      t.seq = (int32_t)(s0 + from);
      t.index = at - before - __shfl_sync(0xffffffffu, upto - tiles, from);
      t.first = __shfl_sync(0xffffffffu, first, from);
      t.tokens = __shfl_sync(0xffffffffu, end - first, from);
      return t;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return ChunkTile{-1, 0, 0, 0};
}

// How a chunk's columns fill tiles of `size`.  Where a token's heads and the
// tokens themselves are evenly spaced, all (token, head) pairs are one run; else a
// tile is `wide` heads of `deep` tokens.
struct Columns {
  uint32_t flat;             // 1: one run
  uint32_t wide, deep;       // wide * deep <= size columns
  uint32_t across;           // tiles across the heads
  Divider by_wide;
};
constexpr uint32_t kColumns = 64;
constexpr int64_t kMaxQueryLd = (int64_t)1 << 38;         // elements: strides of a tensor map end at 2^40 bytes

inline Columns columns_of(uint32_t heads, int64_t q_ld, int64_t q_head_ld, int64_t tokens, uint32_t size = kColumns) {
  Columns c = {};
  c.flat = tokens == 1 || q_ld == heads * q_head_ld;
  c.wide = c.flat ? 1 : heads < size ? heads : size;
  c.deep = size / c.wide;
  c.across = c.flat ? 1 : (heads + c.wide - 1) / c.wide;
  c.by_wide = divider(c.wide);
  return c;
}

inline decltype(&cuTensorMapEncodeTiled) map_encoder() {
  static const auto encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(f);
  }();
  return encode;
}

// The queries as boxes of 64 values of a tile's columns; strides in bytes.
inline bool query_map(CUtensorMap* map, const void* q, uint32_t heads, int64_t tokens, int64_t q_ld, int64_t q_head_ld,
                      const Columns& c) {
  const auto encode = map_encoder();
  if (!encode) return false;
  const cuuint64_t size[3] = {KVO_DEQUANT_VALUES, c.flat ? 1 : (cuuint64_t)heads,
                              (cuuint64_t)(c.flat ? tokens * heads : tokens)};
  const cuuint64_t pitch[2] = {(cuuint64_t)q_head_ld, (cuuint64_t)(c.flat ? q_head_ld : q_ld)};
  const cuuint32_t box[3] = {64, c.wide, c.deep}, every[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), size, pitch, box, every,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Unpacked rows as groups of 64 values, in boxes of `deep` rows of `groups`
// groups, the groups one behind the other.
inline bool value_map(CUtensorMap* map, const void* values, int64_t rows, uint32_t deep, uint32_t groups) {
  const auto encode = map_encoder();
  if (!encode) return false;
  const cuuint64_t size[3] = {64, (cuuint64_t)rows, KVO_DEQUANT_VALUES / 64}, pitch[2] = {KVO_DEQUANT_VALUES * 2, 128};
  const cuuint32_t box[3] = {64, deep, groups}, every[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(values), size, pitch, box, every,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries that query_map can describe; strides in elements.
inline bool query_ok(const void* q, int64_t q_ld, int64_t q_head_ld, int64_t tokens, int64_t heads) {
  if (!q || !aligned(q, 16) || q_ld % 8 || q_head_ld % 8) return false;
  if (tokens > 1 && (q_ld < KVO_DEQUANT_VALUES || q_ld >= kMaxQueryLd)) return false;
  return heads <= 1 || (q_head_ld >= KVO_DEQUANT_VALUES && q_head_ld < kMaxQueryLd);
}

}  // namespace kvo
