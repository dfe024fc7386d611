// What the operators on a kvo_cache share: where a position's row is, and the
// host-side checks of a cache description.
#pragma once

#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "kvo.h"
#include "kvo_device.cuh"
#include "kvo_internal.h"

namespace kvo {

// kvo_cache as kernels take it (by value, in the parameter space).
struct CacheView {
  uint8_t* rows;
  uint8_t* keys;
  float* key_scales;
  const int32_t* __restrict__ table;
  int64_t table_ld;
  int64_t blocks;
  uint32_t block_rows;
  uint32_t table_blocks;
  uint32_t sequences;
};

inline CacheView cache_view(const kvo_cache& c) {
  return CacheView{static_cast<uint8_t*>(c.rows),  static_cast<uint8_t*>(c.keys), c.key_scales,
                   c.table,                        c.table_ld,                    c.blocks,
                   (uint32_t)c.block_rows,         (uint32_t)c.table_blocks,      (uint32_t)c.sequences};
}

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The table geometry and the parts that every call needs.
inline bool cache_ok(const kvo_cache* c) {
  if (!c || c->block_rows < 1 || c->blocks < 1 || c->blocks > INT32_MAX || c->sequences < 1) return false;
  if (c->blocks > INT64_MAX / KVO_ROW_BYTES / c->block_rows) return false;
  if (!c->table) return c->sequences <= c->blocks;
  return aligned(c->table, 4) && c->table_blocks >= 0 && c->table_ld >= c->table_blocks;
}

inline bool cache_rows_ok(const kvo_cache* c) { return c->rows && aligned(c->rows, 16); }

inline bool cache_keys_ok(const kvo_cache* c) {
  if (!c->keys || !aligned(c->keys, 16)) return false;
  if (c->key_type == KVO_BF16) return true;
  return c->key_type == KVO_E4M3 && c->key_scales && aligned(c->key_scales, 4);
}

// The cache row of position p (>= 0) of sequence s (< sequences), or -1 where
// there is none.  Rows are counted in 64 bits: a cache may hold more than
// 2^31 of them.
__host__ __device__ __forceinline__ int64_t cache_row(const CacheView& c, uint32_t s, uint32_t p) {
  const uint32_t b = p / c.block_rows;
  const uint32_t r = p - b * c.block_rows;
  if (!c.table) return b == 0 ? (int64_t)s * c.block_rows + r : -1;
  if (b >= c.table_blocks) return -1;
  const int32_t id = c.table[(int64_t)s * c.table_ld + b];
  if (id < 0 || id >= c.blocks) return -1;
  return (int64_t)id * c.block_rows + r;
}

}  // namespace kvo
