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

// From the context (kvo_api.cu).  Its device status word and the clocks after
// which a wait gives up, for calls that keep no other state in it; KVO_EINVAL
// without a context, KVO_ECUDA for one that must not launch.
kvo_status usable_status(kvo_ctx* ctx, uint32_t** status, int64_t* wait_clocks = nullptr);

// Streaming multiprocessors of the current device (152 where none can be asked).
int device_sms();

// The operators' launches may be scheduled while the work before them on the
// stream still ends, and every thread waits here, before its first access to
// memory, until that has completed and is visible.  The launch after them may
// be scheduled once all their CTAs run.  Replayed from a graph that takes 0.2
// to 0.9 us off a call (one appended token 2.5 to 2.3, 50,023 scores 5.2 to
// 4.85, those of four tokens 8.25 to 7.7, in the form they had).
__device__ __forceinline__ void wait_previous_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_next_grid() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
inline cudaError_t launch_early(void (*kernel)(P...), dim3 grid, uint32_t threads, size_t smem, cudaStream_t stream,
                                const A&... args) {
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.gridDim = grid;
  lc.blockDim = dim3(threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = stream;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, static_cast<P>(args)...);
}

// The larger value; a NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Division of n < 2^31 by a fixed d >= 1 as a product: with s = ceil(log2 d)
// and m = floor(2^32 (2^s - d) / d) + 1, n / d = (n + (n m >> 32)) >> s, and
// the sum stays below 2^32.
struct Divider {
  uint32_t mul, shift;
};

inline Divider divider(uint32_t d) {
  uint32_t s = 0;
  while (((uint64_t)1 << s) < d) ++s;
  return Divider{(uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << s) - d)) / d + 1), s};
}

__host__ __device__ __forceinline__ uint32_t divide(uint32_t n, Divider by) {
  return (n + (uint32_t)((uint64_t)n * by.mul >> 32)) >> by.shift;
}

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
  Divider by_block;          // division by block_rows
};

inline CacheView cache_view(const kvo_cache& c) {
  return CacheView{static_cast<uint8_t*>(c.rows),  static_cast<uint8_t*>(c.keys), c.key_scales,
                   c.table,                        c.table_ld,                    c.blocks,
                   (uint32_t)c.block_rows,         (uint32_t)c.table_blocks,      (uint32_t)c.sequences,
                   divider((uint32_t)c.block_rows)};
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

// The block that position p (below 2^31) of sequence s (< sequences) lies in,
// as the table has it, unchecked; -1 where the table does not reach.  Apart
// from cache_row_in, so that a loop can ask for the entries of later
// positions and look at them only when they have come.
__host__ __device__ __forceinline__ int32_t cache_block(const CacheView& c, uint32_t s, uint32_t p) {
  const uint32_t b = divide(p, c.by_block);
  if (!c.table) return b == 0 ? (int32_t)s : -1;
  return b < c.table_blocks ? c.table[(int64_t)s * c.table_ld + b] : -1;
}

// The cache row of position p in block `id`, or -1 where there is no such
// block.  Rows are counted in 64 bits: a cache may hold more than 2^31.
__host__ __device__ __forceinline__ int64_t cache_row_in(const CacheView& c, int32_t id, uint32_t p) {
  if (id < 0 || id >= c.blocks) return -1;
  return (int64_t)id * c.block_rows + (p - divide(p, c.by_block) * c.block_rows);
}

// The cache row of position p of sequence s, or -1 where there is none.
__host__ __device__ __forceinline__ int64_t cache_row(const CacheView& c, uint32_t s, uint32_t p) {
  return cache_row_in(c, cache_block(c, s, p), p);
}

}  // namespace kvo
