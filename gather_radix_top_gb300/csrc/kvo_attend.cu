// kvo_attend: softmax attention of absorbed MLA queries over cached rows.
//
// One CTA holds up to 64 heads of one query and walks over tiles of 80 or 96
// rows of its list.  Whole 656-byte rows come into shared memory by bulk
// copies, are dequantised once to bf16 in the tensor cores' layout, and both
// products take the rows' operand as A:
//     S^T [rows x heads]       = K [rows x 576] Q^T         (K contiguous)
//     O^T [512 values x heads] += V^T [512 x rows] P^T      (the same bytes, read
//                                along the other dimension, as 4 x 128 values)
// With the heads as columns the accumulators fit: O^T needs 4 x 64 of the 512
// columns of tensor memory, which 128 heads by 512 values as rows would fill,
// and M is full for few heads too.  Shared memory holds the queries (72 KB for
// 64 heads), one dequantised tile (90 KB for 80 rows) and the next tile's raw
// rows (55 KB).  P^T takes the place of the position part, which the second
// product does not read.
//
// Sixteen worker warps dequantise and do the softmax, three warps bring rows,
// one issues the MMAs.  A tile goes through in two parts of 256 values: a part
// is dequantised as soon as the second product of the last tile has released
// its place, and multiplied while the other part is dequantised.
//
// The softmax is over the lanes of S^T.  Its reference is not the running
// maximum but the maximum at some earlier tile: weights of up to 2^64 lose
// nothing in fp32 and bf16 (sums of 2^31 of them times the largest latent stay
// below 2^119), so a column's maximum over four warps is formed for the first
// tile and again only when a logit lies 2^64 above the reference.  The sum of
// the weights stays in registers, per lane, and is reduced once at the end.
//
// Long lists with few queries are split over CTAs, whose normalised partial
// results a second launch joins by their log-sum-exps.
//
// What bounds it.  A tile of 80 rows and 64 heads takes 2.85 us (5,700 clocks),
// of which the MMAs are 2,700: with 64 columns they are bound by shared memory
// (48 clocks each, 65 with 128 columns), which the dequantised tile's stores
// (720), the raw rows (820) and the queries share.  The softmax (about 1,450
// from scores to weights) and the hand-overs are the rest: with one tile in
// shared memory nothing else of the tensor cores' work can run beside it.
//     1,048,576 rows of one query with 128 heads                480 us, 608 TFLOP/s
//     64 queries of 64 heads, each with 2,048 listed positions   50.6 us, 1.9 TB/s
//     2,048 rows of one query with 64 heads                      9.8 us
// Measured on the way, the first of them in us: rows through registers 942
// (next to this much shared memory the SM keeps about 28 KB of loads in
// flight), eight worker warps and one loading warp 672, three loading warps
// 647, references that move seldom and MMAs issued by one elected lane of a
// converged warp 525 (by a divergent thread 664), two parts instead of five
// 501, multiply-adds on fp16 operands in the dequantisation 491.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kvo_cache.cuh"
#include "kvo_tc.cuh"

namespace kvo {
namespace {

constexpr uint32_t kWorkerWarps = 16;                    // four for each quarter of the columns
constexpr uint32_t kMmaWarp = kWorkerWarps;
constexpr uint32_t kLoadWarp = kMmaWarp + 1, kLoadWarps = 3;   // a warp issues a row's copy every 60 clocks
constexpr uint32_t kAttendThreads = (kLoadWarp + kLoadWarps) * 32;
constexpr uint32_t kPitch = 704;                         // of a raw row: an even and an odd row's halves of a store
                                                         // phase fall into different banks

// kHeads: columns of a CTA, 16, 32 or 64.
template <uint32_t kHeads>
struct AttendShape {
  // rows of a tile: what the queries leave room for, raw and dequantised
  static constexpr uint32_t kRows = kHeads == 64 ? 80 : 96;
  static constexpr uint32_t kPasses = (kRows + 63) / 64;           // of 64 rows, the last one maybe part
  static constexpr uint32_t kChunkBytes = kRows * 128;             // 64 values of every row
  static constexpr uint32_t kTileBytes = 9 * kChunkBytes;
  static constexpr uint32_t kQueryBytes = 9 * kHeads * 128;
  static constexpr uint32_t kSmem = 1024 + kTileBytes + kQueryBytes + kRows * kPitch;
  static constexpr uint32_t kTmemCols = kHeads == 64 ? 512 : kHeads == 32 ? 256 : 128;
};
constexpr float kFar = 64.0f;                            // in powers of two
constexpr int64_t kLeastRows = 64;                       // of a split
constexpr float kLog2e = 1.4426950408889634f;

struct AttendArgs {
  CacheView cache;
  const uint8_t* q;
  const int32_t* lens;
  const int32_t* sel;
  uint16_t* out;
  float* lse;
  float* part;               // [splits][queries * heads][512], with several splits
  float* part_lse;           // [splits][queries * heads], base 2
  uint32_t* status;
  int64_t q_ld, q_head_ld;   // bytes
  int64_t sel_ld;
  uint32_t rows, picked, sel_shift;
  uint32_t per_seq, heads, nq;
  uint32_t head_tiles, splits;
  float scale;               // times log2(e)
  int64_t wait_clocks;       // after which a wait gives up
};

struct AttendShared {
  uint64_t k_full[2], s_full, p_full, pv_done[2], voted[4], met[4], raw_full, raw_empty, drained;
  uint32_t tmem;
  uint32_t gave_up;
  uint32_t brought[kLoadWarps];      // per loading warp: tiles whose rows it has brought
  uint32_t there[2][kLoadWarps];     // tile i's rows that are not masked, in i % 2: row r is bit r / 3 of word r % 3
  uint32_t far[2][4];                // per quarter of the columns, in i % 2: tile i needs new references
  float top[4][4][16];               // per quarter of the columns and warp
  float column[kWorkerWarps][16];    // per warp: one value per column
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The fp16 value of a half of `two`, times an fp16, plus an fp32: exact before
// the one rounding to fp32.
__device__ __forceinline__ float fma_low(uint32_t two, uint16_t b, float c) {
  float r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n fma.rn.f32.f16 %0, l, %2, %3;\n}" : "=f"(r) : "r"(two), "h"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float fma_high(uint32_t two, uint16_t b, float c) {
  float r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n fma.rn.f32.f16 %0, h, %2, %3;\n}" : "=f"(r) : "r"(two), "h"(b), "f"(c));
  return r;
}

// Four int8 times a scale as bf16, rounded once.  A byte (plus 128) under the
// byte 0x64 is the fp16 1024 + byte; times the scale, minus (1024 + 128) *
// scale (exact: 4 and 11 bits), that is the exact product.
__device__ __forceinline__ void dequant4(uint32_t bytes, uint16_t scale, float bias, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = bytes ^ 0x80808080u;
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140u), b = __byte_perm(u, 0x64646464u, 0x4342u);
  lo = bf16_pair(fma_low(a, scale, bias), fma_high(a, scale, bias));
  hi = bf16_pair(fma_low(b, scale, bias), fma_high(b, scale, bias));
}

// One arrival for the whole warp, after all its lanes' accesses.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, uint32_t lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Sums of kN columns over the warp's lanes: a step with `kBit` halves the
// columns that a lane keeps, and once one is left adds the lanes' shares.
// v[0] is then column lane / (32 / kN)'s sum.
template <uint32_t kN, uint32_t kBit>
__device__ __forceinline__ void lane_sums(float* v, uint32_t lane) {
  if constexpr (kN > 1) {
    const bool up = lane & kBit;
#pragma unroll
    for (uint32_t c = 0; c < kN / 2; ++c) {
      const float keep = up ? v[c + kN / 2] : v[c], give = up ? v[c] : v[c + kN / 2];
      v[c] = keep + __shfl_xor_sync(0xffffffffu, give, kBit);
    }
  } else {
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], kBit);
  }
  if constexpr (kBit > 1) lane_sums<(kN > 1 ? kN / 2 : 1), kBit / 2>(v, lane);
}

// f(0), f(1), .. f(kN - 1), each with its index as a constant.
template <uint32_t kN, uint32_t kI = 0, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (kI < kN) {
    f(std::integral_constant<uint32_t, kI>{});
    static_for<kN, kI + 1>(f);
  }
}

template <uint32_t kCols>
__device__ __forceinline__ void tmem_ld_cols(uint32_t addr, float* v) {
  if constexpr (kCols == 16)
    tmem_ld16(addr, v);
  else if constexpr (kCols == 8)
    tmem_ld8(addr, v);
  else
    tmem_ld4(addr, v);
}

template <uint32_t kHeads>
__global__ void __launch_bounds__(kAttendThreads, 1) attend_kernel(const __grid_constant__ AttendArgs a) {
  using S = AttendShape<kHeads>;
  constexpr uint32_t kRows = S::kRows, kChunkBytes = S::kChunkBytes;
  constexpr uint32_t kCols = kHeads / 4;                 // of a worker warp
  constexpr uint32_t kScores = 4 * kHeads;               // S^T's first column
  extern __shared__ uint8_t raw[];
  __shared__ AttendShared sh;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t t = blockIdx.y, seq = t / a.per_seq;
  const uint32_t h0 = (blockIdx.x % a.head_tiles) * kHeads, split = blockIdx.x / a.head_tiles;
  const uint32_t tile_at = (smem_u32(raw) + 1023u) & ~1023u, queries = tile_at + S::kTileBytes;
  const uint32_t stage = queries + S::kQueryBytes;

  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return wait_or_give_up(bar, parity, &sh.gave_up, a.wait_clocks);
  };

  wait_previous_grid();
  allow_next_grid();
  const int32_t len = a.lens[t];
  // this CTA's entries of the list: from `first` on, `count` of them.  (With a
  // list nothing here waits for len: an empty query finds all of it masked.)
  const uint32_t all = a.sel ? a.picked << a.sel_shift : len <= 0 ? 0u : min((uint32_t)len, a.rows);
  const uint32_t share = (all + a.splits - 1) / a.splits;
  const uint32_t per = share > kRows ? (share + kRows - 1) / kRows * kRows : (share + 15u) & ~15u;
  const uint32_t first = (uint32_t)min((uint64_t)split * per, (uint64_t)all), count = min(per, all - first);
  const uint32_t tiles = (count + kRows - 1) / kRows;
  // rows of tile i that may be there, rounded up to a step of the second
  // product; a tile's other rows are not touched
  auto rows_of = [&](uint32_t i) -> uint32_t { return (min(kRows, count - i * kRows) + 15u) & ~15u; };

  // a worker warp's columns: heads h0 + quarter * kCols + c; its lanes: rows (or
  // values of O^T) quad * 32 + lane
  const uint32_t quad = warp & 3, quarter = (warp >> 2) & 3;
  const uint32_t head = h0 + quarter * kCols;
  const uint32_t mine = a.heads > head ? min(kCols, a.heads - head) : 0;   // real columns

  if (tiles == 0) {
    if (warp >= kWorkerWarps) return;
    const int64_t out_row = (int64_t)t * a.heads + head;
    if (a.splits > 1) {                                  // the join skips it
      if (quad == 0 && lane < mine) a.part_lse[(int64_t)split * a.nq * a.heads + out_row + lane] = -INFINITY;
      return;
    }
    for (uint32_t c = 0; c < mine; ++c)
      for (uint32_t d = quad * 32 + lane; d < KVO_LATENT_BYTES; d += 128) a.out[(out_row + c) * KVO_LATENT_BYTES + d] = 0;
    if (a.lse && quad == 0 && lane < mine) a.lse[out_row + lane] = -INFINITY;
    return;
  }

  if (tid == 0) {
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(&sh.k_full[i], kWorkerWarps);
      mbar_init(&sh.pv_done[i], 1);
    }
    for (uint32_t i = 0; i < 4; ++i) {
      mbar_init(&sh.voted[i], 4);
      mbar_init(&sh.met[i], 4);
    }
    mbar_init(&sh.s_full, 1);
    mbar_init(&sh.p_full, kWorkerWarps);
    mbar_init(&sh.raw_full, kLoadWarps);
    mbar_init(&sh.raw_empty, kWorkerWarps);
    mbar_init(&sh.drained, 1);
    for (uint32_t i = 0; i < 8; ++i) sh.far[i >> 2][i & 3] = 0;
    sh.gave_up = a.wait_clocks == 0;
  }
  if (warp == kMmaWarp) tmem_alloc(&sh.tmem, S::kTmemCols);
  __syncthreads();

  if (warp >= kLoadWarp) {
    // Lane l of loading warp w brings row 3 l + w of a tile.  Where it is, is
    // looked up in three steps, one tile apart, so that none waits for the one
    // before: the list's entry (tile i + 3), the table's (i + 2), the row
    // (i + 1).  A masked row becomes zeros.
    const uint32_t load = warp - kLoadWarp, r = kLoadWarps * lane + load;
    const uint32_t sub = (1u << a.sel_shift) - 1;
    auto listed = [&](uint32_t i) -> int32_t {           // the list's entry, unchecked
      const uint32_t j = first + i * kRows + r;
      if (i >= tiles || i * kRows + r >= count || r >= kRows) return -1;
      return a.sel ? a.sel[t * a.sel_ld + (j >> a.sel_shift)] : (int32_t)j;
    };
    auto position = [&](uint32_t i, int32_t unit) -> int32_t {   // or -1: masked
      const int64_t p = a.sel ? ((int64_t)unit << a.sel_shift) + ((first + i * kRows + r) & sub) : (int64_t)unit;
      return unit >= 0 && p < len ? (int32_t)p : -1;
    };
    auto block_of = [&](int32_t p) -> int32_t { return p >= 0 ? cache_block(a.cache, seq, (uint32_t)p) : -1; };
    auto row_of = [&](int32_t p, int32_t block) -> int64_t {
      if (p < 0) return -1;
      const int64_t found = cache_row_in(a.cache, block, (uint32_t)p);
      if (found < 0) atomicOr(a.status, kFlagRange);
      return found;
    };
    int32_t unit = listed(0), pos = listed(1);
    const int32_t unit2 = listed(2), pos0 = position(0, unit);
    pos = position(1, pos);
    int32_t block = block_of(pos);
    int64_t row = row_of(pos0, block_of(pos0));
    unit = unit2;
    const uint32_t dst = stage + r * kPitch;
    uint32_t i = 0;
    for (; i < tiles; ++i) {                             // (the workers let go of a tile only once all of it has come)
      const bool ok = i == 0 || wait(&sh.raw_empty, (i - 1) & 1);
      if (!__all_sync(0xffffffffu, ok)) break;
      const uint32_t there = __ballot_sync(0xffffffffu, row >= 0);
      if (row < 0 && r < rows_of(i)) {
        for (uint32_t c = 0; c < KVO_ROW_BYTES / 16; ++c) sts16(dst + 16 * c, make_uint4(0, 0, 0, 0));
        fence_proxy_async_smem();                        // before a later tile's copy to the same place
      }
      __syncwarp();
      if (lane == 0) {
        sh.there[i & 1][load] = there;
        mbar_arrive_expect_tx(&sh.raw_full, __popc(there) * KVO_ROW_BYTES);
      }
      __syncwarp();
      if (row >= 0) bulk_copy_g2s(raw + (dst - smem_u32(raw)), a.cache.rows + row * KVO_ROW_BYTES, KVO_ROW_BYTES, &sh.raw_full);
      row = row_of(pos, block);
      pos = position(i + 2, unit);
      block = block_of(pos);
      unit = listed(i + 3);
    }
    if (lane == 0) sh.brought[load] = i;
  } else {
    // the queries: heads past the last are zeros
    for (uint32_t i = tid; i < kHeads * 72; i += kLoadWarp * 32) {
      const uint32_t r = i / 72, c = i - r * 72;
      const bool real = h0 + r < a.heads;
      copy16_async(queries + (c >> 3) * (kHeads * 128) + swizzled(r, c & 7),
                   real ? a.q + t * a.q_ld + (h0 + r) * a.q_head_ld + c * 16 : a.q, real);
    }
    copy_async_commit();
    copy_async_wait<0>();
    fence_proxy_async_smem();
    tc_fence_before();
    named_sync(5, kLoadWarp * 32);
    tc_fence_after();
  }
  const uint32_t tmem = sh.tmem;

  if (warp < kWorkerWarps) {
    // A thread's part of a tile: 16-byte piece `piece` (of each 128 latent
    // bytes) of rows slot + 64 u.  A warp takes 128 consecutive bytes of four
    // rows at a time; the eight lanes of a store phase hold an even and an odd
    // row, whose swizzled pieces fall into different banks.
    const uint32_t piece = ((lane >> 3) & 1) * 4 + (lane & 3);
    const uint32_t slot = warp * 4 + (lane >> 4) * 2 + ((lane >> 2) & 1);
    // rows 64 apart have the same swizzle: everything else is a fixed offset
    const uint32_t to_lo = tile_at + (piece >> 2) * kChunkBytes + swizzled(slot, 2 * (piece & 3));
    const uint32_t to_hi = tile_at + (piece >> 2) * kChunkBytes + swizzled(slot, 2 * (piece & 3) + 1);
    const uint32_t to_rope = tile_at + 8 * kChunkBytes + swizzled(slot, piece);
    const uint32_t from = stage + slot * kPitch;

    const uint32_t mine_row = quad * 32 + lane;          // of S^T
    if (lane < kCols) sh.column[warp][lane] = 0.0f;
    __syncwarp();
    uint32_t meets = 0;                                  // times the references have moved
    bool unset = true;                                   // some column has no reference yet
    float top = -INFINITY;                               // lane c < kCols: column c's reference
    float sum[kCols];
#pragma unroll
    for (uint32_t c = 0; c < kCols; ++c) sum[c] = 0.0f;
    const uint32_t lanes = tmem + (quad << 21);          // (quad * 32) << 16

    bool come = true;                                    // every tile's rows so far
    for (uint32_t i = 0; i < tiles; ++i) {
      const uint32_t turn = i & 1;
      const uint32_t rows = rows_of(i);
      // the raw rows to bf16, part by part, as the products of the last tile
      // release their places; the second half of them is in registers, and the
      // next rows may come, before its places are free
      come &= wait(&sh.raw_full, turn);
      const bool there =
          mine_row < rows && (sh.there[turn][mine_row % kLoadWarps] >> (mine_row / kLoadWarps) & 1);
      uint32_t scales[S::kPasses][2];                    // this piece's scale of each part, as fp16 pairs
#pragma unroll
      for (uint32_t u = 0; u < S::kPasses; ++u)
        if (slot + 64 * u < rows) {
          const uint4 eight = lds16(from + u * (64 * kPitch) + KVO_LATENT_BYTES);
          scales[u][0] = __byte_perm(eight.x, eight.y, piece >= 4 ? 0x7632u : 0x5410u);
          scales[u][1] = __byte_perm(eight.z, eight.w, piece >= 4 ? 0x7632u : 0x5410u);
        }
#pragma unroll
      for (uint32_t part = 0; part < 2; ++part) {
        uint4 lat[2][S::kPasses], rope[S::kPasses];
#pragma unroll
        for (uint32_t u = 0; u < S::kPasses; ++u)
          if (slot + 64 * u < rows) {
            const uint32_t p = from + u * (64 * kPitch) + 16 * piece + 256 * part;
            lat[0][u] = lds16(p);
            lat[1][u] = lds16(p + 128);
            if (part) rope[u] = lds16(p - 256 + KVO_LATENT_BYTES + 16);
          }
        if (part) {                                        // after a wait that gave up the next rows must not come
          __syncwarp();
          if (lane == 0 && come) mbar_arrive(&sh.raw_empty);
        }
        if (i > 0) wait(&sh.pv_done[part], turn ^ 1);
#pragma unroll
        for (uint32_t k = 0; k < 2; ++k) {
#pragma unroll
          for (uint32_t u = 0; u < S::kPasses; ++u) {
            if (slot + 64 * u >= rows) break;
            const uint16_t s = (uint16_t)(scales[u][part] >> k * 16);
            const float bias = -1152.0f * __half2float(__ushort_as_half(s));
            uint4 x, y;
            dequant4(lat[k][u].x, s, bias, x.x, x.y);
            dequant4(lat[k][u].y, s, bias, x.z, x.w);
            dequant4(lat[k][u].z, s, bias, y.x, y.y);
            dequant4(lat[k][u].w, s, bias, y.z, y.w);
            sts16(to_lo + (4 * part + 2 * k) * kChunkBytes + u * 8192, x);
            sts16(to_hi + (4 * part + 2 * k) * kChunkBytes + u * 8192, y);
          }
        }
        if (part) {
#pragma unroll
          for (uint32_t u = 0; u < S::kPasses; ++u)
            if (slot + 64 * u < rows) sts16(to_rope + u * 8192, rope[u]);
        }
        warp_arrive(&sh.k_full[part], lane);
      }

      // softmax: this thread has row mine_row against kCols heads
      wait(&sh.s_full, turn);
      __syncwarp();
      tc_fence_after();
      float x[kCols];
      tmem_ld_cols<kCols>(lanes + kScores + quarter * kCols, x);
      tmem_ld_wait();
      float most = -INFINITY;
#pragma unroll
      for (uint32_t c = 0; c < kCols; ++c) {
        x[c] = fmaf(x[c], a.scale, -sh.column[warp][c]);
        most = fmaxf(most, x[c]);
      }
      // whether a row of the four warps lies too far above the references: said
      // through a flag and a barrier that is waited for behind the exponentials
      if (__any_sync(0xffffffffu, there && most > kFar) && lane == 0) sh.far[turn][quarter] = 1;
      warp_arrive(&sh.voted[quarter], lane);
#pragma unroll
      for (uint32_t c = 0; c < kCols; ++c) x[c] = exp2_approx(x[c]);
      wait(&sh.voted[quarter], turn);
      const bool far = *(volatile uint32_t*)&sh.far[turn][quarter] != 0;
      if (quad == 0 && lane == 0) sh.far[turn ^ 1][quarter] = 0;
      if (unset || far) {                                // the same in all four warps
        // new references: the columns' largest logits so far.  (Four columns at
        // a time: this is rare, and registers for more would be taken from the
        // rest.)
        float best = -INFINITY;
#pragma unroll
        for (uint32_t c = 0; c < kCols; c += 4) {
          float z[4];
          tmem_ld4(lanes + kScores + quarter * kCols + c, z);
          tmem_ld_wait();
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) {
            float m;
            asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(there ? z[e] * a.scale : -INFINITY));
            if (lane == c + e) best = m;
          }
        }
        if (lane < kCols) sh.top[quarter][quad][lane] = best;
        warp_arrive(&sh.met[quarter], lane);
        const bool all = wait(&sh.met[quarter], meets & 1);
        if (!__all_sync(0xffffffffu, all)) break;
        ++meets;
        float alpha = 1.0f;
        if (lane < kCols) {
          best = fmaxf(fmaxf(sh.top[quarter][0][lane], sh.top[quarter][1][lane]),
                       fmaxf(sh.top[quarter][2][lane], sh.top[quarter][3][lane]));
          if (best > top) {
            alpha = exp2_approx(top - best);             // 0 from -inf
            top = best;
          }
        }
        unset = __any_sync(0xffffffffu, lane < kCols && top == -INFINITY);
        if (__any_sync(0xffffffffu, alpha != 1.0f) && i > 0) {
          if (lane < kCols) sh.column[warp][lane] = alpha;
          __syncwarp();
#pragma unroll 1
          for (uint32_t j = 0; j < 4; ++j)
#pragma unroll 1
            for (uint32_t c = 0; c < kCols; c += 4) {
              float o[4];
              tmem_ld4(lanes + j * kHeads + quarter * kCols + c, o);
              tmem_ld_wait();
#pragma unroll
              for (uint32_t e = 0; e < 4; ++e) o[e] *= sh.column[warp][c + e];
              tmem_st4(lanes + j * kHeads + quarter * kCols + c, o);
            }
#pragma unroll
          for (uint32_t c = 0; c < kCols; ++c) sum[c] *= sh.column[warp][c];
          tmem_st_wait();
          __syncwarp();
        }
        if (lane < kCols) sh.column[warp][lane] = top == -INFINITY ? 0.0f : top;
        __syncwarp();
        tmem_ld_cols<kCols>(lanes + kScores + quarter * kCols, x);
        tmem_ld_wait();
#pragma unroll
        for (uint32_t c = 0; c < kCols; ++c) x[c] = exp2_approx(fmaf(x[c], a.scale, -sh.column[warp][c]));
      }
      // The weights go into the second product as bf16, which its values are
      // (the tensor cores take both operands in one type): half a step is 2^-8
      // of a weight, and of the result no more than that share of sum p |v|.
      // The sum of the weights takes them before the rounding, in fp32, so that
      // the log-sum-exp and the joining of splits lose nothing.
      uint32_t p[kCols / 2];
#pragma unroll
      for (uint32_t c = 0; c < kCols; c += 2) {
        if (there) {                                     // (a row that is not may hold anything)
          sum[c] += x[c];
          sum[c + 1] += x[c + 1];
        }
        p[c / 2] = there ? bf16_pair(x[c], x[c + 1]) : 0u;
      }
      if (mine_row < rows) {
        const uint32_t weights = tile_at + 8 * kChunkBytes;
        if constexpr (kCols == 4) {                      // half a piece
          sts8(weights + swizzled(mine_row, quarter >> 1) + (quarter & 1) * 8, p[0], p[1]);
        } else {
#pragma unroll
          for (uint32_t c = 0; c < kCols / 8; ++c)
            sts16(weights + swizzled(mine_row, quarter * (kCols / 8) + c),
                  make_uint4(p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]));
        }
      }
      tc_fence_before();
      warp_arrive(&sh.p_full, lane);
    }

    const int64_t out_row = (int64_t)t * a.heads + head;
    float* const part = a.part + ((int64_t)split * a.nq * a.heads + out_row) * KVO_LATENT_BYTES;
    lane_sums<kCols, 16>(sum, lane);
    named_sync(1 + quarter, 128);                        // sh.top is free again
    if (lane % (32 / kCols) == 0) sh.top[quarter][quad][lane / (32 / kCols)] = sum[0];
    named_sync(1 + quarter, 128);
    float total = 0.0f;
    if (lane < kCols)
      total = (sh.top[quarter][0][lane] + sh.top[quarter][1][lane]) + (sh.top[quarter][2][lane] + sh.top[quarter][3][lane]);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    const float lse2 = total == 0.0f ? -INFINITY : (top == -INFINITY ? 0.0f : top) + log2f(total);
    if (quad == 0 && lane < mine) {
      if (a.splits > 1)
        a.part_lse[(int64_t)split * a.nq * a.heads + out_row + lane] = lse2;
      else if (a.lse)
        a.lse[out_row + lane] = lse2 * 0.6931471805599453f;
    }
    __syncwarp();
    if (lane < kCols) sh.column[warp][lane] = inv;
    __syncwarp();
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
      if (j % 2 == 0) wait(&sh.pv_done[j / 2], (tiles - 1) & 1);
      __syncwarp();
      tc_fence_after();
      float o[kCols];
      tmem_ld_cols<kCols>(lanes + j * kHeads + quarter * kCols, o);
      tmem_ld_wait();
      const uint32_t d = j * 128 + quad * 32 + lane;
      if (a.splits > 1) {
#pragma unroll
        for (uint32_t c = 0; c < kCols; ++c)
          if (c < mine) part[c * KVO_LATENT_BYTES + d] = o[c] * sh.column[warp][c];
      } else {
#pragma unroll
        for (uint32_t c = 0; c < kCols; ++c)
          if (c < mine)
            reinterpret_cast<__nv_bfloat16*>(a.out)[(out_row + c) * KVO_LATENT_BYTES + d] =
                __float2bfloat16_rn(o[c] * sh.column[warp][c]);
      }
    }
  } else if (warp == kMmaWarp) {
    constexpr uint32_t kQk = mma_desc(1, kHeads, false, false), kPv = mma_desc(1, kHeads, true, true);
    const uint64_t keys = tile_desc(tile_at, 16), heads = tile_desc(queries, 16);
    const uint64_t values = tile_desc(tile_at, kChunkBytes), weights = tile_desc(tile_at + 8 * kChunkBytes, kChunkBytes);
    bool ok = true;
    for (uint32_t i = 0; i < tiles; ++i) {
      const uint32_t turn = i & 1, steps = rows_of(i) / 16;
      // S^T: 64 values of K and Q at a time, four steps of 16.  (M is 128 and a
      // tile has fewer rows: the others are whatever lies behind, and masked.)
#pragma unroll
      for (uint32_t part = 0; part < 2; ++part) {
        ok = ok && wait(&sh.k_full[part], turn);
        __syncwarp();
        fence_proxy_async_smem();                        // the workers' stores, before the MMAs read them
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (uint32_t m = 0; m < (part ? 20 : 16); ++m) {
            const uint32_t c = 4 * part + m / 4, k = m % 4;
            mma_bf16(tmem + kScores, keys + c * (kChunkBytes >> 4) + 2 * k, heads + c * (kHeads * 128 >> 4) + 2 * k,
                     kQk, c + k > 0);
          }
          if (part) mma_commit(&sh.s_full);
        }
        __syncwarp();
      }
      ok = ok && wait(&sh.p_full, turn);
      if (!__all_sync(0xffffffffu, ok)) break;
      fence_proxy_async_smem();
      tc_fence_after();
      // O^T: 128 values at a time, in steps of 16 rows (2,048 bytes)
      if (elect_one()) {
        if (steps == kRows / 16) {
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j) {
#pragma unroll
            for (uint32_t k = 0; k < kRows / 16; ++k)
              mma_bf16(tmem + j * kHeads, values + (2 * j) * (kChunkBytes >> 4) + k * 128, weights + k * 128, kPv,
                       k > 0 || i > 0);
            if (j % 2) mma_commit(&sh.pv_done[j / 2]);
          }
        } else {
          for (uint32_t j = 0; j < 4; ++j) {
            for (uint32_t k = 0; k < steps; ++k)
              mma_bf16(tmem + j * kHeads, values + (2 * j) * (kChunkBytes >> 4) + k * 128, weights + k * 128, kPv,
                       k > 0 || i > 0);
            if (j % 2) mma_commit(&sh.pv_done[j / 2]);
          }
        }
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  // Where any wait gave up, whoever it was, what is in flight finishes before
  // the CTA ends and its memory is given back: the MMAs (the lane that issued
  // them commits) and the last tile's copies.  A loading warp that had given up
  // before that tile arrives for it, so that its phase can end; the tile before
  // had come whole.
  if (sh.gave_up) {
    if (tid == 0) atomicOr(a.status, kFlagTimeout);
    if (warp == kMmaWarp) {
      if (elect_one()) {
        mma_commit(&sh.drained);
        if (!landed(&sh.drained, 0)) atomicOr(a.status, kFlagInflight);
      }
    } else if (warp >= kLoadWarp && lane == 0) {
      uint32_t most = 0;
      for (uint32_t w = 0; w < kLoadWarps; ++w) most = max(most, sh.brought[w]);
      if (sh.brought[warp - kLoadWarp] < most) mbar_arrive(&sh.raw_full);
      if (most && !landed(&sh.raw_full, (most - 1) & 1)) atomicOr(a.status, kFlagInflight);
    }
    __syncthreads();
  }
  if (warp == kMmaWarp) tmem_free(tmem, S::kTmemCols);
}

// The weights exp2(lse - the joint lse) join the splits of one (query, head).
// Partial results are asked for before their weights, and past the first-level
// cache: these grids may have begun before they were written.  A split without
// rows has written nothing but its -inf.
constexpr uint32_t kMaxSplits = 1024;

__device__ __forceinline__ float4 partial(const float* part, int64_t row, uint32_t at) {
  return __ldcg(reinterpret_cast<const float4*>(part + row * KVO_LATENT_BYTES + 4 * at));
}

struct Joined {
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float total = 0.0f;
  __device__ __forceinline__ void add(float w, const float4& v) {
    if (!(w > 0.0f) && !isnan(w)) return;
    total += w;
    o.x = fmaf(w, v.x, o.x);
    o.y = fmaf(w, v.y, o.y);
    o.z = fmaf(w, v.z, o.z);
    o.w = fmaf(w, v.w, o.w);
  }
  __device__ __forceinline__ void write(float base, int64_t r, uint32_t at, uint16_t* out, float* lse) const {
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    reinterpret_cast<uint2*>(out + r * KVO_LATENT_BYTES)[at] =
        make_uint2(bf16_pair(o.x * inv, o.y * inv), bf16_pair(o.z * inv, o.w * inv));
    if (lse && at == 0) lse[r] = total == 0.0f ? -INFINITY : (base + log2f(total)) * 0.6931471805599453f;
  }
};

// Up to 32 splits: group g of 128 threads has every kGroups-th one's values
// from g on, kMost at most.  The weights are formed by every thread for up to
// 8 splits and by every warp, one a lane, for more, so that nothing waits at a
// barrier before the sum: 64 queries of 64 heads over whole sequences of 2,048
// rows, 2 splits, 48.4 us in all, 49.4 with a barrier, 12 with 12 splits 19.8
// and 24.1, one with 32 10.0 and 10.7.
template <uint32_t kMost, uint32_t kGroups>
__global__ void __launch_bounds__(128 * kGroups) join_few_kernel(const float* part, const float* part_lse, uint32_t splits,
                                                                 int64_t rows, uint16_t* out, float* lse) {
  static_assert(kMost * kGroups <= 32);
  __shared__ float4 sums[kGroups > 1 ? kGroups - 1 : 1][128];
  __shared__ float totals[kGroups];
  const int64_t r = blockIdx.x;
  const uint32_t at = threadIdx.x & 127, group = threadIdx.x >> 7, lane = threadIdx.x & 31;
  wait_previous_grid();
  float4 v[kMost];
  constexpr bool kEach = kMost * kGroups <= 8;
  float l[kEach ? kMost : 1], top = -INFINITY;             // of split k, or of split `lane`
#pragma unroll
  for (uint32_t k = 0; k < (kEach ? kMost : 1); ++k) {
    const uint32_t s = kEach ? k : lane;
    l[k] = s < splits ? __ldcg(part_lse + s * rows + r) : -INFINITY;
  }
#pragma unroll
  for (uint32_t k = 0; k < kMost; ++k)
    if (group + k * kGroups < splits) v[k] = partial(part, (group + k * kGroups) * rows + r, at);
#pragma unroll
  for (uint32_t k = 0; k < (kEach ? kMost : 1); ++k) top = fmaxf(top, l[k]);
  if constexpr (!kEach) {
#pragma unroll
    for (uint32_t d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  }
  const float base = top == -INFINITY ? 0.0f : top;
  float w[kEach ? kMost : 1];
#pragma unroll
  for (uint32_t k = 0; k < (kEach ? kMost : 1); ++k) w[k] = exp2f(l[k] - base);
  Joined j;
#pragma unroll
  for (uint32_t k = 0; k < kMost; ++k) {
    if constexpr (kEach)
      j.add(w[k], v[k]);
    else
      j.add(__shfl_sync(0xffffffffu, w[0], group + k * kGroups), v[k]);
  }
  if constexpr (kGroups > 1) {
    if (group) sums[group - 1][at] = j.o;
    if (at == 0) totals[group] = j.total;
    __syncthreads();
    if (group) return;
#pragma unroll
    for (uint32_t g = 1; g < kGroups; ++g) {
      j.total += totals[g];
      j.o.x += sums[g - 1][at].x;
      j.o.y += sums[g - 1][at].y;
      j.o.z += sums[g - 1][at].z;
      j.o.w += sums[g - 1][at].w;
    }
  }
  j.write(base, r, at, out, lse);
}

// More: kGroups groups of 128 threads take every kGroups-th split, kAhead at a time.
template <uint32_t kGroups, uint32_t kAhead>
__global__ void __launch_bounds__(128 * kGroups) join_kernel(const float* part, const float* part_lse, uint32_t splits,
                                                             int64_t rows, uint16_t* out, float* lse) {
  constexpr uint32_t kThreads = 128 * kGroups;
  __shared__ float weight[kMaxSplits];
  __shared__ float red[4 * kGroups];
  __shared__ float4 sums[kGroups - 1][128];
  const int64_t r = blockIdx.x;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = tid >> 7, at = tid & 127;
  wait_previous_grid();
  float4 v[kAhead];
  auto load = [&](uint32_t from) {
#pragma unroll
    for (uint32_t k = 0; k < kAhead; ++k) {
      const uint32_t s = from + k * kGroups;
      if (s < splits) v[k] = partial(part, s * rows + r, at);
    }
  };
  load(group);
  float top = -INFINITY;
  for (uint32_t s = tid; s < splits; s += kThreads) {
    weight[s] = __ldcg(part_lse + s * rows + r);
    top = fmaxf(top, weight[s]);
  }
#pragma unroll
  for (uint32_t d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (lane == 0) red[warp] = top;
  __syncthreads();
#pragma unroll
  for (uint32_t w = 0; w < 4 * kGroups; ++w) top = fmaxf(top, red[w]);
  const float base = top == -INFINITY ? 0.0f : top;
  Joined j;
  for (uint32_t from = group; from < splits; from += kAhead * kGroups) {
#pragma unroll
    for (uint32_t k = 0; k < kAhead; ++k) {
      const uint32_t s = from + k * kGroups;
      j.add(s < splits ? exp2f(weight[s] - base) : 0.0f, v[k]);
    }
    load(from + kAhead * kGroups);
  }
  __syncthreads();
  if (group) sums[group - 1][at] = j.o;
  if (at == 0) red[group] = j.total;
  __syncthreads();
  if (group) return;
  j.total = 0.0f;
  for (uint32_t g = 0; g < kGroups; ++g) j.total += red[g];
  for (uint32_t g = 0; g + 1 < kGroups; ++g) {
    j.o.x += sums[g][at].x;
    j.o.y += sums[g][at].y;
    j.o.z += sums[g][at].z;
    j.o.w += sums[g][at].w;
  }
  j.write(base, r, at, out, lse);
}

// How a call is cut: columns per CTA and splits of every list.
struct Cut {
  uint32_t heads, head_tiles, splits;
};

Cut cut_of(int64_t nq, uint32_t heads, int64_t positions) {
  Cut c;
  // Every query gets the same number of CTAs, from the largest number of
  // positions: a batch just past half, or past all, of the SMs leaves up to half
  // of them without work (2,048 listed positions of 64 heads: 76 queries 53.6
  // us, 77 78.8, 152 86.8, 153 158), and so do uneven lengths.
  // Units of 64 heads by 64 rows: where they do not fill the GPU, fewer heads
  // a CTA leave it less to store and give the rows to more of them.  2,048
  // rows of 64 heads, with 16, 32 and 64 heads a CTA: one query 9.9, 10.2,
  // 11.9 us, two 12.8, 11.4, 12.4, four 15.2, 14.2, 13.5, sixteen 32.8, 24.6,
  // 19.7; 512 rows of one query 8.7, 9.5, 11.2.
  const int64_t units = nq * ((heads + 63) / 64) * ((positions + 63) / 64);
  const uint32_t most_heads = 4 * units <= device_sms() ? 16 : units <= device_sms() ? 32 : 64;
  c.heads = heads <= 16 ? 16 : heads <= 32 ? 32 : 64;
  if (c.heads > most_heads) c.heads = most_heads;
  c.head_tiles = (heads + c.heads - 1) / c.heads;
  const int64_t ctas = nq * c.head_tiles, sms = device_sms(), most = (positions + kLeastRows - 1) / kLeastRows;
  int64_t splits = ctas >= sms ? 1 : sms / ctas;
  if (splits > most) splits = most;
  if (splits > kMaxSplits) splits = kMaxSplits;
  c.splits = (uint32_t)(splits < 1 ? 1 : splits);
  return c;
}

template <uint32_t kHeads>
cudaError_t launch_attend(const AttendArgs& a, cudaStream_t stream) {
  constexpr size_t smem = AttendShape<kHeads>::kSmem;
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!ready[dev & 63]) {
    e = cudaFuncSetAttribute(attend_kernel<kHeads>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    ready[dev & 63] = true;
  }
  return launch_early(attend_kernel<kHeads>, dim3(a.head_tiles * a.splits, a.nq), kAttendThreads, smem, stream, a);
}

}  // namespace
}  // namespace kvo

extern "C" int64_t kvo_attend_work_bytes(int64_t nq, int32_t heads, int64_t positions) {
  if (nq < 1 || nq > KVO_MAX_QUERIES || heads < 1 || heads > KVO_MAX_HEADS || positions < 0 || positions > INT32_MAX - 255)
    return -1;
  const kvo::Cut c = kvo::cut_of(nq, (uint32_t)heads, positions);
  return c.splits == 1 ? 0 : (int64_t)c.splits * nq * heads * (KVO_LATENT_BYTES + 1) * 4;
}

extern "C" kvo_status kvo_attend(kvo_ctx* ctx, const kvo_cache* cache, const kvo_attend_query* s, void* stream) {
  using namespace kvo;
  uint32_t* status = nullptr;
  if (!ctx || !cache_ok(cache) || !s || !cache_rows_ok(cache)) return KVO_EINVAL;
  if (!s->q || !s->lens || !s->out || s->per_seq < 1 || !std::isfinite(s->scale)) return KVO_EINVAL;
  if (s->sel_block < 1 || s->sel_block > KVO_MAX_SCORE_BLOCK || (s->sel_block & (s->sel_block - 1))) return KVO_EINVAL;
  if (s->sel ? s->picked < 0 || s->picked > INT32_MAX : s->rows < 0) return KVO_EINVAL;
  if (s->sel && s->sel_ld < s->picked) return KVO_EINVAL;
  const int64_t nq = (int64_t)cache->sequences * s->per_seq;
  const int64_t positions = s->sel ? s->picked * s->sel_block : s->rows;
  const int64_t need = kvo_attend_work_bytes(nq, s->heads, positions);
  if (need < 0 || s->work_bytes < need || (need && !s->work)) return KVO_EINVAL;
  if (!aligned(s->q, 16) || s->q_ld % 8 || s->q_head_ld % 8 || !aligned(s->out, 16)) return KVO_EINVAL;
  if (!aligned(s->lens, 4) || !aligned(s->sel, 4) || !aligned(s->lse, 4) || !aligned(s->work, 16)) return KVO_EINVAL;
  int64_t wait_clocks = 0;
  const kvo_status st = usable_status(ctx, &status, &wait_clocks);
  if (st != KVO_OK) return st;

  AttendArgs a = {};
  a.wait_clocks = wait_clocks;
  a.cache = cache_view(*cache);
  a.q = static_cast<const uint8_t*>(s->q);
  a.lens = s->lens;
  a.sel = s->sel;
  a.out = s->out;
  a.lse = s->lse;
  a.status = status;
  a.q_ld = s->q_ld * 2;
  a.q_head_ld = s->q_head_ld * 2;
  a.sel_ld = s->sel_ld;
  a.rows = (uint32_t)(s->sel ? 0 : s->rows);
  a.picked = (uint32_t)(s->sel ? s->picked : 0);
  while ((1 << a.sel_shift) < s->sel_block) ++a.sel_shift;
  a.per_seq = (uint32_t)s->per_seq;
  a.heads = (uint32_t)s->heads;
  a.nq = (uint32_t)nq;
  a.scale = s->scale * kLog2e;
  const Cut cut = cut_of(nq, a.heads, positions);
  a.head_tiles = cut.head_tiles;
  a.splits = cut.splits;
  a.part = static_cast<float*>(s->work);
  a.part_lse = a.part + (int64_t)a.splits * nq * a.heads * KVO_LATENT_BYTES;
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  cudaError_t e = cut.heads == 16   ? launch_attend<16>(a, on)
                  : cut.heads == 32 ? launch_attend<32>(a, on)
                                    : launch_attend<64>(a, on);
  if (e == cudaSuccess && a.splits > 1) {
    // Past 32 splits, 1,024 threads for as many outputs as SMs and 512 for more.
    // 64 heads, us: one query of 8,192 rows 15.6 and 17.9, of 65,536 29.5 and
    // 33.6, four of 8,192 22.7 and 21.4.
    const int64_t joins = nq * a.heads;
    const bool wide = joins <= device_sms();
    const auto join = a.splits <= 2    ? join_few_kernel<2, 1>
                      : a.splits <= 4  ? join_few_kernel<4, 1>
                      : a.splits <= 8  ? join_few_kernel<8, 1>
                      : a.splits <= 16 ? join_few_kernel<16, 1>
                      : a.splits <= 32 ? join_few_kernel<16, 2>
                      : wide           ? join_kernel<8, 4>
                                       : join_kernel<4, 8>;
    const uint32_t threads = a.splits <= 16 ? 128 : a.splits <= 32 ? 256 : wide ? 1024 : 512;
    e = launch_early(join, dim3((unsigned)joins), threads, 0, on, a.part, a.part_lse, a.splits, joins, a.out, a.lse);
  }
  return e == cudaSuccess ? KVO_OK : KVO_ECUDA;
}
