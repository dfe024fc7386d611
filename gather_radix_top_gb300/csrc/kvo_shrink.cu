// kvo_shrink_cache: the first, the last and the most attended positions of
// every sequence, up to a budget, copied in their order to another table's
// blocks.
//
// Two launches.  The first finds what stays: one cluster per sequence, a radix
// select over the weights' order-preserving keys (the first and last positions
// have the largest key of all), then an ordered compaction, ties to the lower
// position.  The second copies rows, keys and factors, a warp for four rows:
// their 164 pieces of 16 bytes are all asked for before the first is stored.
//
// Measured on the GPU: 50,023 positions to 8,192 rows 13.6 us (the selection's
// chain of passes and cluster barriers; the copy 4), 33 uneven sequences of up
// to 20,011 to 1,021 23 us, 1,048,576 to 524,288 230 us: 147 for the copy (826
// MB at 5.6 TB/s; every second row of 656 bytes leaves parts of DRAM's bursts
// unused) and 80 for the selection, whose 16 CTAs issue two instructions a clock
// in loops over the keys.  With weights read again in every pass, one at a time,
// it took 270 us, with another pass for what lies above the cut 239.
#include <algorithm>

#include "kvo_cache.cuh"
#include "kvo_topk_body.cuh"

namespace kvo {
namespace {

using namespace topk_detail;

constexpr uint32_t kKeepStatic = 18 * 1024, kKeepSmem = 227 * 1024 - kKeepStatic;

struct ShrinkArgs {
  CacheView from, to;
  const float* weights;
  const int32_t* lens;
  int32_t* kept;
  int32_t* new_lens;
  float* to_weights;         // or NULL
  uint32_t* status;
  int64_t weights_ld, kept_ld, to_weights_ld;
  uint32_t rows, budget, first, last;
  uint32_t key_pieces;       // 16-byte pieces of a key: 0 (none move), 8 or 16
  uint32_t held;             // keys that a CTA has room for, in fours
};

// kDigit: bits of a pass of the radix select.
template <uint32_t kDigit>
struct KeepSmem {
  static constexpr uint32_t kBins = 1u << kDigit, kPasses = (32 + kDigit - 1) / kDigit;
  static constexpr uint32_t kAll = kBins > (uint32_t)kThreads ? kBins : kThreads;
  uint32_t hist[kBins];              // this CTA's, of the current digit
  uint32_t all[kAll];                // the cluster's, and zeros
  uint32_t warp_sum[kWarps], cut[4];
  // Every CTA owns an even share of each pass's bins: this many words.
  __host__ __device__ static constexpr uint32_t owned(uint32_t C) { return kPasses * (kBins / C); }
};

// The n largest of the cluster's keys, ties to the lower position: a radix
// select, whose histograms also tell each CTA how many of its own keys lie
// above the cut and at it, then the ordered compaction.  So the keys are gone
// over once a digit and once more at most.  owned: the passes' bins, zeroed
// before a cluster barrier that precedes this call.
template <uint32_t kDigit, typename Key4, typename Emit>
__device__ __forceinline__ void keep_largest(Key4 key4, uint32_t count, uint32_t n, KeepSmem<kDigit>* sm, uint32_t* owned,
                                             uint32_t (*scratch)[2 * kWarps + 2], uint32_t (*table)[4], Emit emit) {
  const uint32_t tid = threadIdx.x, C = cluster_size(), r = cluster_rank(), per = KeepSmem<kDigit>::kBins / C;
  const uint32_t ngroups = (count + 3) / 4;
  uint32_t prefix = 0, mask = 0, remaining = n, shift = 32, mine[2] = {0, 0};
  for (uint32_t pass = 0;; ++pass) {
    const uint32_t d = min(shift, kDigit), dmask = (1u << d) - 1;
    shift -= d;
    for (uint32_t b = tid; b < KeepSmem<kDigit>::kBins; b += kThreads) sm->hist[b] = 0;
    __syncthreads();
    for (uint32_t g0 = 0; g0 < ngroups; g0 += kThreads) {
      const uint32_t g = g0 + tid;
      const uint4 k = g < ngroups ? key4(g) : make_uint4(0, 0, 0, 0);
      const uint32_t v[4] = {k.x, k.y, k.z, k.w};
      uint32_t bins[4], valid = 0;
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e) {
        bins[e] = v[e] >> shift & dmask;
        valid |= (uint32_t)(4 * g + e < count && (v[e] & mask) == prefix) << e;
      }
      hist_add_warp4(sm->hist, bins, valid);
    }
    __syncthreads();
    for (uint32_t b = tid; b <= dmask; b += kThreads)
      if (const uint32_t v = sm->hist[b]) dsmem_red_add_u32(dsmem_addr(&owned[pass * per + b % per], b / per), v);
    cluster_sync();
    for (uint32_t b = tid; b < KeepSmem<kDigit>::kAll; b += kThreads)
      sm->all[b] = b <= dmask ? dsmem_ld_u32(dsmem_addr(&owned[pass * per + b % per], b / per)) : 0u;
    __syncthreads();
    find_cut<KeepSmem<kDigit>::kAll / kThreads>(sm->all, remaining, sm->warp_sum, sm->cut);
    const uint32_t bucket = sm->cut[0], inside = sm->cut[2];
    remaining -= sm->cut[1];
    prefix |= bucket << shift;
    mask |= dmask << shift;
    const bool done = remaining == inside || shift == 0;
    for (uint32_t b = tid; b <= dmask; b += kThreads) {
      mine[0] += b > bucket ? sm->hist[b] : 0u;
      mine[1] += done && b == bucket ? sm->hist[b] : 0u;
    }
    if (done) break;
    __syncthreads();                                     // before hist and cut change
  }
  uint32_t sums[2], before, at_before;
  block_sum2(mine[0], mine[1], scratch[1], &sums[0], &sums[1]);
  cluster_publish(sums, 2, table, r, C);
  const RadixCut cut{prefix, shift, remaining};
  cut_offsets(table, 0, r, cut.need, &before, &at_before);
  cluster_compact(key4, count, cut, before, at_before, scratch, [&](uint32_t i, uint32_t out) {
    if (out < n) emit(i, out);
  });
}

// A CTA's keys stay in its shared memory, as far as they fit; the passes read
// the weights of the others again.
template <uint32_t kDigit>
__global__ void __launch_bounds__(kThreads, 1) keep_kernel(const __grid_constant__ ShrinkArgs a) {
  extern __shared__ __align__(16) uint8_t dyn_smem[];
  using Smem = KeepSmem<kDigit>;
  static_assert(Smem::kBins % kMaxCluster == 0 && Smem::owned(kMaxCluster) % 4 == 0);
  static_assert(sizeof(Smem) + 4 * 2 * (2 * kWarps + 2) + 16 * kMaxCluster <= kKeepStatic);
  __shared__ Smem sm;
  __shared__ uint32_t scratch[2][2 * kWarps + 2];
  __shared__ uint32_t table[kMaxCluster][4];
  wait_previous_grid();
  allow_next_grid();
  const uint32_t C = cluster_size(), r = cluster_rank(), s = blockIdx.x / C, tid = threadIdx.x;
  const float* const w = a.weights + s * a.weights_ld;
  int32_t* const kept = a.kept + s * a.kept_ld;
  float* const to_w = a.to_weights ? a.to_weights + s * a.to_weights_ld : nullptr;
  const int32_t given = a.lens[s];
  const uint32_t len = given <= 0 ? 0u : min((uint32_t)given, a.rows), n = min(len, a.budget);
  if (r == 0 && tid == 0) a.new_lens[s] = (int32_t)n;
  for (uint32_t j = n + r * kThreads + tid; j < a.budget; j += C * kThreads) {
    kept[j] = -1;
    if (to_w) to_w[j] = 0.0f;
  }
  if (len <= a.budget) {                                 // the same in the whole cluster
    for (uint32_t j = r * kThreads + tid; j < n; j += C * kThreads) {
      kept[j] = (int32_t)j;
      if (to_w) to_w[j] = w[j];
    }
    return;
  }
  const uint32_t chunk = topk_chunk(len, C), lo = min(r * chunk, len), count = min(chunk, len - lo);
  auto key = [&](uint32_t i) -> uint32_t {               // of position lo + i
    const uint32_t p = lo + i;
    return p < a.first || p >= len - a.last ? 0xffffffffu : score_key(__ldg(w + p));
  };
  const bool wide = (reinterpret_cast<uintptr_t>(w + lo) & 15u) == 0;
  auto four = [&](uint32_t g) -> uint4 {
    const uint32_t p = lo + 4 * g;
    if (wide && p >= a.first && p + 4 <= len - a.last && 4 * g + 4 <= count) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(w + p));
      return make_uint4(score_key(f.x), score_key(f.y), score_key(f.z), score_key(f.w));
    }
    uint32_t v[4];
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e) v[e] = 4 * g + e < count ? key(4 * g + e) : 0u;
    return make_uint4(v[0], v[1], v[2], v[3]);
  };
  auto emit = [&](uint32_t i, uint32_t out) {
    kept[out] = (int32_t)(lo + i);
    if (to_w) to_w[out] = __ldg(w + lo + i);
  };
  uint32_t* const owned = reinterpret_cast<uint32_t*>(dyn_smem);
  uint4* const keys = reinterpret_cast<uint4*>(owned + Smem::owned(C));
  for (uint32_t b = tid; b < Smem::owned(C); b += kThreads) owned[b] = 0;
  const uint32_t held = min((count + 3) / 4, a.held);
  for_groups(four, held, [&](uint32_t g, uint4 v) {
    if (g < held) keys[g] = v;
  });
  cluster_sync();
  keep_largest([&](uint32_t g) { return g < held ? keys[g] : four(g); }, count, n, &sm, owned, scratch, table, emit);
}

constexpr uint32_t kMoveThreads = 256, kMoveRows = 4;    // rows of a warp
constexpr uint32_t kRowPieces = KVO_ROW_BYTES / 16, kMoveSteps = (kMoveRows * kRowPieces + 31) / 32;

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ ShrinkArgs a) {
  const uint32_t lane = threadIdx.x & 31, s = blockIdx.y;
  const uint32_t j0 = (blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5)) * kMoveRows;
  wait_previous_grid();
  allow_next_grid();
  const uint32_t n = (uint32_t)a.new_lens[s];
  if (j0 >= n) return;
  // lane l < kMoveRows has row j0 + l's places; one without a source becomes
  // zeros, one without a destination is skipped
  int64_t src = -1, dst = -1;
  if (lane < kMoveRows && j0 + lane < n) {
    src = cache_row(a.from, s, (uint32_t)a.kept[s * a.kept_ld + j0 + lane]);
    dst = cache_row(a.to, s, j0 + lane);
    if (src < 0 || dst < 0) atomicOr(a.status, kFlagRange);
  }
  uint4 v[kMoveSteps];
  int64_t at[kMoveSteps];
#pragma unroll
  for (uint32_t i = 0; i < kMoveSteps; ++i) {
    const uint32_t piece = i * 32 + lane, row = piece / kRowPieces, c = piece - row * kRowPieces;
    const int64_t from = __shfl_sync(0xffffffffu, src, row & 31), to = __shfl_sync(0xffffffffu, dst, row & 31);
    at[i] = row < kMoveRows && to >= 0 ? to * kRowPieces + c : -1;
    v[i] = make_uint4(0, 0, 0, 0);
    if (at[i] >= 0 && from >= 0) v[i] = __ldcs(reinterpret_cast<const uint4*>(a.from.rows) + from * kRowPieces + c);
  }
  uint4 k[2];
  int64_t key_at[2];
  const uint32_t pieces = a.key_pieces, key_shift = pieces == 16 ? 4 : 3;
#pragma unroll
  for (uint32_t i = 0; i < 2; ++i) {
    const uint32_t piece = i * 32 + lane, row = piece >> key_shift, c = piece & (pieces - 1);
    const int64_t from = __shfl_sync(0xffffffffu, src, row & 31), to = __shfl_sync(0xffffffffu, dst, row & 31);
    key_at[i] = pieces && row < kMoveRows && to >= 0 ? to * pieces + c : -1;
    k[i] = make_uint4(0, 0, 0, 0);
    if (key_at[i] >= 0 && from >= 0) k[i] = __ldcs(reinterpret_cast<const uint4*>(a.from.keys) + from * pieces + c);
  }
#pragma unroll
  for (uint32_t i = 0; i < kMoveSteps; ++i)
    if (at[i] >= 0) reinterpret_cast<uint4*>(a.to.rows)[at[i]] = v[i];
#pragma unroll
  for (uint32_t i = 0; i < 2; ++i)
    if (key_at[i] >= 0) reinterpret_cast<uint4*>(a.to.keys)[key_at[i]] = k[i];
  if (pieces == 8 && dst >= 0) a.to.key_scales[dst] = src >= 0 ? a.from.key_scales[src] : 0.0f;
}

cudaError_t launch_keep(ShrinkArgs a, uint32_t sequences, cudaStream_t stream) {
  static int widest[64] = {};                            // clusters of 1,024 threads and all shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int& most = widest[dev & 63];
  if (!most) {
    int both = (int)kMaxCluster;
    for (const void* kern : {(const void*)keep_kernel<8>, (const void*)keep_kernel<11>}) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kKeepSmem);
      if (e != cudaSuccess) return e;
      const int c = best_cluster(kern, kKeepSmem, (int)kMaxCluster);
      if (c < 1) return cudaErrorInvalidConfiguration;
      both = c < both ? c : both;
    }
    most = both;
  }
  // As many CTAs a sequence as the GPU has room for at once, but not so many
  // that one gets less than a tile of the compaction.
  uint32_t C = 1;
  while ((int)C < most && 2 * C * sequences <= (uint32_t)device_sms() && a.rows > C * 4u * kThreads) C *= 2;
  // Three passes of 11 bits for many keys a CTA, four of 8 for few.  Both ways,
  // us, to 1,000 rows, weights even in [0, 1) (and log-normal ones): one sequence of
  // 50,000 14.3 and 13.6 (13.8 and 13.6), of 262,144, 16,384 a CTA, 24.9 and 22.2
  // (20.9 and 19.1), of 500,000 35.8 and 36.8 (29.9 and 28.2); four of 262,144 25.9
  // and 25.5 (21.6 and 22.3); 152 of 200,000 252 and 277 (240 and 241); log-normal,
  // 1,048,576 to half of them 230 and 236.
  const uint32_t chunk = topk_chunk(a.rows, C);
  const bool many = chunk > 24 * 1024;
  const uint32_t bins = many ? KeepSmem<11>::owned(C) : KeepSmem<8>::owned(C);
  a.held = std::min(chunk, kKeepSmem / 4 - bins) / 4;
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  lc.gridDim = dim3(C * sequences);
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = bins * 4 + a.held * 16;
  lc.stream = stream;
  lc.attrs = attr;
  lc.numAttrs = 2;
  return cudaLaunchKernelEx(&lc, many ? keep_kernel<11> : keep_kernel<8>, a);
}

}  // namespace
}  // namespace kvo

extern "C" kvo_status kvo_shrink_cache(kvo_ctx* ctx, const kvo_cache* from, const kvo_cache* to, const kvo_shrink* s,
                                       void* stream) {
  using namespace kvo;
  uint32_t* status = nullptr;
  if (!ctx || !cache_ok(from) || !cache_ok(to) || !s || !cache_rows_ok(from) || !cache_rows_ok(to)) return KVO_EINVAL;
  if (from->sequences != to->sequences || from->sequences > KVO_MAX_QUERIES) return KVO_EINVAL;
  if (from->rows == to->rows && from->table == to->table) return KVO_EINVAL;
  if (to->keys && (!cache_keys_ok(from) || !cache_keys_ok(to) || from->key_type != to->key_type)) return KVO_EINVAL;
  if (!s->weights || !s->lens || !s->kept || !s->new_lens) return KVO_EINVAL;
  if (!aligned(s->weights, 4) || !aligned(s->lens, 4) || !aligned(s->kept, 4) || !aligned(s->new_lens, 4) ||
      !aligned(s->to_weights, 4))
    return KVO_EINVAL;
  if (s->rows < 1 || s->rows > INT32_MAX - 255 || s->budget < 1 || s->budget > INT32_MAX - 255) return KVO_EINVAL;
  if (s->first < 0 || s->last < 0 || (int64_t)s->first + s->last > s->budget) return KVO_EINVAL;
  if (from->sequences > 1 &&
      (s->weights_ld < s->rows || s->kept_ld < s->budget || (s->to_weights && s->to_weights_ld < s->budget)))
    return KVO_EINVAL;
  const kvo_status st = usable_status(ctx, &status);
  if (st != KVO_OK) return st;

  ShrinkArgs a = {};
  a.from = cache_view(*from);
  a.to = cache_view(*to);
  a.weights = s->weights;
  a.lens = s->lens;
  a.kept = s->kept;
  a.new_lens = s->new_lens;
  a.to_weights = s->to_weights;
  a.status = status;
  a.weights_ld = s->weights_ld;
  a.kept_ld = s->kept_ld;
  a.to_weights_ld = s->to_weights_ld;
  a.rows = (uint32_t)s->rows;
  a.budget = (uint32_t)s->budget;
  a.first = (uint32_t)s->first;
  a.last = (uint32_t)s->last;
  a.key_pieces = !to->keys ? 0 : to->key_type == KVO_E4M3 ? 8 : 16;
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  const uint32_t sequences = (uint32_t)from->sequences;
  cudaError_t e = launch_keep(a, sequences, on);
  if (e != cudaSuccess) return KVO_ECUDA;
  const uint32_t most = a.rows < a.budget ? a.rows : a.budget, per = kMoveThreads / 32 * kMoveRows;
  e = launch_early(move_kernel, dim3((most + per - 1) / per, sequences), kMoveThreads, 0, on, a);
  return e == cudaSuccess ? KVO_OK : KVO_ECUDA;
}
