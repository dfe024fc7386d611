// kvo_index_scores: score[t][j] = s_j * sum_h w[t][h] * max(0, q[t][h] . key_j).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "kvo_cache.cuh"

namespace kvo {
namespace {

constexpr int kScoreThreads = 128;

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
  uint32_t per_seq, heads, block;
};

__device__ __forceinline__ float key_float(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float key_float(const __nv_fp8_e4m3* p) { return (float)*p; }

// One thread per (query, position).
template <typename T>
__global__ void __launch_bounds__(kScoreThreads) index_scores_kernel(const __grid_constant__ ScoreArgs a) {
  __shared__ float best[kScoreThreads];
  const uint32_t t = blockIdx.y;
  const uint32_t p = blockIdx.x * kScoreThreads + threadIdx.x;
  const int32_t len = a.lens[t];
  float score = -INFINITY;
  if (p < a.n && (int64_t)p < len) {
    const int64_t row = cache_row(a.cache, t / a.per_seq, p);
    if (row < 0) {
      atomicOr(a.status, kFlagRange);
    } else {
      const T* key = reinterpret_cast<const T*>(a.cache.keys) + row * KVO_KEY_VALUES;
      float sum = 0.0f;
      for (uint32_t h = 0; h < a.heads; ++h) {
        const T* q = reinterpret_cast<const T*>(a.q + t * a.q_ld + h * a.q_head_ld);
        float dot = 0.0f;
        for (int d = 0; d < KVO_KEY_VALUES; ++d) dot = fmaf(key_float(q + d), key_float(key + d), dot);
        sum = fmaf(a.w[t * a.w_ld + h], dot > 0.0f || isnan(dot) ? dot : 0.0f, sum);
      }
      score = a.cache.key_scales ? sum * a.cache.key_scales[row] : sum;
    }
  }
  if (a.block == 1) {
    if (p < a.n) a.scores[t * a.ld + p] = score;
    return;
  }
  best[threadIdx.x] = isnan(score) ? -INFINITY : score;
  __syncthreads();
  if (p < a.n && p % a.block == 0) {
    float m = best[threadIdx.x];
    for (uint32_t i = 1; i < a.block; ++i) m = fmaxf(m, best[threadIdx.x + i]);
    a.scores[t * a.ld + p / a.block] = m;
  }
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
  const int64_t size = cache->key_type == KVO_BF16 ? 2 : 1;
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
  a.block = (uint32_t)s->block;
  const dim3 grid((unsigned)((s->n + kScoreThreads - 1) / kScoreThreads), (unsigned)nq);
  const cudaStream_t st_ = static_cast<cudaStream_t>(stream);
  if (cache->key_type == KVO_BF16)
    index_scores_kernel<__nv_bfloat16><<<grid, kScoreThreads, 0, st_>>>(a);
  else
    index_scores_kernel<__nv_fp8_e4m3><<<grid, kScoreThreads, 0, st_>>>(a);
  return cudaGetLastError() == cudaSuccess ? KVO_OK : KVO_ECUDA;
}
