// kvo_attend: softmax attention of absorbed MLA queries over cached rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvo_cache.cuh"

namespace kvo {
namespace {

constexpr int kAttendThreads = 256;
constexpr int kAttendTile = 64;      // rows whose logits are held at a time
constexpr int kQueryValues = KVO_DEQUANT_VALUES;

struct AttendArgs {
  CacheView cache;
  const uint8_t* q;
  const int32_t* lens;
  const int32_t* sel;
  uint16_t* out;
  float* lse;
  uint32_t* status;
  int64_t q_ld, q_head_ld;   // bytes
  int64_t sel_ld;
  uint32_t rows, picked, sel_shift;
  uint32_t per_seq, heads;
  float scale;
};

// The position that entry j of query t's list names, or -1 (masked).
__device__ __forceinline__ int64_t listed_position(const AttendArgs& a, uint32_t t, uint32_t j, int32_t len) {
  int64_t p = j;
  if (a.sel) {
    const int32_t u = a.sel[t * a.sel_ld + (j >> a.sel_shift)];
    if (u < 0) return -1;
    p = ((int64_t)u << a.sel_shift) + (j & ((1u << a.sel_shift) - 1));
  }
  return p < len ? p : -1;
}

__device__ __forceinline__ float row_value(const uint8_t* row, uint32_t d) {
  if (d >= KVO_LATENT_BYTES)
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row + KVO_LATENT_BYTES + 16)[d - KVO_LATENT_BYTES]);
  const float s = __half2float(reinterpret_cast<const __half*>(row + KVO_LATENT_BYTES)[d >> 6]);
  return __bfloat162float(__float2bfloat16_rn((float)(int8_t)row[d] * s));
}

// One CTA per (query, head): a running maximum and sum over tiles of rows; a
// warp per row for the logits, two output values per thread.
__global__ void __launch_bounds__(kAttendThreads) attend_kernel(const __grid_constant__ AttendArgs a) {
  __shared__ float q[kQueryValues];
  __shared__ float z[kAttendTile];
  __shared__ int64_t row[kAttendTile];
  const uint32_t t = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(a.q + t * a.q_ld + h * a.q_head_ld);
  for (uint32_t d = tid; d < kQueryValues; d += kAttendThreads) q[d] = __bfloat162float(src[d]);
  const int32_t len = a.lens[t];
  const uint32_t all = a.sel ? a.picked << a.sel_shift : (uint32_t)(len <= 0 ? 0 : min((uint32_t)len, a.rows));
  float m = -INFINITY, l = 0.0f, o0 = 0.0f, o1 = 0.0f;
  for (uint32_t j0 = 0; j0 < all; j0 += kAttendTile) {
    __syncthreads();
    if (tid < kAttendTile) {
      const int64_t p = j0 + tid < all ? listed_position(a, t, j0 + tid, len) : -1;
      const int64_t r = p >= 0 ? cache_row(a.cache, t / a.per_seq, (uint32_t)p) : -1;
      if (p >= 0 && r < 0) atomicOr(a.status, kFlagRange);
      row[tid] = r;
    }
    __syncthreads();
    for (uint32_t j = warp; j < kAttendTile; j += kAttendThreads / 32) {
      float sum = 0.0f;
      if (row[j] >= 0) {
        const uint8_t* r = a.cache.rows + row[j] * KVO_ROW_BYTES;
        for (uint32_t d = lane; d < kQueryValues; d += 32) sum = fmaf(q[d], row_value(r, d), sum);
      }
      for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
      if (lane == 0) z[j] = row[j] >= 0 ? sum * a.scale : -INFINITY;
    }
    __syncthreads();
    float top = m;
    for (uint32_t j = 0; j < kAttendTile; ++j) top = fmaxf(top, z[j]);
    if (top == -INFINITY) continue;
    const float keep = expf(m - top);
    m = top;
    l *= keep;
    o0 *= keep;
    o1 *= keep;
    for (uint32_t j = 0; j < kAttendTile; ++j) {
      if (row[j] < 0) continue;
      const uint8_t* r = a.cache.rows + row[j] * KVO_ROW_BYTES;
      const float p = expf(z[j] - m);
      l += p;
      o0 = fmaf(p, row_value(r, tid), o0);
      o1 = fmaf(p, row_value(r, tid + kAttendThreads), o1);
    }
  }
  const float inv = l > 0.0f || isnan(l) ? 1.0f / l : 0.0f;
  uint16_t* out = a.out + ((int64_t)t * a.heads + h) * KVO_LATENT_BYTES;
  reinterpret_cast<__nv_bfloat16*>(out)[tid] = __float2bfloat16_rn(o0 * inv);
  reinterpret_cast<__nv_bfloat16*>(out)[tid + kAttendThreads] = __float2bfloat16_rn(o1 * inv);
  if (a.lse && tid == 0) a.lse[(int64_t)t * a.heads + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace
}  // namespace kvo

extern "C" int64_t kvo_attend_work_bytes(int64_t nq, int32_t heads, int64_t positions) {
  if (nq < 1 || nq > KVO_MAX_QUERIES || heads < 1 || heads > KVO_MAX_HEADS || positions < 0 || positions > INT32_MAX - 255)
    return -1;
  return 0;
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
  const kvo_status st = usable_status(ctx, &status);
  if (st != KVO_OK) return st;

  AttendArgs a = {};
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
  a.scale = s->scale;
  const dim3 grid((unsigned)s->heads, (unsigned)nq);
  attend_kernel<<<grid, kAttendThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? KVO_OK : KVO_ECUDA;
}
