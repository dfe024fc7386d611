// kvo_append_tokens: a token's latent, position part and index key become a
// cache row (and key) in one pass.
//
// Per token: 512 latent values in 8 groups of 64, each scaled to int8; 32
// pairs rotated by pos * inv_freq; 128 key values rounded to e4m3 or bf16.
// One warp per token, so that a group is four lanes, a pair one lane, the
// key four values a lane, and nothing needs shared memory or a barrier.
//
// What bounds it: 60,000 bf16 tokens with e4m3 keys and the dequantised copy
// (201 MB) take 39.4 us, 5.1 TB/s, where a copy of the bytes would take 30:
// 481 warp instructions a token fill the schedulers to 64 % while the loads'
// latency is covered by 35 warps an SM (of 40 that fit).  16,381 fp32 tokens
// (78 MB) take 12.3 us, 6.3 TB/s.  One token takes 2.4 us, most of it launch.  Measured against
// it for the 60,000: lookups before the loads 53 us, CTAs of 256 threads 45.6,
// 64 registers (32 warps an SM) 42.6, half a warp per token (120 registers)
// 56, a persistent loop that loads one token ahead 46.6.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "kvo_cache.cuh"

namespace kvo {
namespace {

constexpr int kAppendThreads = 128;
constexpr double kMaxInvFreq = 1048576.0;   // keeps the low part of inv_freq / 2 pi within 64 bits

struct AppendArgs {
  CacheView cache;
  const uint8_t* latent;
  const uint8_t* rope;
  const uint8_t* key;
  const int32_t* seq;
  const int32_t* pos;
  const int32_t* place;                 // or NULL: pos
  uint16_t* out_bf16;
  uint32_t* status;
  int64_t latent_ld, rope_ld, key_ld;   // elements
  int64_t n;
  uint64_t turn[32];                    // inv_freq / 2 pi, modulo one turn, in units of 2^-64 turns
  uint32_t interleaved;
  uint32_t key_type;
};

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_float(float v) { return v; }

// N consecutive elements (a multiple of 16 bytes in all, or 8) as floats.
template <typename T, int N>
__device__ __forceinline__ void load_floats(const T* p, float* v) {
  constexpr int kBytes = N * (int)sizeof(T);
  if constexpr (kBytes % 16 == 0) {
    uint4 raw[kBytes / 16];
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) raw[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    const T* e = reinterpret_cast<const T*>(raw);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = to_float(e[i]);
  } else {
    static_assert(kBytes == 8, "8 or a multiple of 16 bytes");
    const uint2 raw = __ldg(reinterpret_cast<const uint2*>(p));
    const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = to_float(e[i]);
  }
}

// The smallest fp16 s with 127 * s >= amax, at most 65504: the product with
// 1 / 127 rounded up is at most one step off.  127 * s has 18 significant
// bits, so the comparisons in fp32 are exact.
__device__ __forceinline__ __half group_scale(float amax) {
  uint16_t h = __half_as_ushort(__float2half_ru(amax * (1.0f / 127.0f)));
  if (h >= 0x7c00u) h = 0x7bffu;
  if (h < 0x7bffu && 127.0f * __half2float(__ushort_as_half(h)) < amax) ++h;
  if (h > 0u && 127.0f * __half2float(__ushort_as_half(h - 1)) >= amax) --h;
  return __ushort_as_half(h);
}

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

constexpr float kToInteger = 12582912.0f;   // 1.5 * 2^23: adding it rounds to an integer, in the low bits

// x / s rounded to the nearest integer, ties to even, as kToInteger + q
// (|x| <= 127 s).  The quotient through the reciprocal and one correction
// (x - q s is exact) is exact where the quotient is a tie.  For 16-bit x
// every other quotient is at least 2^-12 from a tie (x has at most 11 bits, s
// 11), so its rounding does not matter.  An fp32 x can be nearer than the
// quotient's last bit: there the remainder decides.
template <bool kWide>
__device__ __forceinline__ float quantise(float x, float s, float inv) {
  float q = x * inv;
  q = fmaf(fmaf(-q, s, x), inv, q);
  float t = q + kToInteger;
  if (kWide) {
    q = t - kToInteger;
    const float r = fmaf(-q, s, x), half = 0.5f * s;
    if (fabsf(r) > half || (fabsf(r) == half && ((int)q & 1))) t += r > 0.0f ? 1.0f : -1.0f;
  }
  return t;
}

// kPlaced: rows go to places of their own.  (Asked of every token instead, it
// takes the 60,000 tokens from 40.0 to 40.4 us.)
template <typename T, bool kPlaced>
__global__ void __launch_bounds__(kAppendThreads, sizeof(T) == 2 ? 10 : 1) append_tokens_kernel(const __grid_constant__ AppendArgs a) {
  const uint32_t lane = threadIdx.x & 31;
  const int64_t i = ((int64_t)blockIdx.x * kAppendThreads + threadIdx.x) >> 5;
  wait_previous_grid();
  allow_next_grid();
  if (i >= a.n) return;

  // the token's values are asked for before its place is looked up, so that
  // the two chains of loads overlap
  const int32_t s = a.seq ? a.seq[i] : (int32_t)(i < INT32_MAX ? i : INT32_MAX);
  const int32_t p = a.pos[i], at = kPlaced ? a.place[i] : p;
  float x[16], k[4];
  load_floats<T, 16>(reinterpret_cast<const T*>(a.latent) + i * a.latent_ld + 16 * lane, x);
  const T* rope = reinterpret_cast<const T*>(a.rope) + i * a.rope_ld;
  const uint32_t i0 = a.interleaved ? 2 * lane : lane, i1 = a.interleaved ? 2 * lane + 1 : lane + 32;
  const float r0 = to_float(rope[i0]), r1 = to_float(rope[i1]);
  if (a.key) load_floats<T, 4>(reinterpret_cast<const T*>(a.key) + i * a.key_ld + 4 * lane, k);

  if (s < 0) return;
  const int64_t row =
      p >= 0 && (!kPlaced || at >= 0) && (uint32_t)s < a.cache.sequences ? cache_row(a.cache, (uint32_t)s, (uint32_t)at) : -1;
  uint16_t* values = a.out_bf16 ? a.out_bf16 + i * KVO_DEQUANT_VALUES : nullptr;
  if (row < 0) {
    if (lane == 0) atomicOr(a.status, kFlagRange);
    if (values) {
      const uint4 zero = make_uint4(0, 0, 0, 0);
      for (uint32_t v = lane; v < KVO_DEQUANT_VALUES / 8; v += 32) reinterpret_cast<uint4*>(values)[v] = zero;
    }
    return;
  }
  uint8_t* dst = a.cache.rows + row * KVO_ROW_BYTES;

  // latent: lanes 4g .. 4g+3 hold group g; a NaN or an infinity shows in its maximum
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < 16; ++e) top = max_nan(top, fabsf(x[e]));
  top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const bool finite = top < INFINITY;
  const __half scale = finite ? group_scale(top) : __ushort_as_half(0x7e00);
  const float sf = __half2float(scale);
  if (!(finite && sf > 0.0f)) {                           // all 64 values are zeros
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = 0.0f;
  } else if (top > 127.0f * 65504.0f) {                   // beyond the largest scale
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = fminf(fmaxf(x[e], -127.0f * 65504.0f), 127.0f * 65504.0f);
  }
  const float by = finite && sf > 0.0f ? sf : 1.0f, inv = rcp_approx(by);
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = quantise<sizeof(T) == 4>(x[e], by, inv);
  uint32_t packed[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t lo = __byte_perm(__float_as_uint(x[4 * w]), __float_as_uint(x[4 * w + 1]), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(x[4 * w + 2]), __float_as_uint(x[4 * w + 3]), 0x0040);
    packed[w] = __byte_perm(lo, hi, 0x5410);
  }
  reinterpret_cast<uint4*>(dst)[lane] = make_uint4(packed[0], packed[1], packed[2], packed[3]);
  if ((lane & 3) == 0) reinterpret_cast<__half*>(dst + KVO_LATENT_BYTES)[lane >> 2] = scale;
  if (values) {
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const __nv_bfloat162 two =
          __floats2bfloat162_rn((x[2 * e] - kToInteger) * sf, (x[2 * e + 1] - kToInteger) * sf);
      v[e] = *reinterpret_cast<const uint32_t*>(&two);
    }
    uint4* o = reinterpret_cast<uint4*>(values + 16 * lane);
    o[0] = make_uint4(v[0], v[1], v[2], v[3]);
    o[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }

  // position part: the angle's turns modulo one are the low 64 bits of
  // pos * turn, off by at most 2 pos * 2^-64 turns; its top 32 bits as a signed
  // number are half turns in [-1, 1).
  const uint64_t turns = (uint64_t)(uint32_t)p * a.turn[lane];
  float sn, cs;
  sincospif((float)(int32_t)(turns >> 32) * 4.656612873077393e-10f, &sn, &cs);
  const __nv_bfloat16 o0 = __float2bfloat16_rn(r0 * cs - r1 * sn), o1 = __float2bfloat16_rn(r1 * cs + r0 * sn);
  __nv_bfloat16* rd = reinterpret_cast<__nv_bfloat16*>(dst + KVO_LATENT_BYTES + 16);
  __nv_bfloat16* vd = reinterpret_cast<__nv_bfloat16*>(values) + KVO_LATENT_BYTES;
  if (a.interleaved) {
    const __nv_bfloat162 two = __halves2bfloat162(o0, o1);
    reinterpret_cast<__nv_bfloat162*>(rd)[lane] = two;
    if (values) reinterpret_cast<__nv_bfloat162*>(vd)[lane] = two;
  } else {
    rd[i0] = o0;
    rd[i1] = o1;
    if (values) {
      vd[i0] = o0;
      vd[i1] = o1;
    }
  }

  if (!a.key) return;
  if (a.key_type == KVO_BF16) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(k[0], k[1]), hi = __floats2bfloat162_rn(k[2], k[3]);
    reinterpret_cast<uint2*>(a.cache.keys + row * (2 * KVO_KEY_VALUES))[lane] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    return;
  }
  // magnitudes as integers order like the floats, infinities and NaNs above all
  uint32_t big = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) big = max(big, __float_as_uint(k[e]) & 0x7fffffffu);
  big = __reduce_max_sync(0xffffffffu, big);
  // 448 = 1.75 * 2^8: the smallest 2^e with 448 * 2^e >= amax, from amax's bits
  int e = (int)(big >> 23) - 127 - 8 + ((big & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, -100);
  const bool whole = big < 0x7f800000u;
  const float down = whole ? __uint_as_float((uint32_t)(127 - e) << 23) : 0.0f;
  uint32_t bytes = 0;
  if (whole) {
    const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(k[0] * down, k[1] * down), __NV_SATFINITE,
                                                             __NV_E4M3);
    const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(k[2] * down, k[3] * down), __NV_SATFINITE,
                                                             __NV_E4M3);
    bytes = (uint32_t)lo | (uint32_t)hi << 16;
  }
  reinterpret_cast<uint32_t*>(a.cache.keys + row * KVO_KEY_VALUES)[lane] = bytes;
  if (lane == 0) a.cache.key_scales[row] = __uint_as_float(whole ? (uint32_t)(127 + e) << 23 : 0x7fffffffu);
}

// inv_freq / 2 pi modulo 1, times 2^64: the quotient in two doubles (1 / 2 pi
// as the nearest double and what that leaves), so that no far position sees
// the rounding of either.  A negative one's is the other's complement: as a
// double, a whole turn less a small part would lose bits of the part.
uint64_t turns_of(double inv_freq) {
  constexpr double kInv = 0.15915494309189535, kInvLow = -9.839338337591243e-18;
  const double x = std::fabs(inv_freq), hi = x * kInv;
  const double lo = std::fma(x, kInv, -hi) + x * kInvLow;
  const uint64_t u = (uint64_t)((hi - std::floor(hi)) * 18446744073709551616.0) +
                     (uint64_t)(int64_t)(lo * 18446744073709551616.0);
  return inv_freq < 0.0 ? 0 - u : u;
}

}  // namespace
}  // namespace kvo

extern "C" kvo_status kvo_append_tokens(kvo_ctx* ctx, const kvo_cache* cache, const kvo_tokens* t, void* stream) {
  using namespace kvo;
  uint32_t* status = nullptr;
  if (!ctx || !cache_ok(cache) || !t || !cache_rows_ok(cache) || t->n < 0) return KVO_EINVAL;
  const int64_t size = t->dtype == KVO_FP32 ? 4 : t->dtype == KVO_BF16 || t->dtype == KVO_FP16 ? 2 : 0;
  if (!size || !t->inv_freq) return KVO_EINVAL;
  for (int i = 0; i < 32; ++i)
    if (!(std::fabs(t->inv_freq[i]) <= kMaxInvFreq)) return KVO_EINVAL;
  if (t->key && !cache_keys_ok(cache)) return KVO_EINVAL;
  if (!aligned(t->out_bf16, 16) || !aligned(t->seq, 4) || !aligned(t->pos, 4) || !aligned(t->place, 4))
    return KVO_EINVAL;
  if (t->n > 0) {
    if (!t->latent || !t->rope || !t->pos) return KVO_EINVAL;
    const struct {
      const void* p;
      int64_t ld, values;
    } in[3] = {{t->latent, t->latent_ld, KVO_LATENT_BYTES}, {t->rope, t->rope_ld, 64}, {t->key, t->key_ld, KVO_KEY_VALUES}};
    for (const auto& x : in) {
      if (!x.p) continue;
      if (!aligned(x.p, 16) || (x.ld * size) % 16 != 0) return KVO_EINVAL;
      if (t->n > 1 && x.ld < x.values) return KVO_EINVAL;
    }
    if (t->n > (int64_t)INT32_MAX * (kAppendThreads / 32)) return KVO_EINVAL;
  }
  const kvo_status st = usable_status(ctx, &status);
  if (st != KVO_OK) return st;
  if (t->n == 0) return KVO_OK;

  AppendArgs a = {};
  a.cache = cache_view(*cache);
  a.latent = static_cast<const uint8_t*>(t->latent);
  a.rope = static_cast<const uint8_t*>(t->rope);
  a.key = static_cast<const uint8_t*>(t->key);
  a.seq = t->seq;
  a.pos = t->pos;
  a.place = t->place;
  a.out_bf16 = t->out_bf16;
  a.status = status;
  a.latent_ld = t->latent_ld;
  a.rope_ld = t->rope_ld;
  a.key_ld = t->key_ld;
  a.n = t->n;
  for (int i = 0; i < 32; ++i) a.turn[i] = turns_of(t->inv_freq[i]);
  a.interleaved = t->interleaved ? 1u : 0u;
  a.key_type = (uint32_t)cache->key_type;
  const dim3 grid((unsigned)((t->n + kAppendThreads / 32 - 1) / (kAppendThreads / 32)));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const auto kernel_for = [&](auto placed) {
    constexpr bool kPlaced = decltype(placed)::value;
    return t->dtype == KVO_BF16   ? append_tokens_kernel<__nv_bfloat16, kPlaced>
           : t->dtype == KVO_FP16 ? append_tokens_kernel<__half, kPlaced>
                                  : append_tokens_kernel<float, kPlaced>;
  };
  const auto kernel = t->place ? kernel_for(std::true_type{}) : kernel_for(std::false_type{});
  return launch_early(kernel, grid, kAppendThreads, 0, s, a) == cudaSuccess ? KVO_OK : KVO_ECUDA;
}
