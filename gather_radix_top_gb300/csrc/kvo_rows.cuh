// Cache rows as the attention kernels take them: int8 latents to bf16, and the
// exponentials of their logits.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace kvo {

constexpr float kLog2e = 1.4426950408889634f;

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

// x = x * scale + (a, b), products and sums of two, as one instruction each; the largest of three.
__device__ __forceinline__ void fma_two(float& x, float& y, float scale, float a, float b) {
  asm("{\n .reg .b64 v, s, t;\n mov.b64 v, {%0, %1};\n mov.b64 s, {%2, %2};\n mov.b64 t, {%3, %4};\n"
      " fma.rn.f32x2 v, v, s, t;\n mov.b64 {%0, %1}, v;\n}"
      : "+f"(x), "+f"(y)
      : "f"(scale), "f"(a), "f"(b));
}
__device__ __forceinline__ void mul_two(float& x, float& y, float by) {
  asm("{\n .reg .b64 v, s;\n mov.b64 v, {%0, %1};\n mov.b64 s, {%2, %2};\n mul.rn.f32x2 v, v, s;\n mov.b64 {%0, %1}, v;\n}"
      : "+f"(x), "+f"(y)
      : "f"(by));
}
__device__ __forceinline__ void add_two(float& x, float& y, float a, float b) {
  asm("{\n .reg .b64 v, t;\n mov.b64 v, {%0, %1};\n mov.b64 t, {%2, %3};\n add.rn.f32x2 v, v, t;\n mov.b64 {%0, %1}, v;\n}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
__device__ __forceinline__ float max_three(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// All lanes' loads of these values have come when this returns: an arrival that
// lets a copy overwrite what they read is not held up by loads that are still
// queued (behind other warps' stores, for longer than a copy takes).  The vote
// needs the values; its outcome changes nothing.
__device__ __forceinline__ void loads_are_in(uint32_t all) {
  if (__any_sync(0xffffffffu, all == 0x9e3779b9u)) __nanosleep(0);
}
__device__ __forceinline__ uint32_t mixed(uint4 v) { return v.x ^ v.y ^ v.z ^ v.w; }

// Whether any of eight fp16 is infinite or NaN.
__device__ __forceinline__ bool any_not_finite(uint4 eight) {
  constexpr uint32_t kInf = 0x7c007c00u;
  return (__vcmpeq2(eight.x & kInf, kInf) | __vcmpeq2(eight.y & kInf, kInf) | __vcmpeq2(eight.z & kInf, kInf) |
          __vcmpeq2(eight.w & kInf, kInf)) != 0;
}

}  // namespace kvo
