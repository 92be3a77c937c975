// Block quantization to 8-bit floating point, shared by every kernel that
// writes codes of weights or rows (the optimizer's states have a scale and an
// inverse of their own, optim_multi.cu):
//   amax  = max over the block's finite |v|, at least 2^-100
//   scale = fl32(amax / F),  F = 448 (e4m3) or 57344 (e5m2)
//   code  = fp8_rn(clamp(fl32(v * fl32(F / amax)), -F, F)), NaN unless v is finite
// One division per block instead of one per value; the product is at most one
// fp32 step away from v / scale, far below the code's own step. The floor of
// 2^-100 keeps F / amax finite and gives a block of zeros a usable scale.
#pragma once

#include <cfloat>
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace qlora {

enum Fp8Format : int { kE4M3 = 0, kE5M2 = 1 };
constexpr int kFp8Block = 128;
constexpr float kFp8Least = 7.888609052210118e-31f;  // 2^-100

template <int FMT>
__device__ __forceinline__ constexpr float fp8_top() {
  return FMT == kE4M3 ? 448.0f : 57344.0f;
}

// What a value that is not finite asks for costs nothing where there is none:
// a maximum of fabsf ignores NaN, and NaN * inv converts to the NaN code; only
// an infinity, which shows as an infinite maximum, needs the next two.
//
// |v| where v is finite, else 0: what enters a block's maximum
__device__ __forceinline__ float fp8_mag(float v) {
  const float a = fabsf(v);
  return a <= FLT_MAX ? a : 0.0f;
}

// The value to convert: v * inv, or NaN where v is not finite (v - v is then NaN,
// else 0; a negative zero added leaves a product of either sign as it is).
__device__ __forceinline__ float fp8_scaled(float v, float inv) { return fmaf(v, inv, -(v - v)); }

// Two values to codes (lo in the low byte): round to nearest even, saturate, NaN stays NaN.
template <int FMT>
__device__ __forceinline__ uint32_t fp8_pack2(float lo, float hi) {
  uint16_t d;
  if (FMT == kE4M3)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

template <int FMT>
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
  return fp8_pack2<FMT>(a, b) | (fp8_pack2<FMT>(c, d) << 16);
}

// Two codes to fp32 (exact: every code is a half).
template <int FMT>
__device__ __forceinline__ float2 fp8_unpack2(uint32_t codes) {
  uint32_t h;
  const uint16_t c = static_cast<uint16_t>(codes);
  if (FMT == kE4M3)
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  else
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(c));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

}  // namespace qlora
