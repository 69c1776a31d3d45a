// Element formats of the 8-bit paged cache: e4m3 or int8 codes, one power-of-two scale per
// block of 16 tokens and KV head.  A power of two makes code * scale exact in bf16 (at most
// 8 significant bits) and a change of scale exact but for what falls below the new step.
#pragma once

#include "common.cuh"
#include "ptx.cuh"

namespace oscar {
namespace kv8 {

constexpr int kE4M3 = OSCAR_KV8_E4M3;
constexpr int kInt8 = OSCAR_KV8_INT8;
constexpr int kExpLo = -100;

template <int F>
__device__ __forceinline__ constexpr float code_max() { return F == kE4M3 ? 448.f : 127.f; }

// Two e4m3 codes (low byte first) -> two fp16, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}

// Two floats -> two e4m3 codes, round to nearest even, saturating (lo in the low byte).
__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four codes of a 32-bit word -> floats.
template <int F>
__device__ __forceinline__ void decode4(uint32_t w, float (&x)[4]) {
  if constexpr (F == kE4M3) {
    const uint32_t a = e4m3x2_to_f16x2(static_cast<uint16_t>(w)), b = e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16));
    const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
    const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&b));
    x[0] = fa.x; x[1] = fa.y; x[2] = fb.x; x[3] = fb.y;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
  }
}

// Four floats in units of the block's scale -> codes, round to nearest even, saturating.
template <int F>
__device__ __forceinline__ uint32_t encode4(const float (&x)[4]) {
  if constexpr (F == kE4M3) {
    return static_cast<uint32_t>(f32x2_to_e4m3x2(x[0], x[1])) |
           (static_cast<uint32_t>(f32x2_to_e4m3x2(x[2], x[3])) << 16);
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = __float2int_rn(fminf(fmaxf(x[i], -127.f), 127.f));
      w |= (static_cast<uint32_t>(c) & 0xffu) << (8 * i);
    }
    return w;
  }
}

// Exponent of the smallest scale 2^e in range with a <= M * 2^e, for a finite a >= 0 that is a
// normal float or 0.  M = 1.75 * 2^8 (e4m3) or 1.984375 * 2^6 (int8): the significand of a decides
// between two neighbouring exponents.
template <int F>
__device__ __forceinline__ int scale_exponent(float a) {
  const uint32_t u = __float_as_uint(a);
  const int x = static_cast<int>(u >> 23) - 127;  // a = 1.f * 2^x (0 and subnormals fall below the range)
  const uint32_t frac = u & 0x7fffffu;
  const int e = F == kE4M3 ? x - 8 + (frac > 0x600000u) : x - 6 + (frac > 0x7e0000u);
  return min(max(e, kExpLo), F == kE4M3 ? 119 : 121);
}

}  // namespace kv8
}  // namespace oscar
