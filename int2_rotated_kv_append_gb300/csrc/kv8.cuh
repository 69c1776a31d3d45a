// Element formats of the 8-bit paged cache: e4m3 or int8 codes, one power-of-two scale per
// block of 16 tokens and KV head.  A power of two makes code * scale exact in bf16 (at most
// 8 significant bits) and a change of scale exact but for what falls below the new step.
#pragma once

#include <math.h>

#include "common.cuh"
#include "ptx.cuh"

namespace oscar {
namespace kv8 {

constexpr int kE4M3 = OSCAR_KV8_E4M3;
constexpr int kInt8 = OSCAR_KV8_INT8;
constexpr int kExpLo = -100;
constexpr int kMaxLen = 0x7fffffff - 2 * kPageSize;  // positions, rounded up to whole pages, are 32-bit numbers

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

// The two 16-bit halves of a word, each a pair of codes -> two fp16 pairs, exact.
template <int F>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (F == kE4M3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // with the sign bit flipped a code is c + 128: as the low byte of an fp16 in [1024, 2048) it
    // counts ones, so subtracting 1152 leaves c
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// The same, times a power of two f (both halves), f1152 = 1152 f: one operation more for e4m3, none for int8.
template <int F>
__device__ __forceinline__ void codes_to_f16_scaled(uint32_t w, __half2 f, __half2 f1152, uint32_t& lo, uint32_t& hi) {
  if constexpr (F == kE4M3) {
    codes_to_f16<F>(w, lo, hi);
    const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&lo), f);
    const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&hi), f);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  } else {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hfma2(*reinterpret_cast<const __half2*>(&a), f, __hneg2(f1152));
    const __half2 y = __hfma2(*reinterpret_cast<const __half2*>(&b), f, __hneg2(f1152));
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// log2 of a scale, a power of two; -infinity for 0.
__device__ __forceinline__ float scale_log2_of(float s) {
  return s > 0.f ? static_cast<float>(static_cast<int>(__float_as_uint(s) >> 23) - 127) : -INFINITY;
}

// Positions of a sequence that a row at position `row` sees: [0, sink_end) and [lo, row], as a list of
// pages: the first nA pages, then pages first_b ... of the window (a page that holds both ends is
// in the first part).
struct Visible {
  int sink_end, lo, end;  // positions
  int n_a, first_b, n;    // pages
  __device__ __forceinline__ int page(int v) const { return v < n_a ? v : first_b + v - n_a; }
  __device__ __forceinline__ bool sees(int pos) const { return pos < end && (pos < sink_end || pos >= lo); }
};

// Rows first_row .. last_row (>= 0) of one sequence together.
__device__ __forceinline__ Visible visible(int first_row, int last_row, int sink, int window) {
  Visible v;
  v.end = last_row + 1;
  v.lo = window > 0 ? max(0, first_row - window + 1) : 0;
  v.sink_end = min(sink, v.lo);
  v.n_a = (v.sink_end + kPageSize - 1) / kPageSize;
  v.first_b = max(v.lo / kPageSize, v.n_a);
  v.n = v.n_a + max(0, (v.end + kPageSize - 1) / kPageSize - v.first_b);
  return v;
}

// Host bound on Visible::n for lengths up to max_seq_len and runs of `rows` rows.
static inline long long max_visible_pages(long long max_seq_len, int sink, int window, long long rows) {
  const long long all = (max_seq_len + kPageSize - 1) / kPageSize;
  if (window <= 0) return all;
  const long long some = (static_cast<long long>(sink) + kPageSize - 1) / kPageSize +
                         (window + rows + 2LL * kPageSize - 3) / kPageSize + 1;
  return some < all ? some : all;
}

}  // namespace kv8
}  // namespace oscar
