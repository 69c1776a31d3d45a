// Fragments of 16 x 8 x 16 products over pages of the 8-bit cache, which the decode (kv8_decode.cu) and the decode of what sequences
// with shared prefixes have of their own (kv8_shared.cu) are made of.
#pragma once

#include "kv8_attn.cuh"

namespace oscar {
namespace kv8 {

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same, onto zeros.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Byte offset of 16-byte chunk c of row r in a stage (the tensor copy's swizzle).
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ uint32_t pack_half2(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Q: lane (g, t) holds query g, channels 16 ks + 4 t .. + 3 (k = 2t, 2t+1, 2t+8, 2t+9 of k-step ks), of `row` (zeros where there
// is none); returns what its logits are to be multiplied with.
template <int D>
__device__ __forceinline__ float load_q(const __nv_bfloat16* row, bool there, int t, float scale_log2, uint32_t (&qa)[D / 16][2]) {
  constexpr int kKs = D / 16;
  const uint2* src = reinterpret_cast<const uint2*>(row + 4 * t);
  uint2 x[kKs];
  uint32_t mx = 0;
#pragma unroll
  for (int ks = 0; ks < kKs; ++ks) {
    x[ks] = there ? __ldg(src + 4 * ks) : make_uint2(0, 0);
    mx = __vmaxu2(mx, __vmaxu2(x[ks].x & 0x7fff7fffu, x[ks].y & 0x7fff7fffu));
  }
  mx = max(mx & 0xffffu, mx >> 16);
  mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  const int e = min(max(static_cast<int>(mx >> 7) - 127, -126), 126);
  const float inv = pow2i(-e);
  const float qs = pow2i(e) * scale_log2;
#pragma unroll
  for (int ks = 0; ks < kKs; ++ks) {
    qa[ks][0] = pack_half2(__uint_as_float(x[ks].x << 16) * inv, __uint_as_float(x[ks].x & 0xffff0000u) * inv);
    qa[ks][1] = pack_half2(__uint_as_float(x[ks].y << 16) * inv, __uint_as_float(x[ks].y & 0xffff0000u) * inv);
  }
  return qs;
}

}  // namespace kv8
}  // namespace oscar
