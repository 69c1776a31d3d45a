// What the decode and the extend over the 8-bit paged cache share: arguments and their checks,
// the page tensor map, the merge of split partials.
#pragma once

#include <math.h>

#include "kv8.cuh"
#include "umma.cuh"

namespace oscar {
namespace kv8 {

struct AttnArgs {
  const __nv_bfloat16* q;
  const uint8_t* pages;
  const float* scales;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* q_start;  // extend: rows of sequence b from q_start[b] on
  __nv_bfloat16* out;
  int batch, rows, max_rows, Hq, H, num_pages, max_pages, max_seq_len, sink, window;
  float scale_log2;
};

static inline bool bad_format(int f) { return f != OSCAR_KV8_E4M3 && f != OSCAR_KV8_INT8; }

// Pointer and workspace checks, and the arguments of the kernels.
static inline oscar_status_t make_args(const oscar_dims_t* dims, int batch, int rows, int max_rows, int max_seq_len,
                                       const void* q, const int32_t* q_start, const uint8_t* pages,
                                       const float* scales, const int32_t* page_table, const int32_t* seq_lens,
                                       int sink, int window, float sm_scale, void* out, const void* workspace,
                                       size_t need, size_t workspace_bytes, AttnArgs* a) {
  if (!q || !pages || !scales || !page_table || !seq_lens || !out || !workspace) return OSCAR_ERR_INVALID_ARG;
  if (misaligned16(q) || misaligned16(pages) || misaligned16(scales) || misaligned16(out)) return OSCAR_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return OSCAR_ERR_INVALID_ARG;
  if (workspace_bytes < need) return OSCAR_ERR_WORKSPACE;
  if (static_cast<long long>(dims->num_pages) * dims->num_kv_heads > 0x7fffffffLL) return OSCAR_ERR_UNSUPPORTED;
  if (window >= max_seq_len) window = 0;  // hides nothing
  const float scale = sm_scale > 0.f ? sm_scale : 1.0f / sqrtf(static_cast<float>(dims->head_dim));
  *a = AttnArgs{static_cast<const __nv_bfloat16*>(q), pages, scales, page_table, seq_lens, q_start,
                static_cast<__nv_bfloat16*>(out), batch, rows, max_rows, dims->num_q_heads, dims->num_kv_heads,
                dims->num_pages, dims->max_pages_per_seq, max_seq_len, sink, window, scale * 1.4426950408889634f};
  return OSCAR_OK;
}

// The pool as a tensor [pages x heads][32 rows: K then V][D] of bytes; a box is one page of one head, its
// 16-byte chunks swizzled within 128-byte (D = 128) or 64-byte (D = 64) rows.
static inline bool encode_page_map(const oscar_dims_t* d, const uint8_t* pages, CUtensorMap* map) {
  umma::EncodeTiledFn fn = umma::encode_tiled();
  if (fn == nullptr) return false;
  const cuuint64_t D = static_cast<cuuint64_t>(d->head_dim);
  const cuuint64_t size[3] = {D, 2 * kPageSize, static_cast<cuuint64_t>(d->num_pages) * d->num_kv_heads};
  const cuuint64_t stride[2] = {D, 2 * kPageSize * D};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(D), 2 * kPageSize, 1}, one[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(pages), size, stride, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

__device__ __forceinline__ int clamped_len(const AttnArgs& a, int b) {
  const int L = __ldg(a.seq_lens + b);
  if (L < 0 || L > a.max_seq_len) {
    record_error(OSCAR_DEVERR_SEQ_LEN);
    return L < 0 ? 0 : a.max_seq_len;
  }
  return L;
}

// 2^e as the product of two floats, for |e| < 250 (below: as good as 0; NaN, of a row that is NaN or empty, as that).
__device__ __forceinline__ void pow2_pair(float e, float& f, float& g) {
  e = fmaxf(e, -250.f);
  const float h = truncf(0.5f * e);
  f = fast_exp2(h);
  g = fast_exp2(e - h);
}

// Numerator and denominator of a row have a unit each: l counts 2^m (weights alone) and o counts 2^(m + r) (weights times V
// scales: near the largest of these products).  With one unit for both, values near either end of the scales' range would
// leave fp32; r is kept, not m + r, which rounds where logits are large.  Two units may be further apart than a float's exponents
// reach: o goes from one to another by a pair.

// Four channels of an output row: 2^e o / l, e the unit r; 0 where nothing was attended (a NaN of the query stays one).
__device__ __forceinline__ void store_out4(__nv_bfloat16* out, float4 o, float l, float e) {
  float f, g;
  pow2_pair(e, f, g);
  const float inv = l == 0.f ? 0.f : f / l;
  const __nv_bfloat162 x = __floats2bfloat162_rn(o.x * inv * g, o.y * inv * g),
                       y = __floats2bfloat162_rn(o.z * inv * g, o.w * inv * g);
  *reinterpret_cast<uint2*>(out) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

// One warp: partials first, first + step, ... of n (o [n][D] unnormalised, ml [n][4] = m, l, r, -; -infinity for the units of a
// partial of nothing): l and four channels r of lane's c4 = lane % (D / 4), in units of the largest m and m + r of all n, the
// latter e above the former.  Eight partials are in flight at once, the first of them while the maxima are found.
template <int D>
__device__ __forceinline__ void merge_part(const float* o, const float* ml, int n, int first, int step, int lane,
                                           float& l, float4& r, float& e) {
  constexpr int kSub = 128 / D, kFly = 8;  // D = 64: two half warps take every second partial
  const int sub = lane / (D / 4), c4 = lane % (D / 4);
  l = 0.f;
  r = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 x[kFly], p[kFly];
  auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kFly; ++k) {
      const int i = i0 + k * step * kSub;
      p[k] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
      x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        p[k] = *reinterpret_cast<const float4*>(ml + 4 * i);
        x[k] = *reinterpret_cast<const float4*>(o + static_cast<size_t>(i) * D + 4 * c4);
      }
    }
  };
  int i0 = first * kSub + sub;
  load(i0);
  float M = -INFINITY, R = -INFINITY;  // a lane's own, then all lanes'
  for (int i = lane; i < n; i += 32) {
    const float4 v = *reinterpret_cast<const float4*>(ml + 4 * i);
    if (v.x > -INFINITY) {
      const float m = fmaxf(M, v.x);
      R = fmaxf(R + (M - m), v.z + (v.x - m));
      M = m;
    }
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, M, off), r2 = __shfl_xor_sync(0xffffffffu, R, off);
    const float m = fmaxf(M, m2);
    if (m > -INFINITY) R = fmaxf(R + (M - m), r2 + (m2 - m));
    M = m;
  }
  e = R;
  const float base = M == -INFINITY ? 0.f : M, base_r = R == -INFINITY ? 0.f : R;
  while (true) {
#pragma unroll
    for (int k = 0; k < kFly; ++k) {
      const float d = p[k].x - base;
      l = fmaf(fast_exp2(d), p[k].y, l);  // (a factor of 0 for a partial of nothing)
      float f, g;
      pow2_pair(d + p[k].z - base_r, f, g);
      r.x = fmaf(f, x[k].x * g, r.x); r.y = fmaf(f, x[k].y * g, r.y);
      r.z = fmaf(f, x[k].z * g, r.z); r.w = fmaf(f, x[k].w * g, r.w);
    }
    i0 += step * kSub * kFly;
    if (!__any_sync(0xffffffffu, i0 < n)) break;
    load(i0);
  }
  if (kSub == 2) {
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    r.x += __shfl_xor_sync(0xffffffffu, r.x, 16);
    r.y += __shfl_xor_sync(0xffffffffu, r.y, 16);
    r.z += __shfl_xor_sync(0xffffffffu, r.z, 16);
    r.w += __shfl_xor_sync(0xffffffffu, r.w, 16);
  }
}

// One warp: the merge of n partials into a row of the output.
template <int D>
__device__ __forceinline__ void merge_row(const float* o, const float* ml, int n, __nv_bfloat16* out, int lane) {
  float l, e;
  float4 r;
  merge_part<D>(o, ml, n, 0, 1, lane, l, r, e);
  if (lane < D / 4) store_out4(out + 4 * lane, r, l, e);
}

}  // namespace kv8
}  // namespace oscar
