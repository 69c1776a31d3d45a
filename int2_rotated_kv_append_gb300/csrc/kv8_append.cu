// Quantising append of the 8-bit paged cache (oscar_kv8_append): bf16 rows -> codes and one
// power-of-two scale per block of 16 tokens and KV head.
//
// One warp per (page, KV head, K | V) block: at most 16 rows of D bf16, all loaded up front
// (16 bytes a lane and row group, so a row's bytes are consecutive lanes), the block's largest
// magnitude by one warp butterfly, codes from the registers.  Nothing is read twice and nothing is shared
// between warps.  Bound by the bytes: 2 in and 1 out per element (six prompts, 56 thousand tokens of 8 heads, D = 128:
// 55 us, 6.3 TB/s, 93% of a plain copy's rate; one token of each of 64 sequences: 2.4 us).
#include "kv8.cuh"

namespace {

using namespace oscar;
using namespace oscar::kv8;

constexpr int kWarps = 4;

struct AppendArgs {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const int32_t* t_start;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* granted;  // null: every sequence
  uint8_t* pages;
  float* scales;
  int H, num_pages, max_pages, max_new;
  long long num_tokens;
};

template <int F, int D>
__global__ void __launch_bounds__(kWarps * 32) kv8_append_kernel(AppendArgs a) {
  constexpr int kLanesPerRow = D / 8;              // 16-byte chunks of a row
  constexpr int kRows = 32 / kLanesPerRow;         // rows per load
  constexpr int kIters = kPageSize / kRows;
  const int lane = threadIdx.x & 31;
  const int unit = blockIdx.y * kWarps + (threadIdx.x >> 5);  // (head, K | V)
  const int b = blockIdx.z;
  const int t0 = __ldg(a.t_start + b), t1 = __ldg(a.t_start + b + 1), L = __ldg(a.seq_lens + b);
  const int n = t1 - t0;
  if (n == 0 || (a.granted != nullptr && __ldg(a.granted + b) == 0)) return;
  if (n < 0 || n > a.max_new || n > L || t0 < 0 || t1 > a.num_tokens || L > a.max_pages * kPageSize) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) record_error(OSCAR_DEVERR_POSITION);
    return;
  }
  const int p_first = L - n;
  const int j = p_first / kPageSize + blockIdx.x;  // page of the sequence
  if (j > (L - 1) / kPageSize || unit >= 2 * a.H) return;
  const int pid = __ldg(a.page_table + static_cast<size_t>(b) * a.max_pages + j);
  if (pid < 0 || pid >= a.num_pages) {
    if (lane == 0) record_error(OSCAR_DEVERR_PAGE_ID);
    return;
  }
  const int h = unit >> 1, side = unit & 1;
  const int o0 = max(p_first - j * kPageSize, 0), o1 = min(L - j * kPageSize, kPageSize);  // new rows of the page
  const int row0 = lane / kLanesPerRow, chunk = lane % kLanesPerRow;
  const __nv_bfloat16* src = (side ? a.v : a.k) + static_cast<size_t>(h) * D + chunk * 8;
  const long long tok0 = static_cast<long long>(t0) + (j * kPageSize - p_first);  // token of the page's row 0
  uint4 x[kIters];
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    const int r = i * kRows + row0;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r >= o0 && r < o1) x[i] = __ldg(reinterpret_cast<const uint4*>(src + (tok0 + r) * a.H * D));
  }
  const size_t block = (static_cast<size_t>(pid) * a.H + h) * 2 + side;
  uint8_t* dst = a.pages + block * (kPageSize * D) + chunk * 8;
  const float stored = o0 > 0 ? a.scales[block] : 0.f;
  // The largest magnitude, as bf16 bits without the sign: they order as the values do,
  // infinity (0x7f80) and NaN above all.
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int c = 0; c < 4; ++c) mx = __vmaxu2(mx, w[c] & 0x7fff7fffu);
  }
  mx = max(mx & 0xffffu, mx >> 16);
  mx = __reduce_max_sync(0xffffffffu, mx);
  const bool has_nan = mx > 0x7f80u;
  if (has_nan) {  // rare: NaN elements become 0, and the maximum is taken anew without them
    if (lane == 0) record_error(OSCAR_DEVERR_VALUE);
    mx = 0;
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if ((w[c] & 0x7fffu) > 0x7f80u) w[c] &= 0xffff0000u;
        if ((w[c] & 0x7fff0000u) > 0x7f800000u) w[c] &= 0xffffu;
        mx = max(mx, max(w[c] & 0x7fffu, (w[c] >> 16) & 0x7fffu));
      }
      x[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    mx = __reduce_max_sync(0xffffffffu, mx);
  }
  mx = min(mx, 0x7f7fu);  // infinities saturate: the scale is that of the largest finite value
  const float need = pow2i(scale_exponent<F>(bf16_bits_to_float(mx)));
  const float scale = fmaxf(stored, need);
  const float inv = 1.f / scale;  // exact: a power of two between 2^-121 and 2^100
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    const int r = i * kRows + row0;
    if (r >= o0 && r < o1) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t o[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float f[4] = {__uint_as_float(w[2 * c] << 16) * inv, __uint_as_float(w[2 * c] & 0xffff0000u) * inv,
                            __uint_as_float(w[2 * c + 1] << 16) * inv,
                            __uint_as_float(w[2 * c + 1] & 0xffff0000u) * inv};
        o[c] = encode4<F>(f);
      }
      *reinterpret_cast<uint2*>(dst + r * D) = make_uint2(o[0], o[1]);
    } else if (r < o0 && scale != stored) {  // an earlier row under a larger scale
      const uint2 old = *reinterpret_cast<const uint2*>(dst + r * D);
      const uint32_t w[2] = {old.x, old.y};
      const float ratio = stored * inv;
      uint32_t o[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float f[4];
        decode4<F>(w[c], f);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] *= ratio;
        o[c] = encode4<F>(f);
      }
      *reinterpret_cast<uint2*>(dst + r * D) = make_uint2(o[0], o[1]);
    }
  }
  if (lane == 0 && scale != stored) a.scales[block] = scale;
}

oscar_status_t append(const oscar_dims_t* dims, int32_t kv_format, int32_t batch, int64_t num_tokens,
                      int32_t max_tokens_per_seq, const void* k, const void* v, const int32_t* t_start,
                      const int32_t* page_table, const int32_t* seq_lens, const int32_t* granted, uint8_t* kv8_pages,
                      float* kv8_scales, void* stream) {
  const oscar_status_t st = check_dims(dims);
  if (st != OSCAR_OK) return st;
  if (kv_format != OSCAR_KV8_E4M3 && kv_format != OSCAR_KV8_INT8) return OSCAR_ERR_INVALID_ARG;
  if (batch < 0 || num_tokens < 0 || num_tokens > 0x7fffffffLL || max_tokens_per_seq < 0) return OSCAR_ERR_INVALID_ARG;
  if (num_tokens == 0) return OSCAR_OK;
  if (batch == 0 || max_tokens_per_seq == 0 || !k || !v || !t_start || !page_table || !seq_lens || !kv8_pages ||
      !kv8_scales)
    return OSCAR_ERR_INVALID_ARG;
  if (misaligned16(k) || misaligned16(v) || misaligned16(kv8_pages) || misaligned16(kv8_scales))
    return OSCAR_ERR_INVALID_ARG;
  const int units = 2 * dims->num_kv_heads;
  const long long most = max_tokens_per_seq < num_tokens ? max_tokens_per_seq : num_tokens;  // of one sequence
  const long long gx = (most + 2 * kPageSize - 2) / kPageSize;
  const int gy = (units + kWarps - 1) / kWarps;
  if (gy > 65535 || batch > 65535) return OSCAR_ERR_UNSUPPORTED;
  if (static_cast<long long>(dims->max_pages_per_seq) * kPageSize > 0x7fffffffLL) return OSCAR_ERR_UNSUPPORTED;
  AppendArgs a{static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), t_start, page_table,
               seq_lens, granted, kv8_pages, kv8_scales, dims->num_kv_heads, dims->num_pages,
               dims->max_pages_per_seq, max_tokens_per_seq, num_tokens};
  const dim3 grid(static_cast<unsigned>(gx), gy, batch);
  const bool d128 = dims->head_dim == 128;
  auto* kernel = kv_format == OSCAR_KV8_E4M3
                     ? (d128 ? kv8_append_kernel<kE4M3, 128> : kv8_append_kernel<kE4M3, 64>)
                     : (d128 ? kv8_append_kernel<kInt8, 128> : kv8_append_kernel<kInt8, 64>);
  kernel<<<grid, kWarps * 32, 0, as_stream(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

}  // namespace

extern "C" oscar_status_t oscar_kv8_append(const oscar_dims_t* dims, int32_t kv_format, int32_t batch,
                                           int64_t num_tokens, int32_t max_tokens_per_seq, const void* k,
                                           const void* v, const int32_t* t_start, const int32_t* page_table,
                                           const int32_t* seq_lens, uint8_t* kv8_pages, float* kv8_scales,
                                           void* stream) {
  return append(dims, kv_format, batch, num_tokens, max_tokens_per_seq, k, v, t_start, page_table, seq_lens, nullptr,
                kv8_pages, kv8_scales, stream);
}

extern "C" oscar_status_t oscar_kv8_append_granted(const oscar_dims_t* dims, int32_t kv_format, int32_t batch,
                                                   int64_t num_tokens, int32_t max_tokens_per_seq, const void* k,
                                                   const void* v, const int32_t* t_start, const int32_t* page_table,
                                                   const int32_t* seq_lens, const int32_t* granted, uint8_t* kv8_pages,
                                                   float* kv8_scales, void* stream) {
  return append(dims, kv_format, batch, num_tokens, max_tokens_per_seq, k, v, t_start, page_table, seq_lens, granted,
                kv8_pages, kv8_scales, stream);
}

oscar_status_t oscar_internal_kv8_append_errors(uint32_t* flags, int reset) {
  return oscar::read_unit_errors(flags, reset) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}
