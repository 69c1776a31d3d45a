// Attention over the 8-bit paged cache: decode (one row per sequence) and extend (the last
// rows of each sequence), full or with a sliding window and sinks.
//
// One warp per (row, query head): lane l holds channels l, l + 32, ... of q and of the output,
// positions one after another with an online softmax.
#include <math.h>

#include "kv8.cuh"

namespace {

using namespace oscar;
using namespace oscar::kv8;

struct AttnArgs {
  const __nv_bfloat16* q;
  const uint8_t* pages;
  const float* scales;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* q_start;  // null: row b is the last position of sequence b
  __nv_bfloat16* out;
  int batch, rows, max_rows, Hq, H, num_pages, max_pages, max_seq_len, sink, window;
  float scale_log2;
};

__device__ __forceinline__ int clamped_len(const AttnArgs& a, int b) {
  const int L = a.seq_lens[b];
  if (L < 0 || L > a.max_seq_len) {
    record_error(OSCAR_DEVERR_SEQ_LEN);
    return L < 0 ? 0 : a.max_seq_len;
  }
  return L;
}

template <int F, int D>
__global__ void __launch_bounds__(128) kv8_attn_kernel(AttnArgs a) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31;
  const int hq = blockIdx.y * 4 + (threadIdx.x >> 5);
  const int b = blockIdx.z;
  if (hq >= a.Hq) return;
  const int L = clamped_len(a, b);
  int row = b, pos = L - 1;
  if (a.q_start != nullptr) {
    const int q0 = a.q_start[b], q1 = a.q_start[b + 1], n = q1 - q0;
    if (n < 0 || n > a.max_rows || q0 < 0 || q1 > a.rows) {
      record_error(OSCAR_DEVERR_POSITION);
      return;
    }
    if (static_cast<int>(blockIdx.x) >= n) return;
    row = q0 + blockIdx.x;
    pos = L - n + blockIdx.x;
    if (pos < 0) record_error(OSCAR_DEVERR_POSITION);
  }
  const int h = hq / (a.Hq / a.H);
  const size_t rq = (static_cast<size_t>(row) * a.Hq + hq) * D;
  float q[C], o[C], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    q[c] = __bfloat162float(a.q[rq + lane + 32 * c]);
    o[c] = 0.f;
  }
  const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  const int sink_end = min(a.sink, lo);
  for (int j = 0; j <= pos; ++j) {
    if (j >= sink_end && j < lo) j = lo;
    const int pid = a.page_table[static_cast<size_t>(b) * a.max_pages + j / kPageSize];
    if (pid < 0 || pid >= a.num_pages) {
      record_error(OSCAR_DEVERR_PAGE_ID);
      continue;
    }
    const size_t block = (static_cast<size_t>(pid) * a.H + h) * 2;
    const uint8_t* k = a.pages + block * (kPageSize * D) + (j % kPageSize) * D + lane;
    const uint8_t* v = k + kPageSize * D;
    float s = 0.f;
    float x[4];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      decode4<F>(k[32 * c], x);
      s = fmaf(q[c], x[0], s);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= a.scales[block] * a.scale_log2;
    const float m_new = fmaxf(m, s);
    const float alpha = fast_exp2(m - m_new), p = fast_exp2(s - m_new);
    m = m_new;
    l = l * alpha + p;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      decode4<F>(v[32 * c], x);
      o[c] = o[c] * alpha + p * x[0] * a.scales[block + 1];
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) a.out[rq + lane + 32 * c] = __float2bfloat16_rn(l > 0.f ? o[c] / l : 0.f);
}

oscar_status_t attention(const oscar_dims_t* dims, int kv_format, int batch, int rows, int max_seq_len, int max_rows,
                         int pages_per_split, const void* q, const int32_t* q_start, const uint8_t* pages,
                         const float* scales, const int32_t* page_table, const int32_t* seq_lens, int sink,
                         int window, float sm_scale, void* out, void* workspace, size_t need, size_t workspace_bytes,
                         void* stream) {
  if (!q || !pages || !scales || !page_table || !seq_lens || !out || !workspace) return OSCAR_ERR_INVALID_ARG;
  if (misaligned16(q) || misaligned16(pages) || misaligned16(scales) || misaligned16(out)) return OSCAR_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return OSCAR_ERR_INVALID_ARG;
  if (need == 0) return OSCAR_ERR_INVALID_ARG;
  if (workspace_bytes < need) return OSCAR_ERR_WORKSPACE;
  const float scale = sm_scale > 0.f ? sm_scale : 1.0f / sqrtf(static_cast<float>(dims->head_dim));
  AttnArgs a{static_cast<const __nv_bfloat16*>(q), pages, scales, page_table, seq_lens, q_start,
             static_cast<__nv_bfloat16*>(out), batch, rows, max_rows, dims->num_q_heads, dims->num_kv_heads,
             dims->num_pages, dims->max_pages_per_seq, max_seq_len, sink, window, scale * 1.4426950408889634f};
  const dim3 grid(max_rows, (dims->num_q_heads + 3) / 4, batch);
  const bool d128 = dims->head_dim == 128;
  auto* kernel = kv_format == OSCAR_KV8_E4M3 ? (d128 ? kv8_attn_kernel<kE4M3, 128> : kv8_attn_kernel<kE4M3, 64>)
                                             : (d128 ? kv8_attn_kernel<kInt8, 128> : kv8_attn_kernel<kInt8, 64>);
  kernel<<<grid, 128, 0, as_stream(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

bool bad_format(int f) { return f != OSCAR_KV8_E4M3 && f != OSCAR_KV8_INT8; }

}  // namespace

extern "C" size_t oscar_kv8_decode_workspace_bytes(const oscar_dims_t* dims, int32_t batch, int32_t max_seq_len,
                                                   int32_t pages_per_split, int32_t sink_len, int32_t window_len) {
  if (check_dims(dims) != OSCAR_OK || batch < 0 || batch > 65535 || max_seq_len < 0 || pages_per_split < 0 ||
      sink_len < 0 || window_len < 0 ||
      max_seq_len > static_cast<long long>(dims->max_pages_per_seq) * kPageSize)
    return 0;
  return 256;
}

extern "C" oscar_status_t oscar_kv8_decode(const oscar_dims_t* dims, int32_t kv_format, int32_t batch,
                                           int32_t max_seq_len, int32_t pages_per_split, const void* q,
                                           const uint8_t* kv8_pages, const float* kv8_scales,
                                           const int32_t* page_table, const int32_t* seq_lens, int32_t sink_len,
                                           int32_t window_len, float sm_scale, void* out, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  const oscar_status_t st = check_dims(dims);
  if (st != OSCAR_OK) return st;
  if (bad_format(kv_format) || batch < 0 || max_seq_len < 0 || pages_per_split < 0 || sink_len < 0 || window_len < 0)
    return OSCAR_ERR_INVALID_ARG;
  if (batch == 0) return OSCAR_OK;
  return attention(dims, kv_format, batch, batch, max_seq_len, 1, pages_per_split, q, nullptr, kv8_pages, kv8_scales,
                   page_table, seq_lens, sink_len, window_len, sm_scale, out, workspace,
                   oscar_kv8_decode_workspace_bytes(dims, batch, max_seq_len, pages_per_split, sink_len, window_len),
                   workspace_bytes, stream);
}

extern "C" size_t oscar_kv8_extend_varlen_workspace_bytes(const oscar_dims_t* dims, int32_t batch, int32_t num_rows,
                                                          int32_t max_seq_len, int32_t max_rows_per_seq,
                                                          int32_t pages_per_split, int32_t sink_len,
                                                          int32_t window_len) {
  if (num_rows < 0 || max_rows_per_seq < 0) return 0;
  return oscar_kv8_decode_workspace_bytes(dims, batch, max_seq_len, pages_per_split, sink_len, window_len);
}

extern "C" oscar_status_t oscar_kv8_extend_varlen(const oscar_dims_t* dims, int32_t kv_format, int32_t batch,
                                                  int32_t num_rows, int32_t max_seq_len, int32_t max_rows_per_seq,
                                                  int32_t pages_per_split, const void* q, const int32_t* q_start,
                                                  const uint8_t* kv8_pages, const float* kv8_scales,
                                                  const int32_t* page_table, const int32_t* seq_lens,
                                                  int32_t sink_len, int32_t window_len, float sm_scale, void* out,
                                                  void* workspace, size_t workspace_bytes, void* stream) {
  const oscar_status_t st = check_dims(dims);
  if (st != OSCAR_OK) return st;
  if (bad_format(kv_format) || batch < 0 || num_rows < 0 || max_seq_len < 0 || max_rows_per_seq < 0 ||
      pages_per_split < 0 || sink_len < 0 || window_len < 0)
    return OSCAR_ERR_INVALID_ARG;
  if (num_rows == 0) return OSCAR_OK;
  if (batch == 0 || max_rows_per_seq == 0 || !q_start) return OSCAR_ERR_INVALID_ARG;
  return attention(dims, kv_format, batch, num_rows, max_seq_len, max_rows_per_seq, pages_per_split, q, q_start,
                   kv8_pages, kv8_scales, page_table, seq_lens, sink_len, window_len, sm_scale, out, workspace,
                   oscar_kv8_extend_varlen_workspace_bytes(dims, batch, num_rows, max_seq_len, max_rows_per_seq,
                                                           pages_per_split, sink_len, window_len),
                   workspace_bytes, stream);
}

oscar_status_t oscar_internal_kv8_attn_errors(uint32_t* flags, int reset) {
  return oscar::read_unit_errors(flags, reset) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}
