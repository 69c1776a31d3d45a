// Attention over the 8-bit paged cache: decode (one row per sequence) and extend (the last
// rows of each sequence), full or with a sliding window and sinks.
//
// One warp per (row, query head): lane l holds channels l, l + 32, ... of q and of the output,
// positions one after another with an online softmax.
#include <math.h>

#include "kv8_attn.cuh"

namespace {

using namespace oscar;
using namespace oscar::kv8;

template <int F, int D>
__global__ void __launch_bounds__(128) kv8_attn_kernel(AttnArgs a) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31;
  const int hq = blockIdx.y * 4 + (threadIdx.x >> 5);
  const int b = blockIdx.z;
  if (hq >= a.Hq) return;
  const int L = clamped_len(a, b);
  int row = b, pos = L - 1;
  if (true) {
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

template <int F, int D>
void launch(const AttnArgs& a, cudaStream_t stream) {
  kv8_attn_kernel<F, D><<<dim3(a.max_rows, (a.Hq + 3) / 4, a.batch), 128, 0, stream>>>(a);
}

}  // namespace

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
  const size_t need = oscar_kv8_extend_varlen_workspace_bytes(dims, batch, num_rows, max_seq_len, max_rows_per_seq,
                                                              pages_per_split, sink_len, window_len);
  if (need == 0) return OSCAR_ERR_INVALID_ARG;
  AttnArgs a;
  const oscar_status_t sa = make_args(dims, batch, num_rows, max_rows_per_seq, max_seq_len, q, q_start, kv8_pages,
                                      kv8_scales, page_table, seq_lens, sink_len, window_len, sm_scale, out, workspace,
                                      need, workspace_bytes, &a);
  if (sa != OSCAR_OK) return sa;
  cudaStream_t s = as_stream(stream);
  const bool d128 = dims->head_dim == 128;
  if (kv_format == OSCAR_KV8_E4M3) d128 ? launch<kE4M3, 128>(a, s) : launch<kE4M3, 64>(a, s);
  else d128 ? launch<kInt8, 128>(a, s) : launch<kInt8, 64>(a, s);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

oscar_status_t oscar_internal_kv8_extend_errors(uint32_t* flags, int reset) {
  return oscar::read_unit_errors(flags, reset) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}
