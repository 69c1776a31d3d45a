// Decode attention over the 8-bit paged cache (oscar_kv8_decode): one query row per sequence,
// full or with a sliding window and sinks.
// The split kernel is described where its body is; a second kernel merges the splits where there are several.
#include "kv8_decode_body.cuh"

namespace {

template <int F, int D>
__global__ void __launch_bounds__(kWarps * 32, 3) kv8_split_kernel(const __grid_constant__ CUtensorMap map,
                                                                   const __grid_constant__ SplitArgs sa) {
  split_body<F, D, false>(map, sa);
}

// One CTA per (sequence, query head): the log-sum-exp merge of its splits, dealt out to four warps.
constexpr int kMergeWarps = 4;
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) kv8_merge_kernel(SplitArgs sa) {
  __shared__ float4 part[kMergeWarps][D / 4];
  __shared__ float sums[kMergeWarps];
  const AttnArgs& a = sa.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t row = blockIdx.x;
  const int b = static_cast<int>(row / a.Hq);
  // (the lengths come from before the split kernel, which waited for whoever wrote them)
  const int L = min(max(__ldg(a.seq_lens + b), 0), a.max_seq_len);
  const Visible vis = visible(L - 1, L - 1, a.sink, a.window);
  const int n = (vis.n + sa.pps - 1) / sa.pps;
  grid_dep_wait();
  if (n <= 1) return;  // the split kernel wrote the output
  const float* o = sa.part_o + row * sa.ns * D;
  const float* ml = sa.part_ml + row * sa.ns * 4;
  float l, e;
  float4 r;
  merge_part<D>(o, ml, n, warp, kMergeWarps, lane, l, r, e);
  if (lane < D / 4) part[warp][lane] = r;
  if (lane == 0) sums[warp] = l;
  __syncthreads();
  if (threadIdx.x < D / 4) {
    for (int w = 1; w < kMergeWarps; ++w) {
      const float4 x = part[w][threadIdx.x];
      l += sums[w];
      r.x += x.x; r.y += x.y; r.z += x.z; r.w += x.w;
    }
    store_out4(a.out + row * D + 4 * threadIdx.x, r, l, e);
  }
}

struct Plan {
  int ns, pps;
  size_t off_ml, total;
};

bool make_plan(const oscar_dims_t* d, int batch, int max_seq_len, int pps, int sink, int window, Plan* p) {
  if (check_dims(d) != OSCAR_OK || batch < 0 || batch > 65535 || max_seq_len < 0 || pps < 0 || sink < 0 || window < 0)
    return false;
  if (max_seq_len > kMaxLen || max_seq_len > static_cast<long long>(d->max_pages_per_seq) * kPageSize) return false;
  if (d->num_kv_heads > 65535 || static_cast<long long>(batch) * d->num_q_heads > 0x7fffffffLL) return false;
  const long long pages = max_visible_pages(max_seq_len, sink, window, 1);
  if (pps == 0) pps = split_pages(pages, static_cast<long long>(batch > 0 ? batch : 1) * d->num_kv_heads);
  if (pps > kMaxPps) pps = kMaxPps;
  const long long ns = pages > 0 ? (pages + pps - 1) / pps : 1;
  if (ns > 65535) return false;
  p->ns = static_cast<int>(ns);
  p->pps = pps;
  const size_t parts = ns > 1 ? static_cast<size_t>(batch) * d->num_q_heads * ns : 0;
  p->off_ml = align_up(parts * d->head_dim * sizeof(float), 256);
  p->total = p->off_ml + align_up(parts * 4 * sizeof(float), 256) + 256;
  return true;
}

template <int F, int D>
cudaError_t launch(const SplitArgs& sa, const CUtensorMap& map, cudaStream_t stream) {
  auto k = kv8_split_kernel<F, D>;
  cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(k), DecodeGeo<D>::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k, dim3(sa.ns, sa.a.H, sa.a.batch), dim3(kWarps * 32), DecodeGeo<D>::kSmem, stream, map, sa);
  if (e != cudaSuccess || sa.ns == 1) return e;
  return launch_pdl(kv8_merge_kernel<D>, dim3(static_cast<unsigned>(sa.a.batch) * sa.a.Hq), dim3(kMergeWarps * 32), 0,
                    stream, sa);
}

}  // namespace

extern "C" size_t oscar_kv8_decode_workspace_bytes(const oscar_dims_t* dims, int32_t batch, int32_t max_seq_len,
                                                   int32_t pages_per_split, int32_t sink_len, int32_t window_len) {
  Plan p;
  return make_plan(dims, batch, max_seq_len, pages_per_split, sink_len, window_len, &p) ? p.total : 0;
}

extern "C" oscar_status_t oscar_kv8_decode(const oscar_dims_t* dims, int32_t kv_format, int32_t batch,
                                           int32_t max_seq_len, int32_t pages_per_split, const void* q,
                                           const uint8_t* kv8_pages, const float* kv8_scales,
                                           const int32_t* page_table, const int32_t* seq_lens, int32_t sink_len,
                                           int32_t window_len, float sm_scale, void* out, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  oscar_status_t st = check_dims(dims);
  if (st != OSCAR_OK) return st;
  if (bad_format(kv_format) || batch < 0 || max_seq_len < 0 || pages_per_split < 0 || sink_len < 0 || window_len < 0)
    return OSCAR_ERR_INVALID_ARG;
  if (batch == 0) return OSCAR_OK;
  Plan plan;
  if (!make_plan(dims, batch, max_seq_len, pages_per_split, sink_len, window_len, &plan)) return OSCAR_ERR_INVALID_ARG;
  SplitArgs sa;
  st = make_args(dims, batch, batch, 1, max_seq_len, q, nullptr, kv8_pages, kv8_scales, page_table, seq_lens, sink_len,
                 window_len, sm_scale, out, workspace, plan.total, workspace_bytes, &sa.a);
  if (st != OSCAR_OK) return st;
  CUtensorMap map;
  if (!encode_page_map(dims, kv8_pages, &map)) return OSCAR_ERR_CUDA;
  char* w = static_cast<char*>(workspace);
  sa.part_o = reinterpret_cast<float*>(w);
  sa.part_ml = reinterpret_cast<float*>(w + plan.off_ml);
  sa.ns = plan.ns;
  sa.pps = plan.pps;
  cudaStream_t s = as_stream(stream);
  const bool d128 = dims->head_dim == 128;
  const cudaError_t e = kv_format == OSCAR_KV8_E4M3
                            ? (d128 ? launch<kE4M3, 128>(sa, map, s) : launch<kE4M3, 64>(sa, map, s))
                            : (d128 ? launch<kInt8, 128>(sa, map, s) : launch<kInt8, 64>(sa, map, s));
  return e == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

oscar_status_t oscar_internal_kv8_decode_errors(uint32_t* flags, int reset) {
  return oscar::read_unit_errors(flags, reset) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}
