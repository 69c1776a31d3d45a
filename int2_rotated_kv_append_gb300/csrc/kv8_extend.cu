// Extend attention over the 8-bit paged cache (oscar_kv8_extend_varlen): the last rows of each sequence,
// causal, full or with a sliding window and sinks, on tcgen05.  The kernel is described where its body is.
#include "kv8_extend_body.cuh"

namespace {

template <int F, int D, int MT, int PARTS>
__global__ void __launch_bounds__(kThreads, 1) kv8_extend_kernel(const __grid_constant__ ExtArgs ea) {
  extend_body<F, D, MT, PARTS, false>(ea);
}

// The merge of the splits, one warp per output row: kMergeRows rows of a tile per CTA.
constexpr int kMergeRows = 4;
template <int D, int TM>
__global__ void __launch_bounds__(kMergeRows * 32) kv8_extend_merge_kernel(ExtArgs ea) {
  const AttnArgs& a = ea.a;
  constexpr int kParts = TM / kMergeRows;
  // (what it reads comes from before the attention kernel, which waited for whoever wrote it)
  const Tile T = tile_of<TM>(a, blockIdx.z, blockIdx.x / kParts);
  grid_dep_wait();
  if (!T.ok) return;
  const int n = (T.blocks + ea.bps - 1) / ea.bps;
  const int r = blockIdx.x % kParts * kMergeRows + (threadIdx.x >> 5);
  if (n <= 1 || r >= T.rows) return;  // (one split: written by the attention kernel)
  const int gqa = a.Hq / a.H, x = T.r0 + r;
  const size_t row = static_cast<size_t>(T.q0 + x / gqa) * a.Hq + blockIdx.y * gqa + x % gqa;
  merge_row<D>(ea.part_o + row * ea.ns * D, ea.part_ml + row * ea.ns * 4, n, a.out + row * D, threadIdx.x & 31);
}

struct Plan {
  int mt, parts, tiles, ns, bps;
  size_t off_ml, total;
};

bool make_plan(const oscar_dims_t* d, int batch, int rows, int max_seq_len, int max_rows, int pps, int sink, int window,
               Plan* p) {
  if (check_dims(d) != OSCAR_OK || batch < 0 || batch > 65535 || rows < 0 || max_rows < 0 || max_seq_len < 0 ||
      pps < 0 || sink < 0 || window < 0)
    return false;
  if (max_seq_len > kMaxLen || max_seq_len > static_cast<long long>(d->max_pages_per_seq) * kPageSize ||
      d->num_kv_heads > 65535)
    return false;
  const int gqa = d->num_q_heads / d->num_kv_heads;
  if (max_rows > rows) max_rows = rows;
  const long long per_seq = static_cast<long long>(max_rows) * gqa;
  p->mt = per_seq > 128 ? 2 : 1;
  p->parts = per_seq > 64 ? 1 : 2;  // (drafts of 8 rows, GQA 8: 97 us with 1, 87 with 2)
  const int tm = 128 * p->mt;
  const long long tiles = (per_seq + tm - 1) / tm;
  const long long pages = max_visible_pages(max_seq_len, sink, window, tm / gqa + 1);
  const long long blocks = (pages + kBlkPages - 1) / kBlkPages;
  long long bps;
  if (pps > 0) {
    bps = (pps + kBlkPages - 1) / kBlkPages;
  } else {
    // tiles that have rows: at most one ragged tile per sequence beyond the even ones
    long long units = static_cast<long long>(rows) * gqa / tm + batch;
    if (units > tiles * batch) units = tiles * batch;
    units *= d->num_kv_heads;
    long long splits = 1;
    // The cheapest of the split counts that fill whole waves of one CTA per SM, a wave taking its blocks and as long as 5
    // (short runs) or 12 more for its start and end; the 12 also stand for the merge and for causal tiles that end
    // early (with 8, 4096 rows of 8192 positions take 481 us in two splits, 357 in one).  Against a fixed 3 (2) CTAs per SM:
    // 8 rows of one sequence of 32768 tokens 51 -> 31 us, of two 64 -> 45, of eight of 16384 92 -> 81, 512 rows of 8192
    // positions 93 -> 81.
    const long long extra = p->mt == 1 ? 5 : 12;
    long long best = 0;
    for (long long w = 1; w <= 8; ++w) {
      const long long n = w * num_sms() / (units > 0 ? units : 1);
      if (n < 1) continue;
      const long long cost = w * ((blocks + n - 1) / n + extra);
      if (best == 0 || cost < best) {
        best = cost;
        splits = n;
      }
    }
    bps = (blocks + splits - 1) / splits;
    if (bps < 4) bps = 4;
  }
  if (bps < 1) bps = 1;
  const long long ns = blocks > 0 ? (blocks + bps - 1) / bps : 1;
  if (ns > 65535 || tiles * ns > 0x7fffffffLL || tiles * 64 > 0x7fffffffLL || bps > 0x7fffffffLL / kBlkPages) return false;
  p->tiles = static_cast<int>(tiles > 0 ? tiles : 1);
  p->ns = static_cast<int>(ns);
  p->bps = static_cast<int>(bps);
  const size_t parts = ns > 1 ? static_cast<size_t>(rows) * d->num_q_heads * ns : 0;
  p->off_ml = align_up(parts * d->head_dim * sizeof(float), 256);
  p->total = p->off_ml + align_up(parts * 4 * sizeof(float), 256) + 256;
  return true;
}

template <int F, int D, int MT, int PARTS>
cudaError_t launch(const ExtArgs& ea, cudaStream_t stream) {
  auto k = kv8_extend_kernel<F, D, MT, PARTS>;
  static const bool regs = has_launch_registers(reinterpret_cast<const void*>(k));
  if (!regs) return cudaErrorInvalidConfiguration;
  cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(k), Geo<D, MT>::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k, dim3(static_cast<unsigned>(ea.tiles * ea.ns), ea.a.H, ea.a.batch), dim3(kThreads),
                 Geo<D, MT>::kSmem, stream, ea);
  if (e != cudaSuccess || ea.ns == 1) return e;
  return launch_pdl(kv8_extend_merge_kernel<D, MT * 128>, dim3(ea.tiles * (MT * 128 / kMergeRows), ea.a.H, ea.a.batch),
                    dim3(kMergeRows * 32), 0, stream, ea);
}

template <int F, int D>
cudaError_t launch_mt(const Plan& p, const ExtArgs& ea, cudaStream_t stream) {
  if (p.mt == 2) return launch<F, D, 2, 1>(ea, stream);
  return p.parts == 2 ? launch<F, D, 1, 2>(ea, stream) : launch<F, D, 1, 1>(ea, stream);
}

}  // namespace

extern "C" size_t oscar_kv8_extend_varlen_workspace_bytes(const oscar_dims_t* dims, int32_t batch, int32_t num_rows,
                                                          int32_t max_seq_len, int32_t max_rows_per_seq,
                                                          int32_t pages_per_split, int32_t sink_len,
                                                          int32_t window_len) {
  Plan p;
  return make_plan(dims, batch, num_rows, max_seq_len, max_rows_per_seq, pages_per_split, sink_len, window_len, &p)
             ? p.total
             : 0;
}

extern "C" oscar_status_t oscar_kv8_extend_varlen(const oscar_dims_t* dims, int32_t kv_format, int32_t batch,
                                                  int32_t num_rows, int32_t max_seq_len, int32_t max_rows_per_seq,
                                                  int32_t pages_per_split, const void* q, const int32_t* q_start,
                                                  const uint8_t* kv8_pages, const float* kv8_scales,
                                                  const int32_t* page_table, const int32_t* seq_lens,
                                                  int32_t sink_len, int32_t window_len, float sm_scale, void* out,
                                                  void* workspace, size_t workspace_bytes, void* stream) {
  oscar_status_t st = check_dims(dims);
  if (st != OSCAR_OK) return st;
  if (bad_format(kv_format) || batch < 0 || num_rows < 0 || max_seq_len < 0 || max_rows_per_seq < 0 ||
      pages_per_split < 0 || sink_len < 0 || window_len < 0)
    return OSCAR_ERR_INVALID_ARG;
  if (num_rows == 0) return OSCAR_OK;
  if (batch == 0 || max_rows_per_seq == 0 || !q_start) return OSCAR_ERR_INVALID_ARG;
  Plan plan;
  if (!make_plan(dims, batch, num_rows, max_seq_len, max_rows_per_seq, pages_per_split, sink_len, window_len, &plan))
    return OSCAR_ERR_INVALID_ARG;
  if (static_cast<long long>(max_rows_per_seq) * (dims->num_q_heads / dims->num_kv_heads) > 0x7fffffffLL ||
      static_cast<long long>(num_rows) * (dims->num_q_heads / dims->num_kv_heads) > 0x7fffffffLL - 256)
    return OSCAR_ERR_UNSUPPORTED;
  ExtArgs ea;
  st = make_args(dims, batch, num_rows, max_rows_per_seq < num_rows ? max_rows_per_seq : num_rows, max_seq_len, q,
                 q_start, kv8_pages, kv8_scales, page_table, seq_lens, sink_len, window_len, sm_scale, out, workspace,
                 plan.total, workspace_bytes, &ea.a);
  if (st != OSCAR_OK) return st;
  char* w = static_cast<char*>(workspace);
  ea.part_o = reinterpret_cast<float*>(w);
  ea.part_ml = reinterpret_cast<float*>(w + plan.off_ml);
  ea.ns = plan.ns;
  ea.bps = plan.bps;
  ea.tiles = plan.tiles;
  cudaStream_t s = as_stream(stream);
  const bool d128 = dims->head_dim == 128;
  const cudaError_t e = kv_format == OSCAR_KV8_E4M3
                            ? (d128 ? launch_mt<kE4M3, 128>(plan, ea, s) : launch_mt<kE4M3, 64>(plan, ea, s))
                            : (d128 ? launch_mt<kInt8, 128>(plan, ea, s) : launch_mt<kInt8, 64>(plan, ea, s));
  return e == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

oscar_status_t oscar_internal_kv8_extend_errors(uint32_t* flags, int reset) {
  return oscar::read_unit_errors(flags, reset) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}
