// Decode attention of sequences that share prefixes (oscar_kv8_decode_shared), over the 8-bit paged cache.
//
// Three kernels.  The first takes every group's prefix once, for all its members: their queries are the rows of tiles on tcgen05,
// as in the extend, and the prefix is cut into splits so that the tiles of all groups fill whole waves.  The lists are on the
// device, so the cut is made there, by every block for itself.  The second is the decode's split kernel over what each member
// has of its own; it begins while the first ends.  The third joins a row's partials of both.
//
// Against reading every member's whole sequence this trades the prefix's bytes, once instead of once a member, for products
// at the tensor cores' rate.
#include "kv8_decode_body.cuh"
#include "kv8_extend_body.cuh"

namespace {

template <int F, int D, int MT, int PARTS>
__global__ void __launch_bounds__(kThreads, 1) kv8_prefix_kernel(const __grid_constant__ SharedArgs args) {
  extend_body<F, D, MT, PARTS, true>(args);
}

template <int F, int D>
__global__ void __launch_bounds__(kWarps * 32, 3) kv8_own_kernel(const __grid_constant__ CUtensorMap map,
                                                                 const __grid_constant__ OwnArgs args) {
  split_body<F, D, true>(map, args);
  // Nothing here waits for the prefix kernel beside it (whose blocks have all waited for what comes before both), but the merge
  // waits for this kernel alone: its last block ends after the prefix kernel.
  if (args.beside_prefix && blockIdx.x + 1 == gridDim.x && blockIdx.y + 1 == gridDim.y && blockIdx.z + 1 == gridDim.z)
    grid_dep_wait();
}

struct MergeArgs {
  AttnArgs a;
  const int32_t* members;
  const int4* info;
  const int* own;
  const float* own_o;  // [num_members][Hq][ns][D], and [4]
  const float* own_ml;
  const float* pre_o;  // [items][H][tm][D], and [4]
  const float* pre_ml;
  int num_members, ns, tm;
};

// One warp per (member, query head).
constexpr int kMergeRows = 4;
template <int D>
__global__ void __launch_bounds__(kMergeRows * 32) kv8_shared_merge_kernel(MergeArgs m) {
  const AttnArgs& a = m.a;
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kMergeRows + (threadIdx.x >> 5);
  grid_dep_wait();
  if (row >= static_cast<long long>(m.num_members) * a.Hq) return;
  const int i = static_cast<int>(row / a.Hq), hq = static_cast<int>(row % a.Hq);
  const int4 info = m.info[i];
  if (info.x < 0) return;  // not a member
  const int b = __ldg(m.members + i);
  if (b < 0 || b >= a.batch) return;
  const int n_own = m.own[i], n = n_own + info.z;
  if (info.z == 0 && n_own <= 1) return;  // written by the kernel before
  const int gqa = a.Hq / a.H, h = hq / gqa, x = info.w * gqa + hq % gqa;
  const float* own_o = m.own_o + row * m.ns * D;
  const float* own_ml = m.own_ml + row * m.ns * 4;
  const size_t at = (static_cast<size_t>(info.x + x / m.tm) * a.H + h) * m.tm + x % m.tm;
  const size_t step = static_cast<size_t>(info.y) * a.H * m.tm;  // from one split to the next
  float l, e;
  float4 r;
  merge_parts<D>([&](int k) { return k < n_own ? own_o + static_cast<size_t>(k) * D : m.pre_o + (at + (k - n_own) * step) * D; },
                 [&](int k) { return k < n_own ? own_ml + 4 * k : m.pre_ml + (at + (k - n_own) * step) * 4; }, n, 0, 1, lane,
                 l, r, e);
  if (lane < D / 4) store_out4(a.out + (static_cast<size_t>(b) * a.Hq + hq) * D + 4 * lane, r, l, e);
}

struct Plan {
  int mt, parts, tm, items;  // of the prefix kernel; items 0: no prefix
  int ns, pps;               // of what is the members' own
  size_t off_ml, off_pre_o, off_pre_ml, off_info, off_own, total;
};

bool make_plan(const oscar_dims_t* d, int batch, int max_seq_len, int max_prefix, int max_own, int members, int groups, Plan* p) {
  if (check_dims(d) != OSCAR_OK || batch < 0 || members < 0 || members > 65535 || groups < 0 || groups > 65535 ||
      max_seq_len < 0 || max_prefix < 0 || max_own < 0 || max_prefix > max_seq_len || max_own > max_seq_len)
    return false;
  if (max_seq_len > kMaxLen || max_seq_len > static_cast<long long>(d->max_pages_per_seq) * kPageSize) return false;
  if (d->num_kv_heads > 65535) return false;
  const int H = d->num_kv_heads, gqa = d->num_q_heads / H;
  // the prefixes: tiles of 256 rows, smaller ones where a group has fewer rows
  const long long rows = static_cast<long long>(members) * gqa, each = groups > 0 ? (rows + groups - 1) / groups : 0;
  p->mt = each > 128 ? 2 : 1;
  p->parts = each > 64 ? 1 : 2;
  p->tm = p->mt * 128 / p->parts;
  const long long most_tiles = rows / p->tm + groups;  // of one KV head: ragged ones, one a group, beyond the even ones
  const long long blocks = (max_prefix / kPageSize + kBlkPages - 1) / kBlkPages;
  p->items = 0;
  if (blocks > 0 && rows > 0 && groups > 0) {
    // Blocks of the grid, for each KV head: those of the waves that take least for as many tiles as are likely (the kernel
    // looks again, with the tiles that there are), and at least one for each tile.
    const long long tiles = rows / p->tm > groups ? rows / p->tm : groups;
    long long best = 0, items = 0;
    for (long long w = 1; w <= 4; ++w) {
      const long long n = w * num_sms() / H;
      if (n < tiles) continue;
      const long long splits = n / tiles, cost = w * ((blocks + splits - 1) / splits + 5);
      if (best == 0 || cost < best) {
        best = cost;
        items = n;
      }
    }
    if (items < most_tiles) items = most_tiles;
    if (items > 0x7fffffffLL) return false;
    p->items = static_cast<int>(items);
  }
  // the rest, as in the decode
  const long long pages = (static_cast<long long>(max_own) + kPageSize - 1) / kPageSize;
  p->pps = split_pages(pages, (members > 0 ? members : 1LL) * H);
  if (p->pps > kMaxPps) p->pps = kMaxPps;
  const long long ns = pages > 0 ? (pages + p->pps - 1) / p->pps : 1;
  if (ns > 65535) return false;
  p->ns = static_cast<int>(ns);
  const size_t own = ns > 1 || p->items > 0 ? static_cast<size_t>(members) * d->num_q_heads * ns : 0;
  const size_t pre = static_cast<size_t>(p->items) * H * p->tm;
  p->off_ml = align_up(own * d->head_dim * sizeof(float), 256);
  p->off_pre_o = p->off_ml + align_up(own * 4 * sizeof(float), 256);
  p->off_pre_ml = p->off_pre_o + align_up(pre * d->head_dim * sizeof(float), 256);
  p->off_info = p->off_pre_ml + align_up(pre * 4 * sizeof(float), 256);
  p->off_own = p->off_info + align_up(static_cast<size_t>(members) * sizeof(int4), 256);
  p->total = p->off_own + align_up(static_cast<size_t>(members) * sizeof(int), 256) + 256;
  return true;
}

template <int F, int D, int MT, int PARTS>
cudaError_t launch_prefix(const Plan& p, const SharedArgs& sh, cudaStream_t stream) {
  auto k = kv8_prefix_kernel<F, D, MT, PARTS>;
  static const bool regs = has_launch_registers(reinterpret_cast<const void*>(k));
  if (!regs) return cudaErrorInvalidConfiguration;
  const cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(k), Geo<D, MT>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(p.items, sh.e.a.H), dim3(kThreads), Geo<D, MT>::kSmem, stream, sh);
}

template <int F, int D>
cudaError_t launch(const Plan& p, const SharedArgs& sh, const OwnArgs& ow, const MergeArgs& me, const CUtensorMap& map,
                   cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (p.items > 0)
    e = p.mt == 2      ? launch_prefix<F, D, 2, 1>(p, sh, stream)
        : p.parts == 2 ? launch_prefix<F, D, 1, 2>(p, sh, stream)
                       : launch_prefix<F, D, 1, 1>(p, sh, stream);
  if (e != cudaSuccess) return e;
  auto k = kv8_own_kernel<F, D>;
  e = set_smem_limit_once(reinterpret_cast<const void*>(k), DecodeGeo<D>::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k, dim3(p.ns, ow.s.a.H, me.num_members), dim3(kWarps * 32), DecodeGeo<D>::kSmem, stream, map, ow);
  if (e != cudaSuccess || (p.items == 0 && p.ns == 1)) return e;
  const long long rows = static_cast<long long>(me.num_members) * me.a.Hq;
  return launch_pdl(kv8_shared_merge_kernel<D>, dim3(static_cast<unsigned>((rows + kMergeRows - 1) / kMergeRows)),
                    dim3(kMergeRows * 32), 0, stream, me);
}

}  // namespace

extern "C" size_t oscar_kv8_decode_shared_workspace_bytes(const oscar_dims_t* dims, int32_t batch, int32_t max_seq_len,
                                                          int32_t max_prefix_len, int32_t max_own_len, int32_t num_members,
                                                          int32_t num_groups) {
  Plan p;
  return make_plan(dims, batch, max_seq_len, max_prefix_len, max_own_len, num_members, num_groups, &p) ? p.total : 0;
}

extern "C" oscar_status_t oscar_kv8_decode_shared(const oscar_dims_t* dims, int32_t kv_format, int32_t batch,
                                                  int32_t max_seq_len, int32_t max_prefix_len, int32_t max_own_len,
                                                  int32_t num_members, int32_t num_groups, const void* q,
                                                  const uint8_t* kv8_pages, const float* kv8_scales,
                                                  const int32_t* page_table, const int32_t* seq_lens,
                                                  const int32_t* members, const int32_t* group_start,
                                                  const int32_t* prefix_lens, float sm_scale, void* out, void* workspace,
                                                  size_t workspace_bytes, void* stream) {
  oscar_status_t st = check_dims(dims);
  if (st != OSCAR_OK) return st;
  if (bad_format(kv_format) || batch < 0 || num_members < 0 || num_groups < 0 || max_seq_len < 0 || max_prefix_len < 0 ||
      max_own_len < 0)
    return OSCAR_ERR_INVALID_ARG;
  Plan plan;
  if (!make_plan(dims, batch, max_seq_len, max_prefix_len, max_own_len, num_members, num_groups, &plan))
    return OSCAR_ERR_INVALID_ARG;
  if (num_members == 0 || num_groups == 0) return OSCAR_OK;
  if (batch == 0 || !members || !group_start || !prefix_lens) return OSCAR_ERR_INVALID_ARG;
  AttnArgs a;
  st = make_args(dims, batch, num_members, 1, max_seq_len, q, nullptr, kv8_pages, kv8_scales, page_table, seq_lens, 0, 0,
                 sm_scale, out, workspace, plan.total, workspace_bytes, &a);
  if (st != OSCAR_OK) return st;
  CUtensorMap map;
  if (!encode_page_map(dims, kv8_pages, &map)) return OSCAR_ERR_CUDA;
  char* w = static_cast<char*>(workspace);
  auto floats = [&](size_t off) { return reinterpret_cast<float*>(w + off); };
  const Groups g{members, group_start, prefix_lens, num_members, num_groups, max_prefix_len};
  int4* info = reinterpret_cast<int4*>(w + plan.off_info);
  int* own = reinterpret_cast<int*>(w + plan.off_own);
  const SharedArgs sh{{a, floats(plan.off_pre_o), floats(plan.off_pre_ml), 0, 0, 0}, g, info, num_sms()};
  const OwnArgs ow{{a, floats(0), floats(plan.off_ml), plan.ns, plan.pps}, g, info, own, max_own_len, plan.items > 0};
  const MergeArgs me{a, members, info, own, floats(0), floats(plan.off_ml), floats(plan.off_pre_o), floats(plan.off_pre_ml),
                     num_members, plan.ns, plan.tm};
  cudaStream_t s = as_stream(stream);
  const bool d128 = dims->head_dim == 128;
  const cudaError_t e = kv_format == OSCAR_KV8_E4M3
                            ? (d128 ? launch<kE4M3, 128>(plan, sh, ow, me, map, s) : launch<kE4M3, 64>(plan, sh, ow, me, map, s))
                            : (d128 ? launch<kInt8, 128>(plan, sh, ow, me, map, s) : launch<kInt8, 64>(plan, sh, ow, me, map, s));
  return e == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

oscar_status_t oscar_internal_kv8_shared_errors(uint32_t* flags, int reset) {
  return oscar::read_unit_errors(flags, reset) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}
