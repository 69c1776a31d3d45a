// Decode attention of sequences that share prefixes (oscar_kv8_decode_shared), over the 8-bit paged cache.
//
// Where that would take longer than each member by itself, as in small calls, or has more tiles than four waves of blocks, it is the
// decode's split kernel over the list, and a merge.  Else three kernels, of which the first two run beside one another.  One takes every group's prefix once, for all its members: their
// queries are the rows of tiles on tcgen05, as in the extend, and the prefix is cut into splits so that the tiles of all groups
// fill whole waves.  The lists are on the device, so the cut is made there, by every block for itself.  The other attends what
// each member has of its own, as the decode does.  The former is bound by products and the latter by memory, and either fills an
// SM, so the SMs are divided among them.  The third joins a row's partials of both.
//
// Against reading every member's whole sequence this trades the prefix's bytes, once instead of once a member, for products
// at the tensor cores' rate.  Measured (GB300; 8 KV heads, D = 128): 64 members of one prefix of 16384 tokens with up to 1024 of
// their own, 32 query heads, 101 MB and 18 GFLOP: 48 us (each by itself 325): 88 prefix CTAs of 40 us (10 before their first
// logits, 12 blocks of 2, 4 for 128 KB of partials), 60 SMs for 35 us with the 67 MB of the members' own, 7 for the merge.  128 of each
// of two prefixes of 31 thousand, 64 query heads, 261 GFLOP: 259 us, 1010 TFLOP/s (2360 each by itself): 128 CTAs of 122 blocks
// at 1.5 GHz (the power limit), tensor pipes 44% busy, as in the extend.
#include "kv8_decode_body.cuh"
#include "kv8_extend_body.cuh"

namespace {

template <int F, int D, int MT, int PARTS>
__global__ void __launch_bounds__(kThreads, 1) kv8_prefix_kernel(const __grid_constant__ SharedArgs args) {
  extend_body<F, D, MT, PARTS, true>(args);
  // The kernel after the two that run beside one another waits for the second of them alone: its last block ends after the first.
  // (The blocks of the first have all waited for what comes before both, so the second waits for nothing.)
  if (args.last && blockIdx.x + 1 == gridDim.x && blockIdx.y + 1 == gridDim.y) grid_dep_wait();
}

// What the members have of their own, behind their groups' prefixes.  The (member, KV head) units' pages lie one after another, in
// the order of the list and kUnitCost empty places behind each unit's, and every warp of the grid takes the same number of places,
// wherever units begin and end: uneven lengths balance, and a block finds out once what is where.  A unit's share of a warp is a piece; piece (unit u, warp w) is stored at
// u + w (no two are at one place, as along the pages one of the two always grows).  Lists of more than kChunk members are cut into
// chunks with a row of blocks each.
//
// A page (16 tokens, K then V, D bytes each) is one tensor copy into a stage of the warp's ring, swizzled so that every
// shared-memory read is free of bank conflicts.  Per page, with the GQA group's queries as the 8 columns:
//   S^T = K Q^T     ldmatrix rows of 16 codes -> fp16 pairs (exact) as A: all 16 tokens in one product;
//   P^T             weights 2^(s - m) times 2^kOwnBoost as fp16, m the running maximum less kOwnLazy at most, so that it seldom
//                   moves: 11 bits, a step of 2^-30 of the largest; two 8 x 8 transposes make it B;
//   O^T += f V^T P^T  f = the page's V scale, in fp32 (with a scale over 2^80, infinite V elements saturated, O counts 2^40).
// That is half the products and half the instructions of the decode's form, whose tokens are the columns and whose weights have 22
// bits: of a page an SM takes 155 clocks, where that takes 235.
constexpr int kChunk = 384;
constexpr int kOwnWarps = 12;  // as many as an SM holds
constexpr int kOwnThreads = kOwnWarps * 32;
static_assert(kChunk == kOwnThreads, "a member a thread");
constexpr int kLeastPages = 4;  // of a warp
constexpr int kUnitCost = 2;    // pages in whose time a warp goes from one unit to the next: as many places without a page
constexpr float kOwnLazy = 8.f;  // log2
constexpr int kOwnBoost = 6;     // 2^(kOwnLazy + kOwnBoost) < 65504
constexpr float kOwnBigScale = 0x1p80f;  // up to here 2^80 times a code (2^9) times 2^kOwnLazy times 2^27 tokens is within fp32

// Pages of a warp's ring, 16 KB.
template <int D>
struct Ring {
  static constexpr int kPage = 2 * kPageSize * D;  // bytes of one page and head
  static constexpr int kStages = 16384 / kPage;
  static constexpr size_t kBytes = static_cast<size_t>(kStages) * kPage;
};

struct OwnArgs {
  AttnArgs a;
  Groups g;
  int4* info;     // [num_members]: as the prefix kernel leaves it for members with a prefix; x < 0: not a member
  int2* own;      // [num_members][H]: first piece of the unit, pieces
  float* part_o;  // [chunks x warps + num_members x KV heads][GQA][D], and [4]
  float* part_ml;
  int max_own;    // tokens
  bool first, last;  // of the two kernels that run beside one another
};

template <int D>
struct OwnGeo {
  static constexpr size_t kSmem = 1024 + kOwnWarps * (Ring<D>::kBytes + Ring<D>::kStages * 8);
};

// What a lane (g, t) = (lane / 4, lane % 4) has of a unit: queries 2t and 2t + 1 (x, y), channels D / 8 g + c.
template <int D>
struct Sums {
  float2 o[D / 8];
  float2 m, l;  // l: of the lane's tokens
};

// The page in stage `st`, its first position pos0, of a sequence of length L; scales sc (K, V), qs: what a query's logits are to be
// multiplied with.
template <int F, int D>
__device__ __forceinline__ void attend_own(uint32_t st, int pos0, int L, float2 sc, float2 qs, const uint32_t (&qa)[D / 16][2],
                                           int lane, Sums<D>& u) {
  constexpr int kKs = D / 16, kNt = D / 8;
  const int g = lane >> 2, t = lane & 3;
  float acc[2][4];  // two chains of products
#pragma unroll
  for (int c4 = 0; c4 < kKs; c4 += 4) {
    uint32_t w0[4], w1[4];  // tokens g and g + 8
    ldmatrix_x4(st + chunk_at<D>(lane & 7, c4 + (lane >> 3)), w0);
    ldmatrix_x4(st + chunk_at<D>(8 + (lane & 7), c4 + (lane >> 3)), w1);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t a0, a1, a2, a3;
      codes_to_f16<F>(w0[c], a0, a2);
      codes_to_f16<F>(w1[c], a1, a3);
      if (c4 + c < 2) mma_f16_first(acc[c & 1], a0, a1, a2, a3, qa[c4 + c][0], qa[c4 + c][1]);
      else mma_f16(acc[c & 1], a0, a1, a2, a3, qa[c4 + c][0], qa[c4 + c][1]);
    }
  }
  // (the scales first: a logit may be within fp32 where its product with one of them is not; towards 0: never infinite, so that
  // logits of 0 stay 0)
  const float2 ks = make_float2(__fmul_rz(sc.x, qs.x), __fmul_rz(sc.x, qs.y));
  float2 s0 = make_float2((acc[0][0] + acc[1][0]) * ks.x, (acc[0][1] + acc[1][1]) * ks.y);  // token g
  float2 s1 = make_float2((acc[0][2] + acc[1][2]) * ks.x, (acc[0][3] + acc[1][3]) * ks.y);  // token g + 8
  const bool tail = pos0 + kPageSize > L;
  if (tail) {
    if (pos0 + g >= L) s0 = make_float2(-INFINITY, -INFINITY);
    if (pos0 + g + 8 >= L) s1 = make_float2(-INFINITY, -INFINITY);
  }
  float2 mx = make_float2(fmaxf(s0.x, s1.x), fmaxf(s0.y, s1.y));
  // (-infinity + kOwnLazy is that: the first logits move it)
  if (__any_sync(0xffffffffu, mx.x > u.m.x + kOwnLazy || mx.y > u.m.y + kOwnLazy)) {
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      mx.x = fmaxf(mx.x, __shfl_xor_sync(0xffffffffu, mx.x, x));
      mx.y = fmaxf(mx.y, __shfl_xor_sync(0xffffffffu, mx.y, x));
    }
    const float2 m = make_float2(fmaxf(u.m.x, mx.x), fmaxf(u.m.y, mx.y));
    const float2 alpha = make_float2(u.m.x == -INFINITY ? 0.f : fast_exp2(u.m.x - m.x), u.m.y == -INFINITY ? 0.f : fast_exp2(u.m.y - m.y));
    u.l = f2mul(u.l, alpha);
#pragma unroll
    for (int c = 0; c < kNt; ++c) u.o[c] = f2mul(u.o[c], alpha);
    u.m = m;
  }
  const float2 m = make_float2(u.m.x == -INFINITY ? 0.f : u.m.x, u.m.y == -INFINITY ? 0.f : u.m.y);
  const float2 p0 = make_float2(fast_exp2(s0.x - m.x), fast_exp2(s0.y - m.y));
  const float2 p1 = make_float2(fast_exp2(s1.x - m.x), fast_exp2(s1.y - m.y));
  u.l.x += p0.x + p1.x;
  u.l.y += p0.y + p1.y;
  const float boost = 1 << kOwnBoost;
  const uint32_t b0 = movmatrix_trans(pack_half2(p0.x * boost, p0.y * boost));
  const uint32_t b1 = movmatrix_trans(pack_half2(p1.x * boost, p1.y * boost));
  // V: tokens 2t, 2t+1, 2t+8, 2t+9, channels kNt g .. kNt g + kNt - 1
  uint32_t w[4][kNt / 4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int r = 2 * t + (c & 1) + 8 * (c >> 1);
    if constexpr (D == 128) {
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[c][0]), "=r"(w[c][1]), "=r"(w[c][2]), "=r"(w[c][3])
                   : "r"(st + chunk_at<D>(kPageSize + r, g))
                   : "memory");
    } else {
      asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];"
                   : "=r"(w[c][0]), "=r"(w[c][1])
                   : "r"(st + chunk_at<D>(kPageSize + r, g >> 1) + 8 * (g & 1))
                   : "memory");
    }
    if (tail && pos0 + r >= L) {  // behind the last token: any bits, NaN included
#pragma unroll
      for (int q = 0; q < kNt / 4; ++q) w[c][q] = 0u;
    }
  }
  const float f = sc.y * (1.f / (1 << kOwnBoost));
#pragma unroll
  for (int q = 0; q < kNt / 4; ++q) {
    uint32_t lo[4], hi[4];  // channels 4 q + e: token pairs (2t, 2t+1) and (2t+8, 2t+9)
    codes_to_f16<F>(__byte_perm(w[0][q], w[1][q], 0x5140), lo[0], lo[1]);
    codes_to_f16<F>(__byte_perm(w[0][q], w[1][q], 0x7362), lo[2], lo[3]);
    codes_to_f16<F>(__byte_perm(w[2][q], w[3][q], 0x5140), hi[0], hi[1]);
    codes_to_f16<F>(__byte_perm(w[2][q], w[3][q], 0x7362), hi[2], hi[3]);
#pragma unroll
    for (int e = 0; e < 4; e += 2) {  // rows g and g + 8 of a product: channels 4 q + e and + 1
      float d[4];
      mma_f16_first(d, lo[e], lo[e + 1], hi[e], hi[e + 1], b0, b1);
      u.o[4 * q + e] = f2fma(make_float2(d[0], d[1]), make_float2(f, f), u.o[4 * q + e]);
      u.o[4 * q + e + 1] = f2fma(make_float2(d[2], d[3]), make_float2(f, f), u.o[4 * q + e + 1]);
    }
  }
}

template <int F, int D>
__global__ void __launch_bounds__(kOwnThreads, 1) kv8_own_kernel(const __grid_constant__ CUtensorMap map,
                                                                 const __grid_constant__ OwnArgs args) {
  constexpr int kStages = Ring<D>::kStages, kPage = Ring<D>::kPage, kNt = D / 8;  // kNt: channels of a lane
  extern __shared__ uint8_t raw[];
  __shared__ long long begins[kChunk + 1];  // places of one head before member i
  __shared__ int from_s[kChunk], seq_s[kChunk], len_s[kChunk];  // member i: its group's prefix, sequence, length
  __shared__ long long sums[kOwnWarps];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const AttnArgs& a = args.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int gqa = a.Hq / a.H;
  const int m0 = blockIdx.y * kChunk, mc = min(kChunk, args.g.num_members - m0);
  const bool tells = blockIdx.x == 0;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOwnWarps * Ring<D>::kBytes) + warp * kStages;
  if (tid == 0) umma::prefetch_map(&map);
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(bars + i), 1);
    mbar_init_fence();
  }
  if (args.first) grid_dep_wait();
  grid_dep_launch_dependents();
  // ---- the lists ----------------------------------------------------------------------------
  const int b = tid < mc ? __ldg(args.g.members + m0 + tid) : -1;
  from_s[tid] = -1;
  __syncthreads();
  bool bad = false;
  for (int g0 = warp * 32; g0 < args.g.num_groups; g0 += kOwnThreads) {
    int start = 0, n = 0, prefix = 0;
    if (g0 + lane < args.g.num_groups && !group_of(args.g, g0 + lane, start, n, prefix)) bad = true;
    const int lo = max(start, m0), hi = bad ? lo : min(start + n, m0 + mc);
    for (uint32_t some = __ballot_sync(0xffffffffu, lo < hi); some != 0; some &= some - 1) {
      const int at = __ffs(some) - 1, end = __shfl_sync(0xffffffffu, hi, at), p = __shfl_sync(0xffffffffu, prefix, at);
      for (int i = __shfl_sync(0xffffffffu, lo, at) + lane; i < end; i += 32) from_s[i - m0] = p;
    }
  }
  bad = __syncthreads_or(bad);
  if (bad && tells && tid == 0) record_error(OSCAR_DEVERR_POSITION);
  const int from = from_s[tid];
  const bool in = !bad && from >= 0, good = b >= 0 && b < a.batch;
  int L = 0, pages = 0;
  if (in && good) {
    L = clamped_len(a, b);
    if (L - from > args.max_own) {
      record_error(OSCAR_DEVERR_SEQ_LEN);
      L = from + args.max_own;
    }
    pages = max((L + kPageSize - 1) / kPageSize - from / kPageSize, 0);
  } else if (tells && in) {
    record_error(OSCAR_DEVERR_POSITION);
  }
  seq_s[tid] = b;
  len_s[tid] = L;
  if (tells && tid < mc && (!in || from == 0)) args.info[m0 + tid] = make_int4(in && good ? 0 : -1, 0, 0, 0);
  if (in && good && from == 0 && L == 0 && tid % gridDim.x == blockIdx.x)  // nothing to attend
    for (int c = 0; c < a.Hq * (D / 8); ++c)
      reinterpret_cast<uint4*>(a.out + static_cast<size_t>(b) * a.Hq * D)[c] = make_uint4(0, 0, 0, 0);
  const int places = pages > 0 ? pages + kUnitCost : 0;
  long long up = places;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += x;
  }
  if (lane == 31) sums[warp] = up;
  __syncthreads();
  long long total = 0;
  up -= places;
#pragma unroll
  for (int w = 0; w < kOwnWarps; ++w) {
    if (w < warp) up += sums[w];
    total += sums[w];
  }
  const long long warps = static_cast<long long>(gridDim.x) * kOwnWarps, all = total * a.H;
  const long long each = max((all + warps - 1) / warps, static_cast<long long>(kLeastPages));
  begins[tid] = up;
  if (tid < mc && tid % gridDim.x == blockIdx.x)
    for (int h = 0; h < a.H; ++h) {
      const long long at = up * a.H + static_cast<long long>(h) * places, w0 = at / each;
      const int unit = (m0 + tid) * a.H + h;
      args.own[unit] = make_int2(static_cast<int>(blockIdx.y * warps + unit + w0),
                                 pages > 0 ? static_cast<int>((at + pages - 1) / each - w0) + 1 : 0);
    }
  if (tid == 0) begins[kChunk] = total;
  __syncthreads();
  // ---- the warp's pages ----------------------------------------------------------------------
  const long long w = static_cast<long long>(blockIdx.x) * kOwnWarps + warp;
  const long long f0 = w * each, f1 = min(f0 + each, all);
  const uint32_t ring = smem_u32(smem) + warp * kStages * kPage;
  const bool issuer = umma::elect_one();
  uint32_t qa[D / 16][2];
  Sums<D> sums_u;
  float2 qs = make_float2(0.f, 0.f);
  int unit = -1, len = 0, exponent = 0;  // the unit at hand, its sequence's length; what its O counts
  bool aborted = false;
  // the piece of `unit`, to the output if it is all of it
  auto flush = [&]() {
    const int i = unit / a.H, h = unit - i * a.H;
    const int places = static_cast<int>(begins[i + 1] - begins[i]);
    const long long at = begins[i] * a.H + static_cast<long long>(h) * places;
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      sums_u.l.x += __shfl_xor_sync(0xffffffffu, sums_u.l.x, x);
      sums_u.l.y += __shfl_xor_sync(0xffffffffu, sums_u.l.y, x);
    }
    const bool whole = from_s[i] == 0 && at >= f0 && at + places - kUnitCost <= f1;
    const size_t piece = blockIdx.y * warps + static_cast<long long>(m0) * a.H + unit + w;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int q = 2 * t + e;
      const float m = e ? sums_u.m.y : sums_u.m.x, l = e ? sums_u.l.y : sums_u.l.x;
      if (q >= gqa) continue;
      __nv_bfloat16* out = a.out + (static_cast<size_t>(seq_s[i]) * a.Hq + h * gqa + q) * D + kNt * g;
      float* part = args.part_o + (piece * gqa + q) * D + kNt * g;
#pragma unroll
      for (int j = 0; j < kNt; j += 4) {
        float4 x;
        x.x = e ? sums_u.o[j].y : sums_u.o[j].x;
        x.y = e ? sums_u.o[j + 1].y : sums_u.o[j + 1].x;
        x.z = e ? sums_u.o[j + 2].y : sums_u.o[j + 2].x;
        x.w = e ? sums_u.o[j + 3].y : sums_u.o[j + 3].x;
        if (whole) store_out4(out + j, x, l, exponent);
        else *reinterpret_cast<float4*>(part + j) = x;
      }
      if (!whole && g == 0)
        *reinterpret_cast<float4*>(args.part_ml + (piece * gqa + q) * 4) =
            make_float4(m, l, m == -INFINITY ? m : static_cast<float>(exponent), 0.f);
    }
  };
  const bool small = all < 0x7fffffff;
  int done = 0;  // places of this warp before the batch at hand
  for (long long f = f0; f < f1; f += 32) {
    // 32 places, a lane each: unit (-1: an empty place), position, page, scales
    const int n = static_cast<int>(min(f1 - f, 32LL));
    int key = -1, pos0 = 0, row = -1;
    float2 sc = make_float2(0.f, 0.f);
    if (lane < n) {
      const long long q = small ? static_cast<int>(f + lane) / a.H : (f + lane) / a.H;
      int lo = 0, hi = mc;  // the last member that begins at q or before
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (begins[mid] <= q) lo = mid;
        else hi = mid;
      }
      const int places = static_cast<int>(begins[lo + 1] - begins[lo]);
      const long long rem = f + lane - begins[lo] * a.H;
      const int h = small ? static_cast<int>(rem) / places : static_cast<int>(rem / places);
      const int place = static_cast<int>(rem - static_cast<long long>(h) * places);
      if (place < places - kUnitCost) {
        const int page = from_s[lo] / kPageSize + place;
        key = lo * a.H + h;
        pos0 = page * kPageSize;
        const int id = __ldg(a.page_table + static_cast<size_t>(seq_s[lo]) * a.max_pages + page);
        if (id < 0 || id >= a.num_pages) {
          record_error(OSCAR_DEVERR_PAGE_ID);
        } else {
          row = id * a.H + h;
          sc = __ldg(reinterpret_cast<const float2*>(a.scales) + row);
        }
      }
    }
    auto issue = [&](int k) {
      const int r = __shfl_sync(0xffffffffu, row, k);
      if (issuer) {
        const int c = done + k;
        const uint32_t bar = smem_u32(bars + c % kStages);
        if (r < 0) {
          mbar_arrive(bar);
        } else {
          mbar_arrive_expect_tx(bar, kPage);
          umma::tma_load_3d(ring + (c % kStages) * kPage, &map, 0, 0, r, bar);
        }
      }
      __syncwarp();
    };
    if (!aborted)
      for (int k = 0; k < min(n, kStages); ++k) issue(k);
    for (int k = 0; k < n; ++k) {
      const int u = __shfl_sync(0xffffffffu, key, k);
      if (u != unit && u >= 0) {
        if (unit >= 0) flush();
        unit = u;
        const int i = u / a.H, h = u - i * a.H;
        len = len_s[i];
        const float x =
            load_q<D>(a.q + (static_cast<size_t>(seq_s[i]) * a.Hq + h * gqa + min(g, gqa - 1)) * D, g < gqa, t, a.scale_log2, qa);
        qs = make_float2(__shfl_sync(0xffffffffu, x, 8 * t), __shfl_sync(0xffffffffu, x, 8 * t + 4));  // queries 2t, 2t + 1
        sums_u.m = make_float2(-INFINITY, -INFINITY);
        sums_u.l = make_float2(0.f, 0.f);
        exponent = 0;
#pragma unroll
        for (int j = 0; j < kNt; ++j) sums_u.o[j] = make_float2(0.f, 0.f);
      }
      if (aborted) continue;
      const int c = done + k;
      const bool ok = mbar_wait_bounded(smem_u32(bars + c % kStages), (c / kStages) & 1);
      if (__any_sync(0xffffffffu, !ok)) {
        // a copy did not land: the rest of this warp's pages are dropped, once the copies in flight are over
        aborted = true;
        if (lane == 0) record_error(OSCAR_DEVERR_TIMEOUT);
        for (int x = k; x < min(n, k + kStages); ++x)
          mbar_wait_bounded(smem_u32(bars + (done + x) % kStages), ((done + x) / kStages) & 1);
        continue;
      }
      const int r = __shfl_sync(0xffffffffu, row, k), p = __shfl_sync(0xffffffffu, pos0, k);
      float2 s = make_float2(__shfl_sync(0xffffffffu, sc.x, k), __shfl_sync(0xffffffffu, sc.y, k));
      if (r >= 0) {
        if (exponent == 0 && s.y > kOwnBigScale) {  // rare
          exponent = kBigUnit;
#pragma unroll
          for (int j = 0; j < kNt; ++j) sums_u.o[j] = f2mul(sums_u.o[j], make_float2(pow2i(-kBigUnit), pow2i(-kBigUnit)));
        }
        if (exponent != 0) s.y *= pow2i(-kBigUnit);
        attend_own<F, D>(ring + (c % kStages) * kPage, p, len, s, qs, qa, lane, sums_u);
      }
      __syncwarp();
      if (k + kStages < n) issue(k + kStages);
    }
    done += n;
  }
  if (unit >= 0) flush();
  // The kernel after the two waits for the second of them alone: its last block ends after the first.
  if (args.last && blockIdx.x + 1 == gridDim.x && blockIdx.y + 1 == gridDim.y) grid_dep_wait();
}

template <int F, int D>
__global__ void __launch_bounds__(kWarps * 32, 3) kv8_list_kernel(const __grid_constant__ CUtensorMap map,
                                                                  const __grid_constant__ ListArgs args) {
  split_body<F, D, true>(map, args);
}

struct MergeArgs {
  AttnArgs a;
  const int32_t* members;
  const int4* info;
  const int2* own;
  const float* own_o;  // as OwnArgs
  const float* own_ml;
  const float* pre_o;  // [items][H][tm][D], and [4]
  const float* pre_ml;
  int num_members, tm;
};

// WARPS of a block's four warps per (member, query head), 32 / WARPS partials at a time: a lane has the units of one.
constexpr int kMergeWarps = 4;
template <int D, int WARPS>
__global__ void __launch_bounds__(kMergeWarps * 32, 6) kv8_shared_merge_kernel(MergeArgs m) {
  __shared__ float4 part[kMergeWarps][D / 4];
  __shared__ float4 units[kMergeWarps];
  constexpr int kPass = 32 / WARPS, kSub = 128 / D, kFly = 8;  // D = 64: two half warps take every second partial
  const AttnArgs& a = m.a;
  const int lane = threadIdx.x & 31, c4 = lane % (D / 4), sub = lane / (D / 4);
  const int warp = threadIdx.x >> 5;
  const long long row = static_cast<long long>(blockIdx.x) * (kMergeWarps / WARPS) + warp / WARPS;
  grid_dep_wait();
  if (row >= static_cast<long long>(m.num_members) * a.Hq) return;
  const int i = static_cast<int>(row / a.Hq), hq = static_cast<int>(row - static_cast<long long>(i) * a.Hq);
  const int gqa = a.Hq / a.H, h = hq / gqa, hd = hq - h * gqa;
  const int4 info = m.info[i];
  const int b = __ldg(m.members + i);
  const int2 own = m.own[static_cast<size_t>(i) * a.H + h];
  if (info.x < 0 || b < 0 || b >= a.batch) return;  // not a member
  const int n_own = own.y, n = n_own + info.z;
  if (info.z == 0 && n_own <= 1) return;  // written by the kernel before
  const int x = info.w * gqa + hd;
  const float* own_o = m.own_o + (static_cast<size_t>(own.x) * gqa + hd) * D + 4 * c4;
  const float* own_ml = m.own_ml + (static_cast<size_t>(own.x) * gqa + hd) * 4;
  const size_t pre = (static_cast<size_t>(info.x + x / m.tm) * a.H + h) * m.tm + x % m.tm;
  const size_t step = static_cast<size_t>(info.y) * a.H * m.tm;  // from one split to the next
  const float* pre_o = m.pre_o + pre * D + 4 * (c4 ^ (x % m.tm & 7));
  float M = -INFINITY, R = -INFINITY, l = 0.f;  // units of l (2^M) and r (2^(M + R)); l: the lane's part
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = warp % WARPS * kPass; k0 < n; k0 += 32) {
    const int cnt = min(n - k0, kPass), k = k0 + lane;
    float4 v = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    if (lane < cnt)
      v = *reinterpret_cast<const float4*>(k < n_own ? own_ml + static_cast<size_t>(k) * gqa * 4 : m.pre_ml + (pre + (k - n_own) * step) * 4);
    float4 y[kFly];
    auto load = [&](int j0) {
#pragma unroll
      for (int e = 0; e < kFly; ++e) {
        const int j = j0 + e * kSub + sub, kk = k0 + j;
        y[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j < cnt)
          y[e] = *reinterpret_cast<const float4*>(kk < n_own ? own_o + static_cast<size_t>(kk) * gqa * D : pre_o + (kk - n_own) * step * D);
      }
    };
    load(0);
    float m1 = v.x, r1 = v.z;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m1, o), r2 = __shfl_xor_sync(0xffffffffu, r1, o);
      const float top = fmaxf(m1, m2);
      if (top > -INFINITY) r1 = fmaxf(r1 + (m1 - top), r2 + (m2 - top));
      m1 = top;
    }
    // onto what there is
    const float top = fmaxf(M, m1), base = top == -INFINITY ? 0.f : top;
    const float unit = fmaxf(R + (M - base), r1 + (m1 - base)), base_r = unit == -INFINITY ? 0.f : unit;
    float f, g;
    pow2_pair(M - base + R - base_r, f, g);
    r.x = r.x * f * g; r.y = r.y * f * g; r.z = r.z * f * g; r.w = r.w * f * g;
    l = l * fast_exp2(M - base) + fast_exp2(v.x - base) * v.y;
    M = top;
    R = unit;
    pow2_pair(v.x - base + v.z - base_r, f, g);
    for (int j0 = 0; j0 < cnt; j0 += kFly * kSub) {
      if (j0 > 0) load(j0);
#pragma unroll
      for (int e = 0; e < kFly; ++e) {
        const int j = min(j0 + e * kSub + sub, 31);
        const float fj = __shfl_sync(0xffffffffu, f, j), gj = __shfl_sync(0xffffffffu, g, j);
        r.x = fmaf(fj, y[e].x * gj, r.x); r.y = fmaf(fj, y[e].y * gj, r.y);
        r.z = fmaf(fj, y[e].z * gj, r.z); r.w = fmaf(fj, y[e].w * gj, r.w);
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (kSub == 2) {
    r.x += __shfl_xor_sync(0xffffffffu, r.x, 16);
    r.y += __shfl_xor_sync(0xffffffffu, r.y, 16);
    r.z += __shfl_xor_sync(0xffffffffu, r.z, 16);
    r.w += __shfl_xor_sync(0xffffffffu, r.w, 16);
  }
  if (WARPS > 1) {  // (a block has one row: all of it is here)
    if (lane < D / 4) part[warp][lane] = r;
    if (lane == 0) units[warp] = make_float4(M, l, R, 0.f);
    __syncthreads();
    if (warp > 0) return;
    float top = M;
    for (int w = 1; w < WARPS; ++w) top = fmaxf(top, units[w].x);
    const float base = top == -INFINITY ? 0.f : top;
    float unit = -INFINITY;
    for (int w = 0; w < WARPS; ++w) unit = fmaxf(unit, units[w].z + (units[w].x - base));
    const float base_r = unit == -INFINITY ? 0.f : unit;
    l = 0.f;
    r = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < WARPS; ++w) {
      const float4 y = part[w][c4], v = units[w];
      float f, g;
      pow2_pair(v.x - base + v.z - base_r, f, g);
      l = fmaf(fast_exp2(v.x - base), v.y, l);
      r.x = fmaf(f, y.x * g, r.x); r.y = fmaf(f, y.y * g, r.y); r.z = fmaf(f, y.z * g, r.z); r.w = fmaf(f, y.w * g, r.w);
    }
    R = unit;
  }
  if (lane < D / 4) store_out4(a.out + (static_cast<size_t>(b) * a.Hq + hq) * D + 4 * c4, r, l, R);
}

struct Plan {
  bool list;                 // every member by itself: ns splits of pps pages
  int ns, pps;
  int mt, parts, tm, items;  // of the prefix kernel; items 0: no prefix
  bool prefix_first;         // of the two kernels
  int chunks, blocks;        // of what is the members' own: rows of blocks, blocks of a row
  size_t off_ml, off_pre_o, off_pre_ml, off_info, off_own, total;
};

bool make_plan(const oscar_dims_t* d, int batch, int max_seq_len, int max_prefix, int max_own, int members, int groups, Plan* p) {
  if (check_dims(d) != OSCAR_OK || batch < 0 || members < 0 || members > 65535 || groups < 0 || groups > 65535 ||
      max_seq_len < 0 || max_prefix < 0 || max_own < 0 || max_prefix > max_seq_len || max_own > max_seq_len)
    return false;
  if (max_seq_len > kMaxLen || max_seq_len > static_cast<long long>(d->max_pages_per_seq) * kPageSize) return false;
  if (d->num_kv_heads > 65535 || static_cast<long long>(members) * d->num_q_heads > 0x7fffffffLL) return false;
  const int H = d->num_kv_heads, gqa = d->num_q_heads / H, sms = num_sms();
  *p = Plan{};
  // ---- prefixes once: tiles of 256 rows, smaller ones where a group has fewer rows (of several groups one holds, as a rule, the
  // sequences by themselves)
  const long long rows = static_cast<long long>(members) * gqa, likely = groups > 1 ? groups - 1 : 1;
  const long long each = (rows + likely - 1) / likely;
  p->mt = each > 128 ? 2 : 1;
  p->parts = each > 64 ? 1 : 2;
  p->tm = p->mt * 128 / p->parts;
  const long long most_tiles = rows / p->tm + groups;  // of one KV head: ragged ones, one a group, beyond the even ones
  const long long blocks = (max_prefix / kPageSize + kBlkPages - 1) / kBlkPages;
  // SMs for what is the members' own (k) beside waves of prefix blocks on the others, or one after the other (k = 0), whichever
  // should take least by these times (us): of a prefix block (128 tokens), of a CTA's start and end, of the merge with its launch,
  // of the bytes of the members' own tokens, of which half the bound is taken as likely.
  const double block_us = p->mt == 2 ? 2.0 : p->parts == 1 ? 1.3 : 0.95, start_us = p->mt == 2 ? 13 : 10, merge_us = 8;
  const double own_bytes = static_cast<double>(members) * H * max_own * d->head_dim;
  auto own_us = [&](int n) { return 8 + own_bytes / fmin(n * 40e3, 5.7e6); };  // 40 KB a us and SM, 5.7 TB/s in all
  int own_sms = sms;
  double best = 0;
  long long items = 0;
  // Or every member by itself, by the decode's times: 8 x 2048 12.8 us (19 over tiles), 16 x 2048 18.9 (20), 32 x 2048 33 (22).
  const double list_us = 7 + (own_bytes + 2.0 * members * H * max_prefix * d->head_dim) / (d->head_dim == 128 ? 6.2e6 : 5e6);
  if (blocks > 0 && rows > 0 && groups > 0 && groups <= kTable && list_us >= block_us + start_us + merge_us) {  // (the least below)
    const long long tiles = rows / p->tm > likely ? rows / p->tm : likely;
    for (int k = 0; k < sms; k += 4) {
      for (int w = 1; w <= 4; ++w) {
        const long long n = static_cast<long long>(w) * (sms - k) / H;
        if (n < tiles) continue;
        const double prefix = w * (static_cast<double>((blocks + n / tiles - 1) / (n / tiles)) * block_us + start_us);
        const double us = (k == 0 ? prefix + own_us(sms) : fmax(prefix, own_us(k))) + merge_us;
        if (items == 0 || us < best) {
          best = us;
          items = n;
          own_sms = k == 0 ? sms : k;
        }
      }
    }
    if (items > 0 && items < most_tiles) items = most_tiles;  // (0: more tiles than four waves have blocks)
    if (items > 0x7fffffffLL) return false;
  }
  p->list = items == 0 || list_us < best;
  size_t own;  // rows of partials
  if (p->list) {
    const long long most = static_cast<long long>(max_prefix) + max_own;
    const long long pages = ((most < max_seq_len ? most : max_seq_len) + kPageSize - 1) / kPageSize;
    p->pps = split_pages(pages, (members > 0 ? members : 1LL) * H);
    if (p->pps > kMaxPps) p->pps = kMaxPps;
    const long long ns = pages > 0 ? (pages + p->pps - 1) / p->pps : 1;
    if (ns > 65535 || ns * members * H > 0x7fffffffLL) return false;
    p->ns = static_cast<int>(ns);
    own = ns > 1 ? static_cast<size_t>(ns) * rows * H : 0;
  } else {
    p->items = static_cast<int>(items);
    // what takes longer goes first, if it leaves room for the other
    p->prefix_first = items * H <= sms - own_sms;
    // blocks of a chunk, fewer where their warps would have nothing
    p->chunks = (members + kChunk - 1) / kChunk;
    const long long chunk = members < kChunk ? members : kChunk, pages = (static_cast<long long>(max_own) + kPageSize - 1) / kPageSize;
    const long long use = (chunk * H * (pages + kUnitCost) + kOwnWarps * kLeastPages - 1) / (kOwnWarps * kLeastPages);
    const long long most = own_sms / p->chunks < use ? own_sms / p->chunks : use;
    p->blocks = static_cast<int>(most < 1 ? 1 : most);
    const long long pieces = static_cast<long long>(p->chunks) * p->blocks * kOwnWarps + static_cast<long long>(members) * H;
    if (pieces > 0x7fffffffLL) return false;
    own = static_cast<size_t>(pieces) * gqa;
  }
  const size_t pre = static_cast<size_t>(p->items) * H * p->tm;
  p->off_ml = align_up(own * d->head_dim * sizeof(float), 256);
  p->off_pre_o = p->off_ml + align_up(own * 4 * sizeof(float), 256);
  p->off_pre_ml = p->off_pre_o + align_up(pre * d->head_dim * sizeof(float), 256);
  p->off_info = p->off_pre_ml + align_up(pre * 4 * sizeof(float), 256);
  p->off_own = p->off_info + align_up(static_cast<size_t>(members) * sizeof(int4), 256);
  p->total = p->off_own + align_up(static_cast<size_t>(members) * sizeof(int2) * H, 256) + 256;
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
cudaError_t launch(const Plan& p, const ListArgs& li, const SharedArgs& sh, const OwnArgs& ow, const MergeArgs& me,
                   const CUtensorMap& map, cudaStream_t stream) {
  cudaError_t e;
  if (p.list) {
    auto k = kv8_list_kernel<F, D>;
    e = set_smem_limit_once(reinterpret_cast<const void*>(k), DecodeGeo<D>::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k, dim3(p.ns, me.a.H, me.num_members), dim3(kWarps * 32), DecodeGeo<D>::kSmem, stream, map, li);
    if (e != cudaSuccess || p.ns == 1) return e;
  } else {
    auto k = kv8_own_kernel<F, D>;
    e = set_smem_limit_once(reinterpret_cast<const void*>(k), OwnGeo<D>::kSmem);
    if (e != cudaSuccess) return e;
    for (const bool prefix : {p.prefix_first, !p.prefix_first}) {
      if (!prefix) e = launch_pdl(k, dim3(p.blocks, p.chunks), dim3(kOwnThreads), OwnGeo<D>::kSmem, stream, map, ow);
      else if (p.mt == 2) e = launch_prefix<F, D, 2, 1>(p, sh, stream);
      else if (p.parts == 2) e = launch_prefix<F, D, 1, 2>(p, sh, stream);
      else e = launch_prefix<F, D, 1, 1>(p, sh, stream);
      if (e != cudaSuccess) return e;
    }
  }
  const long long rows = static_cast<long long>(me.num_members) * me.a.Hq;
  if (p.list && p.ns > 8)  // few rows of many partials
    return launch_pdl(kv8_shared_merge_kernel<D, kMergeWarps>, dim3(static_cast<unsigned>(rows)), dim3(kMergeWarps * 32), 0, stream,
                      me);
  return launch_pdl(kv8_shared_merge_kernel<D, 1>, dim3(static_cast<unsigned>((rows + kMergeWarps - 1) / kMergeWarps)),
                    dim3(kMergeWarps * 32), 0, stream, me);
}

}  // namespace

extern "C" size_t oscar_kv8_decode_shared_workspace_bytes(const oscar_dims_t* dims, int32_t batch, int32_t max_seq_len,
                                                          int32_t max_prefix_len, int32_t max_own_len, int32_t num_members,
                                                          int32_t num_groups) {
  Plan p;
  return make_plan(dims, batch, max_seq_len, max_prefix_len, max_own_len, num_members, num_groups, &p) ? p.total : 0;
}

extern "C" oscar_status_t oscar_kv8_decode_shared_plan(const oscar_dims_t* dims, int32_t batch, int32_t max_seq_len,
                                                       int32_t max_prefix_len, int32_t max_own_len, int32_t num_members,
                                                       int32_t num_groups, int32_t* tile_rows, int32_t* prefix_blocks,
                                                       int32_t* own_blocks) {
  const oscar_status_t st = check_dims(dims);
  if (st != OSCAR_OK) return st;
  Plan p;
  if (!make_plan(dims, batch, max_seq_len, max_prefix_len, max_own_len, num_members, num_groups, &p)) return OSCAR_ERR_INVALID_ARG;
  if (tile_rows) *tile_rows = p.list ? 0 : p.tm;
  if (prefix_blocks) *prefix_blocks = p.items * dims->num_kv_heads;
  if (own_blocks) *own_blocks = p.list ? p.ns * dims->num_kv_heads * num_members : p.blocks * p.chunks;
  return OSCAR_OK;
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
  int2* own = reinterpret_cast<int2*>(w + plan.off_own);
  const ListArgs li{{a, floats(0), floats(plan.off_ml), plan.ns, plan.pps}, g, info, own, max_own_len};
  const SharedArgs sh{{a, floats(plan.off_pre_o), floats(plan.off_pre_ml), 0, 0, 0}, g, info, plan.prefix_first, !plan.prefix_first};
  const OwnArgs ow{a, g, info, own, floats(0), floats(plan.off_ml), max_own_len, !plan.prefix_first, plan.prefix_first};
  const MergeArgs me{a, members, info, own, floats(0), floats(plan.off_ml), floats(plan.off_pre_o), floats(plan.off_pre_ml),
                     num_members, plan.tm};
  cudaStream_t s = as_stream(stream);
  const bool d128 = dims->head_dim == 128;
  auto go = [&](auto f) {
    constexpr int F = decltype(f)::value;
    return d128 ? launch<F, 128>(plan, li, sh, ow, me, map, s) : launch<F, 64>(plan, li, sh, ow, me, map, s);
  };
  const cudaError_t e = kv_format == OSCAR_KV8_E4M3 ? go(std::integral_constant<int, kE4M3>{})
                                                    : go(std::integral_constant<int, kInt8>{});
  return e == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

oscar_status_t oscar_internal_kv8_shared_errors(uint32_t* flags, int reset) {
  return oscar::read_unit_errors(flags, reset) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}
