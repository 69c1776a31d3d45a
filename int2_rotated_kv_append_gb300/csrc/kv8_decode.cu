// Decode attention over the 8-bit paged cache (oscar_kv8_decode): one query row per sequence,
// full or with a sliding window and sinks.
//
// Split kernel: one CTA of 4 warps per (split, KV head, sequence), each warp every 4th page of the
// split.  A page (16 tokens, K then V, D bytes each) is one tensor copy into the warp's ring of
// kStages stages, swizzled so that every shared-memory read below is free of bank conflicts.  Per
// page and warp, with the GQA group's queries as the 8 rows of a 16-row fp16 tile:
//   S = Q K^T       ldmatrix rows of 16 codes -> fp16 pairs (exact) as the B operand.  Q is scaled by a power of
//                   two to below 2 so that fp16 holds it to 2^-25 of its largest element;
//   p = 2^(s - m)   m the page's own maximum, so the largest weight is 1; as two fp16 parts, hi = p * 2^14 and
//                   lo = (p - hi) * 2^26, it keeps 22 bits down to 2^-29 and a step of 2^-50 below,
//                   whatever the other pages hold.  The fragments of S are already those of P: hi parts in
//                   rows 0..7, lo parts in rows 8..15 of the same A operand;
//   O += f (P V)    f = 2^(m - running maximum) * the page's V scale, in fp32.  In a split with a scale over 2^90 (infinite V
//                   elements, saturated) O counts 2^40, so that sums of such values stay within fp32.
// Bound by the bytes of the pages (2 D per token and KV head): 64 sequences of 1024 to 16384 tokens, 8 KV heads,
// D = 128, 1.12 GB: 186 us with the merge, 6.0 TB/s, 89% of a plain copy's rate.  A page costs about 200
// instructions a warp; one sequence of 32768 tokens (67 MB) takes 20 us, half of it the start of the
// chain (length, page ids, first pages) and the merge.
// Then the warps are merged, and a second kernel merges the splits where there are several.
#include <math.h>

#include "kv8_attn.cuh"
#include "umma.cuh"

namespace {

using namespace oscar;
using namespace oscar::kv8;

constexpr int kWarps = 4;
constexpr float kHi = 16384.f, kLo = 4096.f;  // p * kHi and the rest * kLo as fp16
constexpr float kBigScale = 0x1p90f;  // up to here 2^90 times a code (2^9) times 2^27 tokens is within fp32
constexpr int kBigUnit = 40;
constexpr int kMaxPps = 512;  // page ids and scales of a split in shared memory

template <int D>
struct Geo {
  static constexpr int kPage = 2 * kPageSize * D;  // bytes of one page and head
  static constexpr int kStages = 16384 / kPage;    // 16 KB a warp
  static constexpr size_t kRing = static_cast<size_t>(kWarps) * kStages * kPage;
  static constexpr size_t kSmem = 1024 + kRing + kWarps * kStages * 8 + kMaxPps * 12;
};

struct SplitArgs {
  AttnArgs a;
  float* part_o;   // [batch][Hq][ns][D]
  float* part_ml;  // [batch][Hq][ns][4]
  int ns, pps;
};

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

// Byte offset of 16-byte chunk c of row r in a stage (the tensor copy's swizzle).
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ uint32_t pack_half2(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int F, int D>
__global__ void __launch_bounds__(kWarps * 32, 3) kv8_split_kernel(const __grid_constant__ CUtensorMap map,
                                                                   SplitArgs sa) {
  constexpr int kKs = D / 16;  // k-steps of QK; 16-byte chunks of a row
  constexpr int kNt = D / 8;   // n-tiles of PV; channels of a lane and token
  constexpr int kStages = Geo<D>::kStages, kPage = Geo<D>::kPage;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Geo<D>::kRing);
  float2* scale_s = reinterpret_cast<float2*>(bars + kWarps * kStages);
  int* pid_s = reinterpret_cast<int*>(scale_s + kMaxPps);
  const AttnArgs& a = sa.a;
  const int s = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int gqa = a.Hq / a.H;
  if (tid == 0) umma::prefetch_map(&map);
  grid_dep_wait();
  grid_dep_launch_dependents();
  const int L = clamped_len(a, b);
  const Visible vis = visible(L - 1, L - 1, a.sink, a.window);
  const int v0 = s * sa.pps, npg = min(sa.pps, vis.n - v0);
  if (npg <= 0) {
    if (s == 0)  // an empty sequence
      for (int i = tid; i < gqa * (D / 8); i += kWarps * 32)
        reinterpret_cast<uint4*>(a.out + (static_cast<size_t>(b) * a.Hq + h * gqa) * D)[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  for (int i = tid; i < npg; i += kWarps * 32) {
    int pid = __ldg(a.page_table + static_cast<size_t>(b) * a.max_pages + vis.page(v0 + i));
    if (pid < 0 || pid >= a.num_pages) {
      record_error(OSCAR_DEVERR_PAGE_ID);
      pid = -1;
    }
    pid_s[i] = pid;
  }
  uint64_t* my_bars = bars + warp * kStages;
  const uint32_t my_ring = smem_u32(smem) + warp * kStages * kPage;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(my_bars + i), 1);
    mbar_init_fence();
  }
  __syncthreads();
  const int n_my = (npg - warp + kWarps - 1) / kWarps;  // pages warp, warp + 4, ... of the split
  auto issue = [&](int i) {  // one lane
    const int pid = pid_s[warp + i * kWarps];
    const uint32_t bar = smem_u32(my_bars + i % kStages);
    if (pid < 0) {
      mbar_arrive(bar);
      return;
    }
    mbar_arrive_expect_tx(bar, kPage);
    umma::tma_load_3d(my_ring + (i % kStages) * kPage, &map, 0, 0, pid * a.H + h, bar);
  };
  const bool issuer = umma::elect_one();
  if (issuer)
    for (int i = 0; i < min(n_my, kStages); ++i) issue(i);

  // the scales, while the first pages are on their way
  bool big = false;
  for (int i = tid; i < npg; i += kWarps * 32)
    if (pid_s[i] >= 0) {
      const float2 x = __ldg(reinterpret_cast<const float2*>(a.scales) + static_cast<size_t>(pid_s[i]) * a.H + h);
      scale_s[i] = make_float2(x.x, x.y * (1.f / kHi));
      big = big || x.y > kBigScale;
    }

  // Q: lane (g, t) holds query g, channels 16 ks + 4 t .. + 3 (k = 2t, 2t+1, 2t+8, 2t+9 of k-step ks)
  uint32_t qa[kKs][2];
  float qs = 0.f;
  {
    const uint2* src =
        reinterpret_cast<const uint2*>(a.q + (static_cast<size_t>(b) * a.Hq + h * gqa + min(g, gqa - 1)) * D + 4 * t);
    uint2 x[kKs];
    uint32_t mx = 0;
#pragma unroll
    for (int ks = 0; ks < kKs; ++ks) {
      x[ks] = g < gqa ? __ldg(src + 4 * ks) : make_uint2(0, 0);
      mx = __vmaxu2(mx, __vmaxu2(x[ks].x & 0x7fff7fffu, x[ks].y & 0x7fff7fffu));
    }
    mx = max(mx & 0xffffu, mx >> 16);
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int e = min(max(static_cast<int>(mx >> 7) - 127, -126), 126);
    const float inv = pow2i(-e);
    qs = pow2i(e) * a.scale_log2;
#pragma unroll
    for (int ks = 0; ks < kKs; ++ks) {
      qa[ks][0] = pack_half2(__uint_as_float(x[ks].x << 16) * inv, __uint_as_float(x[ks].x & 0xffff0000u) * inv);
      qa[ks][1] = pack_half2(__uint_as_float(x[ks].y << 16) * inv, __uint_as_float(x[ks].y & 0xffff0000u) * inv);
    }
  }
  // O: query g, channels kNt (2t) + j and kNt (2t + 1) + j
  float2 o[kNt];
#pragma unroll
  for (int j = 0; j < kNt; ++j) o[j] = make_float2(0.f, 0.f);
  float m_run = -INFINITY, l_run = 0.f;  // l: this lane's tokens
  big = __syncthreads_or(big);  // scales
  if (big) {
    for (int i = tid; i < npg; i += kWarps * 32)
      if (pid_s[i] >= 0) scale_s[i].y *= pow2i(-kBigUnit);
    __syncthreads();
  }
  bool aborted = false;
  int i = 0;
  for (; i < n_my; ++i) {
    const bool ok = mbar_wait_bounded(smem_u32(my_bars + i % kStages), (i / kStages) & 1);
    if (__any_sync(0xffffffffu, !ok)) {
      aborted = true;
      break;
    }
    const int k = warp + i * kWarps;
    if (pid_s[k] >= 0) {
      const uint32_t st = my_ring + (i % kStages) * kPage;
      const float2 sc = scale_s[k];
      // (first: a logit may be within fp32 where its product with one of them is not; towards 0: never infinite, so that
      // logits of 0 stay 0)
      const float k_scale = __fmul_rz(sc.x, qs);
      const int pos0 = vis.page(v0 + k) * kPageSize;
      float acc[2][2][4];  // two chains of products per eight tokens
#pragma unroll
      for (int th = 0; th < 2; ++th) {
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[th][0][c] = acc[th][1][c] = 0.f;
#pragma unroll
        for (int c4 = 0; c4 < kKs; c4 += 4) {
          uint32_t w[4];
          ldmatrix_x4(st + chunk_at<D>(8 * th + (lane & 7), c4 + (lane >> 3)), w);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t b0, b1;
            codes_to_f16<F>(w[c], b0, b1);
            mma_f16(acc[th][c & 1], qa[c4 + c][0], 0u, qa[c4 + c][1], 0u, b0, b1);
          }
        }
      }
      // this lane's tokens: 2t, 2t+1, 2t+8, 2t+9
      float sx[4] = {acc[0][0][0] + acc[0][1][0], acc[0][0][1] + acc[0][1][1], acc[1][0][0] + acc[1][1][0],
                     acc[1][0][1] + acc[1][1][1]};
      const bool full = pos0 + kPageSize <= vis.end && (pos0 + kPageSize <= vis.sink_end || pos0 >= vis.lo);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        sx[c] *= k_scale;
        if (!full && !vis.sees(pos0 + 2 * t + (c & 1) + 8 * (c >> 1))) sx[c] = -INFINITY;
      }
      float mp = fmaxf(fmaxf(sx[0], sx[1]), fmaxf(sx[2], sx[3]));
      mp = fmaxf(mp, __shfl_xor_sync(0xffffffffu, mp, 1));
      mp = fmaxf(mp, __shfl_xor_sync(0xffffffffu, mp, 2));
      const float m_new = fmaxf(m_run, mp);
      if (__any_sync(0xffffffffu, m_new > m_run)) {
        const float alpha = m_run == -INFINITY ? 0.f : fast_exp2(m_run - m_new);
        l_run *= alpha;
#pragma unroll
        for (int j = 0; j < kNt; ++j) o[j] = f2mul(o[j], make_float2(alpha, alpha));
        m_run = m_new;
      }
      const float f = mp == -INFINITY ? 0.f : fast_exp2(mp - m_run);
      const float m_use = mp == -INFINITY ? 0.f : mp;
      float p[4];
      __half2 hi[2];
      uint32_t pa[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) p[c] = fast_exp2(sx[c] - m_use);
      l_run = fmaf(f, (p[0] + p[1]) + (p[2] + p[3]), l_run);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        hi[c] = __floats2half2_rn(p[2 * c] * kHi, p[2 * c + 1] * kHi);
        const float2 back = __half22float2(hi[c]);
        pa[2 * c] = *reinterpret_cast<const uint32_t*>(&hi[c]);
        pa[2 * c + 1] = pack_half2(fmaf(p[2 * c], kHi, -back.x) * kLo, fmaf(p[2 * c + 1], kHi, -back.y) * kLo);
      }
      const float fv = f * sc.y;
      const float2 fv2 = make_float2(fv, fv), lo2 = make_float2(1.f / kLo, 1.f / kLo);
      // V: this lane's tokens, channels kNt g .. kNt g + kNt - 1
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
        if (pos0 + kPageSize > vis.end && pos0 + r >= vis.end) {  // behind the last token: any bits, NaN included
#pragma unroll
          for (int q = 0; q < kNt / 4; ++q) w[c][q] = 0u;
        }
      }
#pragma unroll
      for (int q = 0; q < kNt / 4; ++q) {
        uint32_t b0[4], b1[4];  // channels 4 q + e: token pairs (2t, 2t+1) and (2t+8, 2t+9)
        codes_to_f16<F>(__byte_perm(w[0][q], w[1][q], 0x5140), b0[0], b0[1]);
        codes_to_f16<F>(__byte_perm(w[0][q], w[1][q], 0x7362), b0[2], b0[3]);
        codes_to_f16<F>(__byte_perm(w[2][q], w[3][q], 0x5140), b1[0], b1[1]);
        codes_to_f16<F>(__byte_perm(w[2][q], w[3][q], 0x7362), b1[2], b1[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          mma_f16(d, pa[0], pa[1], pa[2], pa[3], b0[e], b1[e]);
          o[4 * q + e] = f2fma(f2fma(make_float2(d[2], d[3]), lo2, make_float2(d[0], d[1])), fv2, o[4 * q + e]);
        }
      }
    }
    __syncwarp();
    if (issuer && i + kStages < n_my) issue(i + kStages);
  }
  if (aborted) {  // a copy did not land: drop this warp's pages, once the copies in flight are over
    if (lane == 0) record_error(OSCAR_DEVERR_TIMEOUT);
    for (int k = i; k < min(n_my, i + kStages); ++k)
      mbar_wait_bounded(smem_u32(my_bars + k % kStages), (k / kStages) & 1);
    m_run = -INFINITY;
    l_run = 0.f;
#pragma unroll
    for (int j = 0; j < kNt; ++j) o[j] = make_float2(0.f, 0.f);
  }
  l_run += __shfl_xor_sync(0xffffffffu, l_run, 1);
  l_run += __shfl_xor_sync(0xffffffffu, l_run, 2);
  // merge of the warps through shared memory (the ring is free: every copy has landed)
  __syncthreads();
  float* ml = reinterpret_cast<float*>(smem);     // [kWarps][8][2]
  float* ow = ml + kWarps * 16;                   // [kWarps][8][D]
  if (t == 0) {
    ml[(warp * 8 + g) * 2] = m_run;
    ml[(warp * 8 + g) * 2 + 1] = l_run;
  }
  if (g < gqa) {
    float* row = ow + (warp * 8 + g) * D + 2 * t * kNt;
#pragma unroll
    for (int j = 0; j < kNt; j += 4) {
      *reinterpret_cast<float4*>(row + j) = make_float4(o[j].x, o[j + 1].x, o[j + 2].x, o[j + 3].x);
      *reinterpret_cast<float4*>(row + kNt + j) = make_float4(o[j].y, o[j + 1].y, o[j + 2].y, o[j + 3].y);
    }
  }
  __syncthreads();
  const bool single = vis.n <= sa.pps;  // the only split of this sequence
  const float unit = big ? kBigUnit : 0.f;
  for (int idx = tid; idx < gqa * (D / 4); idx += kWarps * 32) {
    const int qi = idx / (D / 4), c4 = idx % (D / 4);
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[(w * 8 + qi) * 2]);
    float l = 0.f;
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = ml[(w * 8 + qi) * 2];
      const float wt = mw == -INFINITY ? 0.f : fast_exp2(mw - M);
      const float4 x = *reinterpret_cast<const float4*>(ow + (w * 8 + qi) * D + 4 * c4);
      l = fmaf(wt, ml[(w * 8 + qi) * 2 + 1], l);
      r.x = fmaf(wt, x.x, r.x); r.y = fmaf(wt, x.y, r.y); r.z = fmaf(wt, x.z, r.z); r.w = fmaf(wt, x.w, r.w);
    }
    const size_t row = static_cast<size_t>(b) * a.Hq + h * gqa + qi;
    if (single) {
      store_out4(a.out + row * D + 4 * c4, r, l, unit);
    } else {
      const size_t part = row * sa.ns + s;
      *reinterpret_cast<float4*>(sa.part_o + part * D + 4 * c4) = r;
      if (c4 == 0) *reinterpret_cast<float4*>(sa.part_ml + part * 4) = make_float4(M, l, M == -INFINITY ? M : unit, 0.f);
    }
  }
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
  if (pps == 0) {
    // Splits that fill whole waves of the 3 CTAs an SM holds, of 16 to 128 pages (longer ones leave uneven lengths
    // unbalanced): the cheapest of four wave counts, a wave taking its pages and as long as 16 more for start and end.
    // Against splits = slots / units rounded up: 8 x 8192 37 -> 30 us, 12 x 4096 31 -> 26, 32 x 4096 68 -> 58, 1 x 32768
    // the same.
    const long long units = static_cast<long long>(batch > 0 ? batch : 1) * d->num_kv_heads;
    const long long slots = 3LL * num_sms(), most = (pages + 4 * kWarps - 1) / (4 * kWarps);
    const long long least = (pages + 127) / 128;
    const long long waves = (least * units + slots - 1) / slots;
    long long best = 0;
    for (long long w = waves; w < waves + 4; ++w) {
      const long long splits = w * slots / units < most ? w * slots / units : most;
      if (splits < 1 || splits > 65535) continue;
      const long long len = (pages + splits - 1) / splits, cost = w * (len + 16);
      if (best == 0 || cost < best) {
        best = cost;
        pps = static_cast<int>(len);
      }
    }
    if (pps < 4 * kWarps) pps = 4 * kWarps;
  }
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
  cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(k), Geo<D>::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k, dim3(sa.ns, sa.a.H, sa.a.batch), dim3(kWarps * 32), Geo<D>::kSmem, stream, map, sa);
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
