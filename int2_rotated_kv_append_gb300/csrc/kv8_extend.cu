// Extend attention over the 8-bit paged cache (oscar_kv8_extend_varlen): the last rows of each sequence,
// causal, full or with a sliding window and sinks, on tcgen05.
//
// One CTA per (split, tile, KV head, sequence).  A tile is MT x 128 query rows, a row being one (position, query
// head of the group): MT = 2 for prompts, 1 where a sequence has at most 128 rows (drafts).  The pages that any row
// of the tile sees go through in blocks of 8 (128 tokens).  Roles of the 16 warps:
//   warps 13, 15  page ids and scales of the coming blocks; K and V codes into a ring by bulk copies;
//   warps 8..11   codes -> fp16 (exact) K and V operands in shared memory, two blocks deep, once per CTA (with MT = 1
//                 warps 4..7 take the V side);
//   warps 12, 14  issue S = Q K^T and O += P V (A = P from TMEM): apart, so that neither's waits hold up the other;
//   warps 0..7    softmax, one thread per row, one warpgroup per 128 rows: 128 logits from TMEM, weights back to
//                 TMEM as fp16.
// With at most 64 rows in a tile (PARTS = 2) every row is there twice, as tile rows r and r + 64: one takes the first
// 64 tokens of each block, the other the rest, each with a maximum, a sum and an accumulator of its own, and the
// weights of the other's tokens stay 0.  That halves what a thread does per block (2300 -> 1500 clocks); the two
// are merged at the end.
// TMEM (512 columns): with MT = 2 one logit buffer (128) for both row tiles, which is free again once a row tile has
// it in registers, so that the next logits of either tile are formed while both compute weights; a weight
// buffer (64) and an accumulator (D) per row tile.  With MT = 1 two logit buffers alternate, and Q is the products'
// left side from TMEM, so that at D = 128 its place in shared memory becomes a third stage of codes.
// Q is scaled per row by a power of two to below 2, where fp16 holds it to 2^-25 of the row's largest element; a page's K
// scale multiplies its 16 logits.  V scales 2^v go into the weights: the operand is 2^(s - m + v - r + 4) where m + r, the row's
// own, is at least the largest s + v that the row sees less 12, by which it may be passed before it moves; the sum has
// 2^(s - m), m likewise for s alone.  What the mask hides from a row has no part in its m and r (but that a page has one v).
// The weight of a row's largest logit is a power of two, which costs it no rounding.  O is rescaled in TMEM when r moves.
// Sums are fp32 over the unrounded weights.
// As long as the largest V scale so far is at most 2^kTame times a block's smallest, weights are fp16 (11 bits: a tenth of the
// output's own rounding) with the block's largest v, and the codes carry the ratio of their page's scale to it (exact).
// Then, whatever other tokens of its pages make of a row's r, a weight's smallest step is 2^-20 of the row's largest (2^-28
// where V scales are alike).  In other blocks ("wild": an infinite V element that was saturated, say) each page has its own v
// in the weights and the operands are bf16, weights (8 bits) and codes (exact) alike, with fp32's range of exponents:
// there r may stay kWildUp lower, so that a page whose scale comes from a token hidden from the row takes no bits from the
// row's other pages.
//
// Measured (GB300, 2070 MHz): 8192 rows over 16384 positions, 32 query heads, 8 KV heads, D = 128, e4m3: 1.21 ms,
// 1360 TFLOP/s, 71% of a cuBLAS bf16 product's rate (6.3 ms where the V scales of all pages are up to 2^20 apart).  A
// block takes 3300 clocks where the products alone would take 2050: the softmax of a row tile (1900: 512 of them exponentials, the rest the latencies of its waits and
// loads) and the expansion (about 2000 for K and V) run beside them on the same schedulers and the same
// shared-memory port.  One to eight rows of 8 sequences of up to 32768 positions (bound by 274 MB of codes): 87 us,
// 3.1 TB/s: a block takes about 1700 clocks where
// the codes would arrive in 1400, a CTA 5000 before its first block, and uneven lengths leave the last CTAs alone.
#include <math.h>

#include <type_traits>

#include "kv8_attn.cuh"
#include "umma.cuh"

namespace {

using namespace oscar;
using namespace oscar::kv8;

constexpr int kThreads = 512;
constexpr int kTok = 128;
constexpr int kBlkPages = kTok / kPageSize;
constexpr int kInfo = 6;          // blocks whose scales and positions are kept
static_assert(kInfo % 2 == 0, "two warps take turns");
// log2: how far a logit may pass the maximum in use (with 8, some row of a warp passed it in most blocks, and the
// rescale took 550 of 3400 clocks)
constexpr float kLazy = 11.9f;
constexpr int kBoost = 4;         // weights are stored times 2^kBoost: 2^(kLazy + kBoost) < 65504
constexpr float kTame = 8.f;      // log2 (the rare path takes 2 to 5 times as long: with 4, V scales that differ by 2^6 took it)
constexpr float kWildUp = 76.f;   // 2^(kWildUp + kLazy + kBoost) times a code (2^9) times 2^27 tokens is within fp32
// Bounds of lb (below) for blocks that are not wild: under kLbLo there are only scales of 0, above kLbHi weights under 2^-100
constexpr float kLbLo = -100.f, kLbHi = 126.f;
constexpr float kFar = 1048576.f;  // logits above this: sums with them lose what is small beside them
constexpr int kQkWarp = 12, kFetchK = 13, kPvWarp = 14, kFetchV = 15;
// Registers a thread: 512 x 128 at launch, divided among the warpgroups by setmaxnreg
constexpr int kRegsLaunch = 128;
template <int MT>
struct Regs {
  static constexpr int kSoftmax = MT == 2 ? 184 : 240, kExpand = MT == 2 ? 80 : 104, kIssue = 64;
  static_assert((MT == 2 ? 2 * kSoftmax + kExpand : kSoftmax + 2 * kExpand) + kIssue == 4 * kRegsLaunch,
                "the warpgroups share what was launched");
};

// What the fetching warp finds out about a block, for the warps that expand it and those that weigh it.
struct alignas(16) BlockInfo {
  float k_scale[kBlkPages];  // 1 where there is no page
  int pos[kBlkPages];        // first position; kNoPage: none
  __half v_ratio[kBlkPages];  // a page's V scale over the largest
  __half v_log2[kBlkPages];   // log2 of the V scale; -infinity: 0, or no page
  float v_top;                // the largest of them
  uint32_t flags;
};
constexpr int kNoPage = 0x7fffffff - kPageSize;
// flags: every row of row tile 0 / 1 sees the whole block; some row is behind the last token; V scales far apart
constexpr uint32_t kFull0 = 1, kTail = 4, kWild = 8;

template <int D, int MT>
struct Geo {
  static constexpr uint32_t kOp = kTok * D * 2;   // one fp16 operand: D / 64 blocks of 128 rows x 128 bytes
  // Stages of codes: whole pages of a block where two of them fit (half as many copies to issue), else K or V of a block
  static constexpr bool kWhole = MT == 1 || D == 64;
  static constexpr uint32_t kStage = (kWhole ? 2 : 1) * kTok * D;
  static constexpr bool kQStage = MT == 1 && D == 128;  // Q's rows, once they are in TMEM, become a third stage
  static constexpr int kRing = D == 128 ? (kQStage ? 3 : 2) : 4;
  static constexpr uint32_t kK = 0;
  static constexpr uint32_t kV = kK + 2 * kOp;
  static constexpr uint32_t kRaw = kV + 2 * kOp;
  static constexpr uint32_t kQ = kRaw + (kQStage ? 2 : kRing) * kStage;
  static constexpr uint32_t kBars = kQ + MT * kOp;
  static_assert(!kQStage || kOp == kStage, "Q has the place of a stage");
  // raw full, raw empty | K full, K empty, V full, V empty (2 each) | S full, S free, P full, PV done (2 each) |
  // info full, info free | Q in TMEM | end
  static constexpr int kNumBars = 2 * kRing + 8 + 8 + 2 * kInfo + 2;
  static constexpr bool kQTmem = MT == 1;
  static constexpr uint32_t kScale = kBars + ((kNumBars * 8 + 15) & ~15);  // [kInfo] BlockInfo
  static constexpr uint32_t kQs = kScale + kInfo * sizeof(BlockInfo);
  static constexpr uint32_t kMisc = kQs + MT * 128 * 4;
  static constexpr size_t kSmem = 1024 + kMisc + 16;
  static_assert(kSmem <= 232448, "what a CTA may have");
};

struct ExtArgs {
  AttnArgs a;
  float* part_o;   // [rows x Hq][ns][D]
  float* part_ml;  // [rows x Hq][ns][4]
  int ns, bps, tiles;
};

// A tile's rows and the pages they see.
struct Tile {
  int q0, n, L, r0, rows;  // first query row and rows of the sequence, its length; first row of the tile, rows
  Visible vis;
  int blocks;
  bool ok;
};

template <int TM>
__device__ __forceinline__ Tile tile_of(const AttnArgs& a, int b, int tile) {
  Tile t;
  t.q0 = __ldg(a.q_start + b);
  const int q1 = __ldg(a.q_start + b + 1);
  t.L = clamped_len(a, b);
  t.n = q1 - t.q0;
  t.ok = t.n >= 0 && t.n <= a.max_rows && t.q0 >= 0 && q1 <= a.rows;
  if (!t.ok) {
    record_error(OSCAR_DEVERR_POSITION);
    return t;
  }
  const int gqa = a.Hq / a.H;
  t.r0 = tile * TM;
  t.rows = min(TM, t.n * gqa - t.r0);
  t.ok = t.rows > 0;
  if (!t.ok) return t;
  const int first = t.L - t.n + t.r0 / gqa, last = t.L - t.n + (t.r0 + t.rows - 1) / gqa;
  if (first < 0) record_error(OSCAR_DEVERR_POSITION);
  t.vis = visible(max(first, 0), last, a.sink, a.window);
  if (last < 0) t.vis.n = 0;
  t.blocks = (t.vis.n + kBlkPages - 1) / kBlkPages;
  return t;
}

template <uint32_t N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <uint32_t N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w));
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ uint32_t half2_bits(float x, float y) {
  const __half2 v = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t bfloat2_bits(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The lowest n of 16 bits (n < 0: none).
__device__ __forceinline__ uint32_t low_bits(int n) { return (1u << min(max(n, 0), 16)) - 1u; }

template <int F, int D, int MT, int PARTS>
__global__ void __launch_bounds__(kThreads, 1) kv8_extend_kernel(ExtArgs ea) {
  using G = Geo<D, MT>;
  extern __shared__ uint8_t raw_smem[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(sm);
  const AttnArgs& a = ea.a;
  const int split = blockIdx.x / ea.tiles, tile = ea.tiles - 1 - blockIdx.x % ea.tiles;  // the longest tiles first
  const int h = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gqa = a.Hq / a.H;
  grid_dep_wait();
  grid_dep_launch_dependents();
  const Tile T = tile_of<MT * 128>(a, b, tile);
  if (!T.ok) return;
  const int blk0 = split * ea.bps, cnt = min(ea.bps, T.blocks - blk0);
  // output row (query row, head) of tile row r
  auto out_row = [&](int r) {
    const int x = T.r0 + r;
    return static_cast<size_t>(T.q0 + x / gqa) * a.Hq + h * gqa + x % gqa;
  };
  if (cnt <= 0) {
    if (split == 0)  // rows without any position
      for (int i = tid; i < T.rows * (D / 8); i += kThreads)
        reinterpret_cast<uint4*>(a.out + out_row(i / (D / 8)) * D)[i % (D / 8)] = make_uint4(0, 0, 0, 0);
    return;
  }

  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + G::kBars);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  constexpr int kRawFull = 0, kRawEmpty = G::kRing, kOpFull = 2 * G::kRing, kOpEmpty = kOpFull + 4,
                kSFull = kOpEmpty + 4, kSFree = kSFull + 2, kPFull = kSFree + 2, kPvDone = kPFull + 2, kInfoFull = kPvDone + 2,
                kInfoFree = kInfoFull + kInfo, kQFull = kInfoFree + kInfo, kEnd = kQFull + 1;
  // (operand barriers: 2 x side + buffer)
  BlockInfo* infos = reinterpret_cast<BlockInfo*>(sm + G::kScale);
  float* q_scale = reinterpret_cast<float*>(sm + G::kQs);
  // TMEM base; whether the codes in each V operand are bf16 (written and read as the operand itself)
  volatile uint32_t* misc = reinterpret_cast<uint32_t*>(sm + G::kMisc);
  const int active = (T.rows + 127) / 128;
  if (tid == 0) {
    for (int i = 0; i < G::kRing; ++i) {
      mbar_init(bar(kRawFull + i), G::kWhole ? 2 : 1);
      mbar_init(bar(kRawEmpty + i), MT == 2 ? 128 : 256);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(kOpFull + i), 128);
      mbar_init(bar(kOpEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kSFull + i), 1);
      mbar_init(bar(kSFree + i), 128);
      mbar_init(bar(kPFull + i), 128);
      mbar_init(bar(kPvDone + i), 1);
    }
    for (int i = 0; i < kInfo; ++i) {
      mbar_init(bar(kInfoFull + i), 1);
      mbar_init(bar(kInfoFree + i), 4 * active + 4);  // the warps that weigh, and those that expand V
    }
    mbar_init(bar(kQFull), 128 * active);
    mbar_init(bar(kEnd), 2);
    mbar_init_fence();
  }
  __syncthreads();
  const int wg = warp >> 2;
  const bool fetches = warp == kFetchK || warp == kFetchV;  // these start at once; the others get Q and TMEM ready
  if (warp == kQkWarp) umma::tmem_alloc(sb + G::kMisc, 512);
  // Q as fp16, K-major with the 128-byte swizzle: a lane takes 8 channels of a row, and every load is in flight at once
  if (wg < 3) {
    constexpr int kLanes = D / 8, kAtOnce = 12 * 32 / kLanes;  // lanes of a row; rows of one round of the 12 warps
    constexpr int kRounds = (MT * 128 / PARTS + kAtOnce - 1) / kAtOnce;
    const int c = lane % kLanes, r0 = tid / kLanes;
    int x = T.r0 + r0, i = x / gqa, hd = x - i * gqa;
    const __nv_bfloat16* src = a.q + (static_cast<size_t>(T.q0) * a.Hq + h * gqa) * D + 8 * c;
    uint4 v[kRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      v[k] = make_uint4(0u, 0u, 0u, 0u);
      if (r0 + k * kAtOnce < T.rows)
        v[k] = __ldg(reinterpret_cast<const uint4*>(src + (static_cast<size_t>(i) * a.Hq + hd) * D));
      i += kAtOnce / gqa;
      hd += kAtOnce % gqa;
      if (hd >= gqa) {
        hd -= gqa;
        ++i;
      }
    }
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const int r = r0 + k * kAtOnce;
      uint32_t mx = __vmaxu2(__vmaxu2(v[k].x & 0x7fff7fffu, v[k].y & 0x7fff7fffu),
                             __vmaxu2(v[k].z & 0x7fff7fffu, v[k].w & 0x7fff7fffu));
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mx = max(mx & 0xffffu, mx >> 16);
      const int e = min(max(static_cast<int>(mx >> 7) - 127, -126), 126);
      const float inv = pow2i(-e);
      const uint32_t in[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
      uint32_t y[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        y[q] = half2_bits(__uint_as_float(in[q] << 16) * inv, __uint_as_float(in[q] & 0xffff0000u) * inv);
      if (r < active * 128 / PARTS) {
#pragma unroll
        for (int copy = 0; copy < PARTS; ++copy) {
          const int rr = r + copy * (128 / PARTS);
          st_shared_v4(sb + G::kQ + (rr >> 7) * G::kOp + umma::sw128_offset(rr & 127, 8 * c, 128), y[0], y[1], y[2],
                       y[3]);
          if (c == 0) q_scale[rr] = pow2i(e) * a.scale_log2;
        }
      }
    }
  }
  if (!fetches) {
    fence_async();
    umma::fence_before_sync();
    asm volatile("bar.sync 1, %0;" ::"n"(kThreads - 64) : "memory");
    umma::fence_after_sync();
  }
  const uint32_t tmem = fetches ? 0u : misc[0];
  // logits, weights, accumulators
  const uint32_t s_tmem[2] = {tmem, MT == 2 ? tmem : tmem + 384};
  const uint32_t p_tmem[2] = {tmem + 128, tmem + 192};
  const uint32_t o_tmem[2] = {tmem + 256, tmem + 256 + D};
  const uint32_t q_tmem = tmem + 192;

  if (wg < MT) {
    // ---- softmax ---------------------------------------------------------------------------
    reg_inc<Regs<MT>::kSoftmax>();
    if (wg < active) {
      const int tr = wg * 128 + (tid & 127);                       // row of the products
      const int r = tr % (MT * 128 / PARTS), part = PARTS == 2 ? (tid >> 6) & 1 : 0;  // tile row; its part of every block
      constexpr int kCols = kTok / PARTS, kPages = kBlkPages / PARTS;  // of a part
      const uint32_t t_lane = static_cast<uint32_t>((warp & 3) * 32) << 16;
      if (G::kQTmem) {
#pragma unroll
        for (int half = 0; half < D / 64; ++half) {
          uint32_t x[32];
#pragma unroll
          for (int c = 0; c < 8; ++c)
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(x[4 * c]), "=r"(x[4 * c + 1]), "=r"(x[4 * c + 2]), "=r"(x[4 * c + 3])
                         : "r"(sb + G::kQ + wg * G::kOp + umma::sw128_offset(tr & 127, half * 64 + 8 * c, 128))
                         : "memory");
          umma::tmem_st32(q_tmem + t_lane + 32 * half, x);
        }
        umma::tmem_st_wait();
        umma::fence_before_sync();
        mbar_arrive(bar(kQFull));
      }
      const float qs = q_scale[tr];
      const int last_r = min(T.rows, wg * 128 + 128) - 1;  // rows behind it are zeros and not stored
      const int pos = T.L - T.n + (T.r0 + min(r, last_r)) / gqa;
      const int after = a.window > 0 ? max(pos - a.window, -1) : -1;  // visible: behind it, or a sink
      if (PARTS == 2) {  // the other part's weights are 0
        uint32_t z[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) z[e] = 0u;
        umma::tmem_st32(p_tmem[0] + t_lane + (part ^ 1) * (kCols / 2), z);
        umma::tmem_st_wait();
      }
      float m = -INFINITY, l = 0.f, r_unit = -INFINITY;
      bool ok = true;
      for (int j = 0; j < cnt; ++j) {
        const int sbuf = MT == 2 ? wg : j & 1;  // barrier and buffer of the logits
        const int info = j % kInfo;
        // (the block's info was there before its K was expanded, so before these logits)
        ok = ok && mbar_wait_bounded(bar(kSFull + sbuf), MT == 2 ? j & 1 : (j >> 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        umma::fence_after_sync();
        const BlockInfo& bi = infos[info];
        const uint32_t flags = bi.flags;
        uint32_t v[kCols / 32][32];
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) umma::tmem_ld32(s_tmem[sbuf] + t_lane + part * kCols + 32 * c, v[c]);
        umma::tmem_ld_wait();
        // bit c: the row sees token c of the part's page pg
        auto seen = [&](int pg) {
          const int pp = bi.pos[part * kPages + pg];
          return low_bits(pos - pp + 1) & (~low_bits(after - pp + 1) | low_bits(a.sink - pp));
        };
        // (exact; never infinite: towards 0, so that logits of 0 stay 0; never 0: -infinity stays that)
        auto k_scale = [&](float k) { return fmaxf(__fmul_rz(k, qs), 1.2e-38f); };
        // mx: the block's largest logit; vx: the largest of logit - mx + v.  m, r and what they count move where they have to.
        auto settle = [&](float mx, float vx) {
          // The product before is over: its weights' columns and O are free.  (Every phase of this barrier is waited
          // for in its turn: a parity says nothing two phases ahead.)
          if (j > 0) {
            ok = mbar_wait_bounded(bar(kPvDone + (MT == 2 ? wg : 0)), (j - 1) & 1);
            umma::fence_after_sync();
          }
          if (mx > m + kLazy || (m == -INFINITY && mx > -INFINITY)) {
            l *= fast_exp2(m - mx);
            r_unit += m - mx;
            m = mx;
          }
          const float top = mx == -INFINITY ? mx : mx - m + vx;
          const bool r_move = top > r_unit + kLazy || (r_unit == -INFINITY && top > -INFINITY);
          if (__any_sync(0xffffffffu, r_move)) {
            float gap = j > 0 && r_move ? fmaxf(r_unit - top, -240.f) : 0.f;  // (below: 0 in the end)
            if (r_move) r_unit = top;
            while (__any_sync(0xffffffffu, gap < 0.f)) {  // by up to 2^-120 at a time
              const float alpha = fast_exp2(fmaxf(gap, -120.f));
              gap = fminf(gap + 120.f, 0.f);
#pragma unroll 1  // (rare: kept small for the instruction cache)
              for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                umma::tmem_ld16(o_tmem[wg] + t_lane + 16 * c, o);
                umma::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                umma::tmem_st16(o_tmem[wg] + t_lane + 16 * c, o);
              }
              umma::tmem_st_wait();
            }
          }
        };
        if ((flags & kWild) == 0) {
          umma::fence_before_sync();
          mbar_arrive(bar(kSFree + sbuf));
          const float v_top = bi.v_top;
          float ks[kPages];
#pragma unroll
          for (int c = 0; c < kPages; c += 4) {
            const float4 x = *reinterpret_cast<const float4*>(bi.k_scale + part * kPages + c);
            ks[c] = k_scale(x.x); ks[c + 1] = k_scale(x.y); ks[c + 2] = k_scale(x.z); ks[c + 3] = k_scale(x.w);
          }
          if ((flags & (kFull0 << wg)) == 0) {
#pragma unroll
            for (int pg = 0; pg < kPages; ++pg) {
              const uint32_t see = seen(pg);
#pragma unroll
              for (int c = 0; c < 16; ++c)
                if ((see & (1u << c)) == 0) v[pg >> 1][(pg & 1) * 16 + c] = 0xff800000u;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kInfoFree + info));
          float mx = -INFINITY;
#pragma unroll
          for (int pg = 0; pg < kPages; ++pg) {
            const uint32_t* x = &v[pg >> 1][(pg & 1) * 16];
            float y = __uint_as_float(x[0]);
#pragma unroll
            for (int c = 1; c + 1 < 16; c += 2) y = fmax3(y, __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
            y = fmaxf(y, __uint_as_float(x[15]));
            mx = fmaxf(mx, y * ks[pg]);
          }
          settle(mx, v_top);
          // weights 2^(s - m + lb), lb = v - r + kBoost; the sum takes the 2^lb out again
          const float lb = fminf(fmaxf(v_top + (r_unit == -INFINITY ? 0.f : kBoost - r_unit), kLbLo), kLbHi);
          float off = lb - (m == -INFINITY ? 0.f : m);
          const bool far = fabsf(m) > kFar && m > -INFINITY;
          // rare: m is taken away before anything smaller is added, from the rounded product that m came from (a packed
          // subtraction would be fused with the packed product)
          if (__any_sync(0xffffffffu, far)) {
            const float m_far = far ? m : 0.f;
#pragma unroll
            for (int pg = 0; pg < kPages; ++pg) {
              const float k = far ? ks[pg] : 1.f;
#pragma unroll
              for (int c = 0; c < 16; c += 2) {
                uint32_t* x = &v[pg >> 1][(pg & 1) * 16 + c];
                const float2 y = f2mul(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), make_float2(k, k));
                x[0] = __float_as_uint(__fsub_rn(y.x, m_far));
                x[1] = __float_as_uint(__fsub_rn(y.y, m_far));
              }
              if (far) ks[pg] = 1.f;
            }
            if (far) off = lb;
          }
          const float2 off2 = make_float2(off, off);
          float2 sum[4];  // four chains of additions
#pragma unroll
          for (int c = 0; c < 4; ++c) sum[c] = make_float2(0.f, 0.f);
#pragma unroll
          for (int half = 0; half < kCols / 64; ++half) {
            uint32_t p[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const int col = half * 64 + 2 * c;
              const float k = ks[col >> 4];
              const float2 e = f2fma(make_float2(__uint_as_float(v[col >> 5][col & 31]),
                                                 __uint_as_float(v[col >> 5][(col & 31) + 1])),
                                     make_float2(k, k), off2);
              const float2 w = make_float2(fast_exp2(e.x), fast_exp2(e.y));
              sum[c & 3] = f2add(sum[c & 3], w);
              p[c] = half2_bits(w.x, w.y);
            }
            umma::tmem_st32(p_tmem[wg] + t_lane + part * (kCols / 2) + 32 * half, p);
          }
          umma::tmem_st_wait();
          umma::fence_before_sync();
          mbar_arrive(bar(kPFull + (MT == 2 ? wg : 0)));
          sum[0] = f2add(f2add(sum[0], sum[1]), f2add(sum[2], sum[3]));
          l = fmaf(sum[0].x + sum[0].y, fast_exp2(-lb), l);
        } else {
          // Rare: a page at a time, once for the largest and once for the weights (little code, for the instruction cache).
          float mx = -INFINITY, vx = -INFINITY;
#pragma unroll 1
          for (int pg = 0; pg < 2 * kPages; ++pg) {
            const int at = pg % kPages;
            if (pg == kPages) settle(mx, vx - kWildUp);
            uint32_t x[16];
            __syncwarp();
            umma::tmem_ld16(s_tmem[sbuf] + t_lane + part * kCols + 16 * at, x);
            umma::tmem_ld_wait();
            const uint32_t see = seen(at);
            const float k = k_scale(bi.k_scale[part * kPages + at]), v = __half2float(bi.v_log2[part * kPages + at]);
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if ((see & (1u << c)) == 0) x[c] = 0xff800000u;
            if (pg < kPages) {
              float y = -INFINITY;
#pragma unroll
              for (int c = 0; c < 16; ++c) y = fmaxf(y, __uint_as_float(x[c]));
              y *= k;
              if (y > -INFINITY) {
                const float m_all = fmaxf(mx, y);
                vx = fmaxf(vx + (mx - m_all), v + (y - m_all));
                mx = m_all;
              }
            } else {
              // (for the products and for the sum: their units may be further apart than a float's exponents reach)
              const float off = v + (r_unit == -INFINITY ? 0.f : kBoost - r_unit), m_use = m == -INFINITY ? 0.f : m;
              float sum = 0.f;
              uint32_t p[8];
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const float x0 = __fmul_rn(__uint_as_float(x[2 * c]), k) - m_use;
                const float x1 = __fmul_rn(__uint_as_float(x[2 * c + 1]), k) - m_use;
                sum += fast_exp2(x0) + fast_exp2(x1);
                p[c] = bfloat2_bits(fast_exp2(x0 + off), fast_exp2(x1 + off));
              }
              l += sum;
              umma::tmem_st8(p_tmem[wg] + t_lane + part * (kCols / 2) + 8 * at, p);
            }
          }
          umma::tmem_st_wait();
          umma::fence_before_sync();
          mbar_arrive(bar(kSFree + sbuf));
          mbar_arrive(bar(kPFull + (MT == 2 ? wg : 0)));
          if (lane == 0) mbar_arrive(bar(kInfoFree + info));  // (the stores' wait was the whole warp's)
        }
      }
      if (ok) ok = mbar_wait_bounded(bar(kPvDone + (MT == 2 ? wg : 0)), (cnt - 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok && lane == 0) record_error(OSCAR_DEVERR_TIMEOUT);
      umma::fence_after_sync();
      const bool single = T.blocks <= ea.bps;
      const bool store = r < T.rows;
      const size_t row = store ? out_row(r) : 0;
      float u = r_unit - kBoost;  // the accumulators count 2^(m + u)
      if (!ok) l = 0.f;
      float u0 = 1.f, u1 = 1.f, v0 = 0.f, v1 = 0.f;  // the parts' accumulators to the merged ones' unit; which saw nothing
      bool none0 = false, none1 = false;
      const float* theirs = nullptr;
      if (PARTS == 2) {
        // The two parts of a row are merged through the operands' memory (every product is over): each part hands over
        // the channels that the other stores.
        constexpr int kRow = D / 2 + 4;
        float* mine = reinterpret_cast<float*>(sm + G::kK) + (tid & 127) * kRow;
        theirs = reinterpret_cast<const float*>(sm + G::kK) + ((tid & 127) ^ 64) * kRow;
#pragma unroll 2
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[16];
          __syncwarp();
          umma::tmem_ld16(o_tmem[wg] + t_lane + (part ^ 1) * (D / 2) + 16 * c, o);
          umma::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<uint4*>(mine + 16 * c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
        none0 = l == 0.f;
        if (none0) m = u = -INFINITY;
        *reinterpret_cast<float4*>(mine + D / 2) = make_float4(m, l, u, 0.f);
        asm volatile("bar.sync 2, 128;" ::: "memory");
        const float4 x = *reinterpret_cast<const float4*>(theirs + D / 2);
        none1 = x.y == 0.f;
        const float top = fmaxf(m, x.x), base = top == -INFINITY ? 0.f : top;
        const float t0 = m - base + u, t1 = x.x - base + x.z, top_t = fmaxf(t0, t1), base_t = top_t == -INFINITY ? 0.f : top_t;
        l = (none0 ? 0.f : l * fast_exp2(m - base)) + (none1 ? 0.f : x.y * fast_exp2(x.x - base));
        pow2_pair(t0 - base_t, u0, u1);
        pow2_pair(t1 - base_t, v0, v1);
        m = top;
        u = top_t;
      }
      float f, g;
      pow2_pair(u, f, g);
      const float inv = l == 0.f ? 0.f : f / l;
#pragma unroll 2
      for (int c = part * (D / 32); c < (PARTS == 2 ? (part + 1) * (D / 32) : D / 16); ++c) {
        uint32_t o[16];
        __syncwarp();
        umma::tmem_ld16(o_tmem[wg] + t_lane + 16 * c, o);
        umma::tmem_ld_wait();
        if (PARTS == 2) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            o[e] = __float_as_uint((none0 ? 0.f : __uint_as_float(o[e]) * u0 * u1) +
                                   (none1 ? 0.f : theirs[16 * (c - part * (D / 32)) + e] * v0 * v1));
        }
        if (store && single) {
          uint32_t y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[e] = l == 0.f ? 0u : bfloat2_bits(__uint_as_float(o[2 * e]) * inv * g, __uint_as_float(o[2 * e + 1]) * inv * g);
          }
          uint4* dst = reinterpret_cast<uint4*>(a.out + row * D + 16 * c);
          dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
          dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
        } else if (store) {
          float4* dst = reinterpret_cast<float4*>(ea.part_o + (row * ea.ns + split) * D + 16 * c);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            dst[e] = l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                              : make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                            __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
        }
      }
      if (store && !single && part == 0)
        *reinterpret_cast<float4*>(ea.part_ml + (row * ea.ns + split) * 4) =
            l == 0.f ? make_float4(-INFINITY, 0.f, -INFINITY, 0.f) : make_float4(m, l, u, 0.f);
    }
  } else if (wg < 3) {
    // ---- codes -> fp16 operands: K and V in turn (MT = 2), V or K (MT = 1: warpgroups 1 and 2) ------------
    reg_dec<Regs<MT>::kExpand>();
    const int pt = tid & 127;
    constexpr int kChunks = D / 16;               // 16-byte chunks of a row of codes
    constexpr int kUnits = kTok * kChunks / 128;  // a thread's chunks: rows r0, r0 + kStep, ...
    constexpr int kStep = 128 / kChunks;
    // Lanes of the second 64 channels take the neighbouring row, so that the eight lanes of a shared-memory access meet
    // all banks both where they read (chunk c) and where they write (chunk 2 (c % 4) ^ row % 8).
    const int c = pt % kChunks, r0 = (pt / kChunks) ^ (c >> 2);
    // whole pages: a page's K rows, then its V rows
    const uint32_t src0 = sb + G::kRaw + c * 16 + (G::kWhole ? (r0 >> 4) * (2 * kPageSize * D) + (r0 & 15) * D : r0 * D);
    constexpr uint32_t kSrcStep = (G::kWhole ? 2 : 1) * kStep * D;
    // channels 16 c .. + 15 of row r: chunks 2 (c % 4), + 1 of 64-channel block c / 4
    const uint32_t dst0 = sb + G::kK + (c >> 2) * (kTok * 128) + r0 * 128 + (((2 * (c & 3)) ^ (r0 & 7)) << 4);
    const uint32_t dst1 = sb + G::kK + (c >> 2) * (kTok * 128) + r0 * 128 + (((2 * (c & 3) + 1) ^ (r0 & 7)) << 4);
    bool ok = true;
#pragma unroll 1
    for (int x = 0; x < (MT == 2 ? 2 : 1) * cnt; ++x) {
      const int j = MT == 2 ? x >> 1 : x, side = MT == 2 ? x & 1 : 2 - wg;
      const int op = 2 * side + (j & 1), rx = G::kWhole ? j : x, st = rx % G::kRing;
      ok = mbar_wait_bounded(bar(kRawFull + st), (rx / G::kRing) & 1) &&
           mbar_wait_bounded(bar(kInfoFull + j % kInfo), (j / kInfo) & 1);
      if (!ok) break;
      // every load first: the units are independent, and a load waits for nothing but itself
      uint32_t w[kUnits][4];
#pragma unroll
      for (int i = 0; i < kUnits; ++i)
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                     : "r"(src0 + st * G::kStage + (G::kWhole ? side * (kPageSize * D) : 0) + i * kSrcStep)
                     : "memory");
      if (MT == 1 || !G::kWhole || side == 1) mbar_arrive(bar(kRawEmpty + st));  // read: the next codes may come
      ok = j < 2 || mbar_wait_bounded(bar(kOpEmpty + op), ((j >> 1) - 1) & 1);
      if (!ok) break;
      const BlockInfo& bi = infos[j % kInfo];
      if (side == 1 && (bi.flags & kTail)) {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
          const int r = r0 + i * kStep;
          if (bi.pos[r >> 4] + (r & 15) >= T.L)
            w[i][0] = w[i][1] = w[i][2] = w[i][3] = 0u;  // any bits: behind the last token, or no page
        }
      }
      const uint32_t to = (side * 2 + (j & 1)) * G::kOp;  // the K buffers, then the V buffers
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const __half ratio = side == 1 ? bi.v_ratio[(r0 + i * kStep) >> 4] : __ushort_as_half(0x3c00);
        const __half2 f = __half2half2(ratio), f1152 = __hmul2(f, __half2half2(__ushort_as_half(0x6480)));
        uint32_t y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) codes_to_f16_scaled<F>(w[i][e], f, f1152, y[2 * e], y[2 * e + 1]);
        st_shared_v4(dst0 + to + i * (kStep * 128), y[0], y[1], y[2], y[3]);
        st_shared_v4(dst1 + to + i * (kStep * 128), y[4], y[5], y[6], y[7]);
      }
      if (side == 1) {
        const uint32_t wild = bi.flags & kWild;
        if (wild) {  // rare: this thread's values once more, as bf16 (exact)
#pragma unroll 1
          for (int i = 0; i < 2 * kUnits; ++i) {
            const uint32_t at = (i & 1 ? dst1 : dst0) + to + (i >> 1) * (kStep * 128);
            uint32_t y[4];
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
                         : "r"(at)
                         : "memory");
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&y[e]));
              y[e] = bfloat2_bits(x.x, x.y);
            }
            st_shared_v4(at, y[0], y[1], y[2], y[3]);
          }
        }
        if (pt == 0) misc[1 + (j & 1)] = wild;
      }
      fence_async();
      mbar_arrive(bar(kOpFull + op));
      if (side == 1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kInfoFree + j % kInfo));
      }
    }
    if (!ok && lane == 0) record_error(OSCAR_DEVERR_TIMEOUT);
  } else {
    reg_dec<Regs<MT>::kIssue>();
    if (warp == kFetchK || warp == kFetchV) {
      // ---- page ids, scales, copies of codes: K by one warp, V by another (whole pages: four each) --------------
      const int side = warp == kFetchV;
      const int32_t* table = a.page_table + static_cast<size_t>(b) * a.max_pages;
      // Four blocks at a time, a page a lane: the ids are loaded two groups ahead and the scales one,
      // so that neither is waited for.
      auto look_up = [&](int g) {  // page id (-2: none)
        const int v = blk0 * kBlkPages + g * 32 + lane;
        return g * 32 + lane < cnt * kBlkPages && v < T.vis.n ? __ldg(table + T.vis.page(v)) : -2;
      };
      auto checked = [&](int id) {
        if (id != -2 && (id < 0 || id >= a.num_pages)) record_error(OSCAR_DEVERR_PAGE_ID);
        return id >= 0 && id < a.num_pages ? id : -1;
      };
      auto scales = [&](int id) {
        return id >= 0 && (G::kWhole || side == 0)
                   ? __ldg(reinterpret_cast<const float2*>(a.scales) + static_cast<size_t>(id) * a.H + h)
                   : make_float2(1.f, 0.f);
      };
      // every row of row tile t sees the positions up to p_lo[t] that are behind p_after[t], or in the sink
      int p_lo[MT], p_after[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        p_lo[t] = T.L - T.n + (T.r0 + t * 128) / gqa;
        p_after[t] = a.window > 0 ? T.L - T.n + (T.r0 + min(T.rows, t * 128 + 128) - 1) / gqa - a.window : -1;
      }
      const bool issuer = umma::elect_one();
      int pid = -1, pid1 = checked(look_up(0)), pid2 = look_up(1);
      float2 sc = make_float2(1.f, 0.f), sc1 = scales(pid1);
      float v_top = -INFINITY;  // log2 of the largest V scale of all blocks looked at
      float v_own = -INFINITY, v_blk = -INFINITY;  // of this lane's page and block
      bool wild = false;
      bool ok = true;
      int issued = 0;
      for (int j = 0; j < cnt && ok; ++j) {
        const int info = j % kInfo;
        if ((j & 3) == 0) {
          pid = pid1;
          sc = sc1;
          pid1 = checked(pid2);
          sc1 = scales(pid1);
          pid2 = look_up((j >> 2) + 2);
          // of the lane's block (8 lanes): largest so far and smallest V scale
          v_own = scale_log2_of(sc.y);
          float hi = v_own, lo = v_own == -INFINITY ? INFINITY : v_own;
#pragma unroll
          for (int o = 1; o < kBlkPages; o <<= 1) {
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
          }
          v_blk = hi;
#pragma unroll
          for (int o = kBlkPages; o < 32; o <<= 1) {
            const float before = __shfl_up_sync(0xffffffffu, hi, o);
            if (lane >= o) hi = fmaxf(hi, before);
          }
          hi = fmaxf(hi, v_top);
          v_top = __shfl_sync(0xffffffffu, hi, 31);
          wild = lo < hi - kTame;
        }
        const bool mine = (lane >> 3) == (j & 3);  // this lane holds a page of block j
        const bool copies = mine && pid >= 0 && (!G::kWhole || ((lane >> 2) & 1) == side);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, copies)) * ((G::kWhole ? 2 : 1) * kPageSize * D);
        const int x = G::kWhole ? j : 2 * j + side, st = x % G::kRing;
        if (G::kQStage && x == 2) ok = mbar_wait_bounded(bar(kQFull), 0);
        if (x >= G::kRing) ok = mbar_wait_bounded(bar(kRawEmpty + st), (x / G::kRing - 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        constexpr int kCopies = G::kWhole ? kBlkPages / 2 : kBlkPages;
        int ids[kCopies];
#pragma unroll
        for (int c = 0; c < kCopies; ++c)
          ids[c] = __shfl_sync(0xffffffffu, pid, (j & 3) * kBlkPages + c + (G::kWhole ? side * kCopies : 0));
        if (issuer) {  // (one lane: eight lanes with a copy each take longer than one lane with eight)
          if (bytes > 0) mbar_arrive_expect_tx(bar(kRawFull + st), bytes);
          else mbar_arrive(bar(kRawFull + st));
          const uint32_t dst = sb + G::kRaw + st * G::kStage;
#pragma unroll
          for (int c = 0; c < kCopies; ++c) {
            if (ids[c] < 0) continue;
            const uint8_t* src = a.pages + (static_cast<size_t>(ids[c]) * a.H + h) * (2 * kPageSize * D);
            if (G::kWhole) bulk_g2s(dst + (side * kCopies + c) * (2 * kPageSize * D), src, 2 * kPageSize * D, bar(kRawFull + st));
            else bulk_g2s(dst + c * (kPageSize * D), src + side * (kPageSize * D), kPageSize * D, bar(kRawFull + st));
          }
        }
        __syncwarp();
        issued = j + 1;
        if (side == (G::kWhole ? j & 1 : 0)) {  // (whole pages: the two warps take turns)
          if (j >= kInfo) ok = mbar_wait_bounded(bar(kInfoFree + info), (j / kInfo - 1) & 1);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          const int pos = pid < 0 ? kNoPage : T.vis.page((blk0 + j) * kBlkPages + (lane & 7)) * kPageSize;
          auto any = [&](bool x) { return __any_sync(0xffffffffu, mine & x); };
          uint32_t flags = 0;
#pragma unroll
          for (int t = 0; t < MT; ++t)
            if (!any((pos > p_lo[t] - (kPageSize - 1)) | ((pos <= p_after[t]) & (pos > a.sink - kPageSize))))
              flags |= kFull0 << t;
          if (any((pid < 0) | (pos > T.L - kPageSize))) flags |= kTail;
          if (any(wild)) flags |= kWild;
          if (mine) {
            BlockInfo& bi = infos[info];
            bi.k_scale[lane & 7] = sc.x;
            // (exact; for a wild block's bf16 the codes as they are)
            bi.v_ratio[lane & 7] = __float2half_rn(wild ? 1.f : fast_exp2(v_own == -INFINITY ? v_own : v_own - v_blk));
            bi.v_log2[lane & 7] = __float2half_rn(v_own);
            bi.pos[lane & 7] = pos;
            if ((lane & 7) == 0) {
              bi.v_top = v_blk;
              bi.flags = flags;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kInfoFull + info));
        }
      }
      if (!ok) {  // wait for the copies in flight
        if (lane == 0) record_error(OSCAR_DEVERR_TIMEOUT);
        constexpr int kBack = G::kWhole ? G::kRing : G::kRing / 2;
        for (int j = max(0, issued - kBack); j < issued; ++j) {
          const int x = G::kWhole ? j : 2 * j + side;
          mbar_wait_bounded(bar(kRawFull + x % G::kRing), (x / G::kRing) & 1);
        }
      }
    } else if (warp == kQkWarp || warp == kPvWarp) {
      // ---- products ---------------------------------------------------------------------------------
      // The whole warp goes through this code and one elected lane issues: with uniform control flow the
      // operands stay in uniform registers (65 clocks a 128 x 128 x 16 product with A in TMEM, the pipe's rate, where a branch
      // on the lane number took 112).
      constexpr uint32_t kIdQk = umma::idesc_f16_f32(128, kTok, false), kIdPv = umma::idesc_f16_f32_b_mn(128, D),
                         kIdPvBf16 = umma::idesc_bf16_f32_b_mn(128, D);
      const bool issuer = umma::elect_one();
      bool ok = true;
      auto wait = [&](int i, int parity) { ok = ok && mbar_wait_bounded(bar(i), parity & 1); };
      const int nt = MT == 2 ? active : 1;
      if (warp == kQkWarp) {
        if (G::kQTmem) wait(kQFull, 0);
        for (int j = 0; j < cnt && ok; ++j) {
          const int buf = j & 1;
          const uint64_t dk = umma::desc_k_sw128(sb + G::kK + buf * G::kOp);
          wait(kOpFull + buf, j >> 1);
          for (int t = 0; t < nt; ++t) {
            // the logit buffer has been read: by the row tile before (MT = 2), two blocks ago (MT = 1)
            if (MT == 1) {
              if (j >= 2) wait(kSFree + buf, (j >> 1) - 1);
            } else if (t == 1) {
              wait(kSFree + 0, j);
            } else if (j > 0) {
              wait(kSFree + (nt - 1), j - 1);
            }
            if (!__all_sync(0xffffffffu, ok)) {
              ok = false;
              break;
            }
            umma::fence_after_sync();
            const int sbuf = MT == 2 ? t : buf;
            const uint64_t dq = umma::desc_k_sw128(sb + G::kQ + t * G::kOp);
            if (issuer) {
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t off = ((ks >> 2) * (kTok * 128) + (ks & 3) * 32) >> 4;  // within the address field
                if (G::kQTmem) umma::mma_f16_ts(s_tmem[sbuf], q_tmem + ks * 8, dk + off, kIdQk, ks > 0);
                else umma::mma_bf16(s_tmem[sbuf], dq + off, dk + off, kIdQk, ks > 0);
              }
              umma::commit(bar(kSFull + sbuf));
              if (t == nt - 1) umma::commit(bar(kOpEmpty + buf));
            }
            __syncwarp();
          }
        }
      } else {
        for (int j = 0; j < cnt && ok; ++j) {
          const int buf = j & 1;
          const uint64_t dv = umma::desc_mn_sw128(sb + G::kV + buf * G::kOp, kTok * 128);
          wait(kOpFull + 2 + buf, j >> 1);
          const uint32_t id = __shfl_sync(0xffffffffu, misc[1 + buf], 0) ? kIdPvBf16 : kIdPv;
          for (int t = 0; t < nt; ++t) {
            wait(kPFull + t, j);
            if (!__all_sync(0xffffffffu, ok)) {
              ok = false;
              break;
            }
            umma::fence_after_sync();
            if (issuer) {
#pragma unroll
              for (int ks = 0; ks < kTok / 16; ++ks)
                umma::mma_f16_ts(o_tmem[t], p_tmem[t] + ks * 8, dv + ks * (2048 >> 4), id, j > 0 || ks > 0);
              umma::commit(bar(kPvDone + t));
              if (t == nt - 1) umma::commit(bar(kOpEmpty + 2 + buf));
            }
            __syncwarp();
          }
        }
      }
      if (!ok && lane == 0) record_error(OSCAR_DEVERR_TIMEOUT);
      if (issuer) umma::commit(bar(kEnd));  // every product is over before TMEM is freed
      mbar_wait_bounded(bar(kEnd), 0);
    }
  }
  __syncwarp();
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  if (warp == kQkWarp) umma::tmem_dealloc(misc[0], 512);
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

// Whether the kernel has the launch registers that its warpgroups divide among themselves (if it had
// fewer, they would wait for registers that nobody gives back).
bool has_launch_registers(const void* f) {
  cudaFuncAttributes at{};
  return cudaFuncGetAttributes(&at, f) == cudaSuccess && at.numRegs == kRegsLaunch;
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
