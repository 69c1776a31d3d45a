// Append to the 8-bit paged cache with rotary positions (oscar_kv8_rope_append): the keys are rotated on their way to codes,
// and the queries of the same tokens beside them, in one launch.
//
// A block has one page of one sequence (or a share of its heads, where there are few pages).  Its angles' cosines and sines
// are computed once into shared memory, for all heads; then every warp takes items: a (head, K | V) block of the page,
// rotated in fp32 (K), its largest magnitude by a warp butterfly, then its codes; or 16 rows of queries.  The next item's rows
// are on their way into shared memory meanwhile, the first one's beside the cosines.  The rotated key is not rounded before it
// becomes a code.  Bound by the bytes: 2 (Hq + 2 Hkv) in, 2 Hq + 2 Hkv out per channel: six prompts, 56 thousand tokens, 32 query
// and 8 KV heads, D = 128, 1.11 GB: 169 us, 6.6 TB/s, 98% of a plain copy of as many bytes (187 with each item's rows loaded into
// registers; as long with 20 warps an SM as with 16).  One token of each of 64 sequences: 4.0 us.
#include <type_traits>

#include "kv8.cuh"
#include "rope.cuh"

namespace {

using namespace oscar;
using namespace oscar::kv8;
using namespace oscar::rope;

constexpr int kWarps = 4, kThreads = kWarps * 32;

struct AppendArgs {
  Rope rope;
  const __nv_bfloat16* q;  // null: keys and values alone
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* q_out;
  long long q_stride, k_stride, v_stride, q_out_stride;
  const int32_t* t_start;
  const int32_t* positions;  // null: the positions in the sequence
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* granted;  // null: every sequence
  uint8_t* pages;
  float* scales;
  int Hq, H, num_pages, max_pages, max_new;
  long long num_tokens;
};

__device__ __forceinline__ void unpack8(uint4 v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint4* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// The larger, or NaN where either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <int F, int D, bool IL>
__global__ void __launch_bounds__(kThreads, 4) kv8_rope_append_kernel(AppendArgs a) {
  constexpr int kUnits = D / 16;           // of a row, 16 channels each
  constexpr int kRows = 32 / kUnits;       // rows of a warp at once
  constexpr int kIters = kPageSize / kRows;
  // (cos, sin) of row r, pair 8 u + j at [r][j][u]: a half warp reads 16 neighbouring values of two rows, which the padding
  // puts in different banks
  constexpr int kRowPad = D / 2 + (D == 128 ? 8 : 4);
  __shared__ float2 table[kPageSize][kRowPad];
  __shared__ uint4 stages[kWarps][2][2 * kIters][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.z;
  const int t0 = __ldg(a.t_start + b), t1 = __ldg(a.t_start + b + 1), L = __ldg(a.seq_lens + b);
  const int n = t1 - t0;
  if (n == 0) return;
  const bool refused = a.granted != nullptr && __ldg(a.granted + b) == 0;
  if (n < 0 || n > a.max_new || t0 < 0 || t1 > a.num_tokens || (!refused && (n > L || L > a.max_pages * kPageSize))) {
    if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) record_error(OSCAR_DEVERR_POSITION);
    return;
  }
  const int items_kv = 2 * a.H;
  if (refused) {  // its queries become zeros
    const int r0 = blockIdx.x * kPageSize, rows = min(n - r0, kPageSize), row16 = a.Hq * (D / 8);
    if (a.q != nullptr && rows > 0)
      for (int i = blockIdx.y * kThreads + tid; i < rows * row16; i += gridDim.y * kThreads)
        reinterpret_cast<uint4*>(a.q_out + (t0 + r0 + i / row16) * a.q_out_stride)[i % row16] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int p_first = L - n;
  const int j = p_first / kPageSize + blockIdx.x;  // page of the sequence
  if (j > (L - 1) / kPageSize) return;
  const int o0 = max(p_first - j * kPageSize, 0), o1 = min(L - j * kPageSize, kPageSize);  // new rows of the page
  const long long tok0 = static_cast<long long>(t0) + (j * kPageSize - p_first);  // token of the page's row 0
  const int unit = lane % kUnits, row0 = lane / kUnits;
  const bool turned = unit * 16 < a.rope.rotary;
  const int c0 = first_channel<8, IL>(unit, a.rope.rotary), c1 = second_channel<8, IL>(unit, a.rope.rotary);
  const int items_q = a.q != nullptr ? (a.Hq * (o1 - o0) + kPageSize - 1) / kPageSize : 0, items = items_kv + items_q;
  // A lane's pairs of (row, query head), of 16 of the page's, are kRows apart.
  auto first_pair = [&](int item, int& r, int& hd) {
    const int y = (item - items_kv) * kPageSize + row0;
    r = y / a.Hq;
    hd = y - r * a.Hq;
    r += o0;
  };
  auto next_pair = [&](int& r, int& hd) {
    r += kRows / a.Hq;
    hd += kRows % a.Hq;
    if (hd >= a.Hq) {
      hd -= a.Hq;
      ++r;
    }
  };
  // A lane's vectors of an item, on their way to memory that it alone reads, while it works on the item before.
  auto fetch = [&](int item, int buf) {
    uint4* to = &stages[warp][buf][0][lane];
    if (item >= items) {
    } else if (item >= items_kv) {
      int r, hd;
      first_pair(item, r, hd);
#pragma unroll
      for (int i = 0; i < kIters; ++i) {
        const __nv_bfloat16* src = a.q + (tok0 + min(r, o1 - 1)) * a.q_stride + hd * D;
        copy16(to + 64 * i, src + c0, r < o1);
        copy16(to + 64 * i + 32, src + c1, r < o1);
        next_pair(r, hd);
      }
    } else {
      const __nv_bfloat16* src = (item & 1 ? a.v : a.k) + static_cast<size_t>(item >> 1) * D;
      const long long stride = item & 1 ? a.v_stride : a.k_stride;
#pragma unroll
      for (int i = 0; i < kIters; ++i) {
        const int r = i * kRows + row0;
        const bool is_new = r >= o0 && r < o1;
        const __nv_bfloat16* row = src + (tok0 + (is_new ? r : o0)) * stride;
        copy16(to + 64 * i, row + c0, is_new);
        copy16(to + 64 * i + 32, row + c1, is_new);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const int item0 = blockIdx.y * kWarps + warp, step = gridDim.y * kWarps;
  fetch(item0, 0);
  int pid = __ldg(a.page_table + static_cast<size_t>(b) * a.max_pages + j);
  if (pid < 0 || pid >= a.num_pages) {  // (the queries go on)
    if (tid == 0 && blockIdx.y == 0) record_error(OSCAR_DEVERR_PAGE_ID);
    pid = -1;
  }
  const int half = a.rope.rotary / 2;
  for (int i = tid; i < (o1 - o0) * half; i += kThreads) {
    const int r = o0 + i / half, p = i % half;
    const int pos = a.positions != nullptr ? __ldg(a.positions + tok0 + r) : j * kPageSize + r;
    table[r][(p & 7) * kUnits + (p >> 3)] = cos_sin(__ldg(a.rope.turns + p), pos, a.rope.magnitude);
  }
  __syncthreads();
  int buf = 0;
  for (int item = item0; item < items; item += step, buf ^= 1) {
    fetch(item + step, buf ^ 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    const uint4* in = &stages[warp][buf][0][lane];
    if (item >= items_kv) {
      int r, hd;
      first_pair(item, r, hd);
#pragma unroll
      for (int i = 0; i < kIters; ++i) {
        if (r < o1) {
          uint4 v0 = in[64 * i], v1 = in[64 * i + 32];
          if (turned) {
            float y[16];
            unpack8(v0, y);
            unpack8(v1, y + 8);
            turn_unit<8, IL>(y, [&](int p) { return table[r][p * kUnits + unit]; });
            v0 = pack8(y);
            v1 = pack8(y + 8);
          }
          __nv_bfloat16* dst = a.q_out + (tok0 + r) * a.q_out_stride + hd * D;
          *reinterpret_cast<uint4*>(dst + c0) = v0;
          *reinterpret_cast<uint4*>(dst + c1) = v1;
        }
        next_pair(r, hd);
      }
      continue;
    }
    if (pid < 0) continue;
    const int h = item >> 1, side = item & 1;
    const size_t block = (static_cast<size_t>(pid) * a.H + h) * 2 + side;
    uint8_t* dst = a.pages + block * (kPageSize * D);
    const float stored = o0 > 0 ? a.scales[block] : 0.f;
    // Rows of a lane, rotated (K).  They are formed twice, for the largest magnitude and for the codes: 64 values kept would take
    // the registers of half the warps that an SM holds.
    const bool turns = side == 0 && turned;
    auto values = [&](int i, float (&x)[16]) {
      asm volatile("" ::: "memory");  // (a row at a time)
      const int r = i * kRows + row0;
      unpack8(in[64 * i], x);
      unpack8(in[64 * i + 32], x + 8);
      if (turns && r >= o0 && r < o1) turn_unit<8, IL>(x, [&](int p) { return table[r][p * kUnits + unit]; });
    };
    float top = 0.f;  // (a NaN stays one)
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      float x[16];
      values(i, x);
#pragma unroll
      for (int c = 0; c < 16; ++c) top = max_nan(top, fabsf(x[c]));
    }
    // As bits they order as the values do, infinity and NaN above all.
    uint32_t mx = __reduce_max_sync(0xffffffffu, __float_as_uint(top) & 0x7fffffffu);
    const bool has_nan = mx > 0x7f800000u;
    if (has_nan) {  // rare: NaN elements become 0, and the maximum is taken anew without them
      if (lane == 0) record_error(OSCAR_DEVERR_VALUE);
      top = 0.f;
#pragma unroll 1
      for (int i = 0; i < kIters; ++i) {
        float x[16];
        values(i, x);
#pragma unroll
        for (int c = 0; c < 16; ++c) top = fmaxf(top, fabsf(x[c]));  // (of a number and a NaN: the number)
      }
      mx = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
    }
    mx = min(mx, 0x7f7fffffu);  // infinities saturate: the scale is that of the largest finite value
    const float need = pow2i(scale_exponent<F>(__uint_as_float(mx)));
    const float scale = fmaxf(stored, need);
    const float inv = 1.f / scale;  // exact: a power of two between 2^-121 and 2^100
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const int r = i * kRows + row0;
      uint2* at0 = reinterpret_cast<uint2*>(dst + r * D + c0);
      uint2* at1 = reinterpret_cast<uint2*>(dst + r * D + c1);
      if (r >= o0 && r < o1) {
        float x[16];
        values(i, x);
        uint32_t o[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float f[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = has_nan && x[4 * c + e] != x[4 * c + e] ? 0.f : x[4 * c + e] * inv;
          o[c] = encode4<F>(f);
        }
        *at0 = make_uint2(o[0], o[1]);
        *at1 = make_uint2(o[2], o[3]);
      } else if (r < o0 && scale != stored) {  // an earlier row under a larger scale
        const uint2 old0 = *at0, old1 = *at1;
        const uint32_t v[4] = {old0.x, old0.y, old1.x, old1.y};
        const float ratio = stored * inv;
        uint32_t o[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float f[4];
          decode4<F>(v[c], f);
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] *= ratio;
          o[c] = encode4<F>(f);
        }
        *at0 = make_uint2(o[0], o[1]);
        *at1 = make_uint2(o[2], o[3]);
      }
    }
    if (lane == 0 && scale != stored) a.scales[block] = scale;
  }
}

}  // namespace

extern "C" oscar_status_t oscar_kv8_rope_append(
    const oscar_dims_t* dims, const oscar_rope_t* rope, int32_t kv_format, int32_t batch, int64_t num_tokens,
    int32_t max_tokens_per_seq, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
    int64_t v_stride, const int32_t* t_start, const int32_t* positions, const int32_t* page_table, const int32_t* seq_lens,
    const int32_t* granted, uint8_t* kv8_pages, float* kv8_scales, void* q_out, int64_t q_out_stride, void* stream) {
  oscar_status_t st = check_dims(dims);
  if (st != OSCAR_OK) return st;
  st = check_rope(rope, dims);
  if (st != OSCAR_OK) return st;
  if (kv_format != OSCAR_KV8_E4M3 && kv_format != OSCAR_KV8_INT8) return OSCAR_ERR_INVALID_ARG;
  if (batch < 0 || num_tokens < 0 || num_tokens > 0x7fffffffLL || max_tokens_per_seq < 0) return OSCAR_ERR_INVALID_ARG;
  if (num_tokens == 0) return OSCAR_OK;
  if (batch == 0 || max_tokens_per_seq == 0 || !k || !v || !t_start || !page_table || !seq_lens || !kv8_pages ||
      !kv8_scales || !q != !q_out)
    return OSCAR_ERR_INVALID_ARG;
  const int D = dims->head_dim, H = dims->num_kv_heads, Hq = dims->num_q_heads;
  if (misaligned16(k) || misaligned16(v) || misaligned16(kv8_pages) || misaligned16(kv8_scales) || bad_stride(k_stride, H, D, 2) ||
      bad_stride(v_stride, H, D, 2))
    return OSCAR_ERR_INVALID_ARG;
  if (q && (misaligned16(q) || misaligned16(q_out) || bad_stride(q_stride, Hq, D, 2) || bad_stride(q_out_stride, Hq, D, 2) ||
            bad_in_place(q, q_stride, q_out, q_out_stride, num_tokens)))
    return OSCAR_ERR_INVALID_ARG;
  if (batch > 65535 || static_cast<long long>(dims->max_pages_per_seq) * kPageSize > 0x7fffffffLL) return OSCAR_ERR_UNSUPPORTED;
  const long long most = max_tokens_per_seq < num_tokens ? max_tokens_per_seq : num_tokens;  // of one sequence
  const long long gx = (most + 2 * kPageSize - 2) / kPageSize;
  // Pages that get tokens, about; where they are few, their heads are dealt out to several blocks.
  const long long pages = num_tokens / kPageSize + batch;
  const long long rows = most < kPageSize ? most : kPageSize;
  const long long items = 2LL * H + (q ? (Hq * rows + kPageSize - 1) / kPageSize : 0);
  long long gy = 4LL * num_sms() / pages, gy_most = (items + kWarps - 1) / kWarps;
  gy = gy < 1 ? 1 : (gy > gy_most ? gy_most : gy);
  if (gy > 65535) gy = 65535;
  AppendArgs a{{rope->turns, rope->rotary_dim, rope->magnitude}, static_cast<const __nv_bfloat16*>(q),
               static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v),
               static_cast<__nv_bfloat16*>(q_out), q_stride, k_stride, v_stride, q_out_stride, t_start, positions,
               page_table, seq_lens, granted, kv8_pages, kv8_scales, Hq, H, dims->num_pages, dims->max_pages_per_seq,
               max_tokens_per_seq, num_tokens};
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy), batch);
  const bool d128 = D == 128, il = rope->interleaved != 0;
  auto pick = [&](auto f) {
    constexpr int F = decltype(f)::value;
    return d128 ? (il ? kv8_rope_append_kernel<F, 128, true> : kv8_rope_append_kernel<F, 128, false>)
                : (il ? kv8_rope_append_kernel<F, 64, true> : kv8_rope_append_kernel<F, 64, false>);
  };
  auto* kernel = kv_format == OSCAR_KV8_E4M3 ? pick(std::integral_constant<int, kE4M3>{})
                                             : pick(std::integral_constant<int, kInt8>{});
  kernel<<<grid, kThreads, 0, as_stream(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

oscar_status_t oscar_internal_kv8_rope_append_errors(uint32_t* flags, int reset) {
  return oscar::read_unit_errors(flags, reset) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}
