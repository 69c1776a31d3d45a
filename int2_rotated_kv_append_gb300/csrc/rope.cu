// Rotary positions of query and key rows (oscar_rope), and the frequencies they turn by (oscar_rope_turns, on the host).
//
// A thread has one unit (16 channels of bf16) of one token and goes over the heads, so that the angles' cosines and sines
// are read once: a block computes them for its tokens, one each a thread, into shared memory.  A warp's loads are whole
// rows of neighbouring heads.  Bound by the bytes, each element once in and once out: 16384 tokens of 40 heads, D = 128, bf16, 336 MB:
// 54.3 us, 6.2 TB/s, as long as a plain copy of as many bytes; 64 tokens 2.5 us.
#include "rope.cuh"

namespace {

using namespace oscar;
using namespace oscar::rope;

constexpr int kThreads = 256;

struct Rows {
  const void* in;
  void* out;
  long long in_stride, out_stride;  // elements
  int heads;
};

struct RopeArgs {
  Rope rope;
  const int32_t* positions;
  Rows q, k;
  long long tokens;
};

template <typename T>
struct Vec;  // 16 bytes
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void unpack(uint4 v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<__half> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void unpack(uint4 v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = p.x;
      x[2 * i + 1] = p.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 p = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void unpack(uint4 v, float* x) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};

// TOK tokens of a block.  A thread has one head's row in flight, at five blocks an SM: 16384 tokens take 54.3 us, 57.5 at four, 55.5 with
// two rows at four, 58 with the first rows loaded behind the cosines.
template <typename T, int D, bool IL, int TOK>
__global__ void __launch_bounds__(kThreads, TOK == 1 ? 4 : 5) rope_kernel(RopeArgs a) {
  constexpr int E = Vec<T>::E, kUnits = D / (2 * E);
  constexpr int kGroups = kThreads / (TOK * kUnits);  // heads of a token at once
  __shared__ float2 table[TOK][D / 2];
  const long long t0 = static_cast<long long>(blockIdx.x) * TOK;
  const int half = a.rope.rotary / 2;
  const int unit = threadIdx.x % kUnits, tok = threadIdx.x / (kUnits * kGroups);
  const long long t = t0 + tok;
  const bool turned = unit * 2 * E < a.rope.rotary;
  const int c0 = first_channel<E, IL>(unit, a.rope.rotary), c1 = second_channel<E, IL>(unit, a.rope.rotary);
  const int all = a.q.heads + a.k.heads;
  // (channels that pass through, in place, are left alone)
  const bool idle = !turned && a.q.in == a.q.out && a.k.in == a.k.out;
  int h = t < a.tokens && !idle ? threadIdx.x / kUnits % kGroups : all;
  uint4 v0, v1;
  auto load = [&]() {
    if (h >= all) return;
    const T* src = h >= a.q.heads ? static_cast<const T*>(a.k.in) + t * a.k.in_stride + (h - a.q.heads) * D
                                  : static_cast<const T*>(a.q.in) + t * a.q.in_stride + h * D;
    v0 = *reinterpret_cast<const uint4*>(src + c0);
    v1 = *reinterpret_cast<const uint4*>(src + c1);
  };
  load();  // the first head's row, beside the cosines
  for (int i = threadIdx.x; i < TOK * half; i += kThreads) {
    const int s = i / half, p = i - s * half;
    if (t0 + s < a.tokens) table[s][p] = cos_sin(__ldg(a.rope.turns + p), __ldg(a.positions + t0 + s), a.rope.magnitude);
  }
  __syncthreads();
  float2 cs[E];
  if (turned) {
#pragma unroll
    for (int j = 0; j < E; ++j) cs[j] = table[tok][unit * E + j];
  }
  while (h < all) {
    T* dst = h >= a.q.heads ? static_cast<T*>(a.k.out) + t * a.k.out_stride + (h - a.q.heads) * D
                            : static_cast<T*>(a.q.out) + t * a.q.out_stride + h * D;
    if (turned) {
      float x[2 * E];
      Vec<T>::unpack(v0, x);
      Vec<T>::unpack(v1, x + E);
      turn_unit<E, IL>(x, [&](int j) { return cs[j]; });
      v0 = Vec<T>::pack(x);
      v1 = Vec<T>::pack(x + E);
    }
    *reinterpret_cast<uint4*>(dst + c0) = v0;
    *reinterpret_cast<uint4*>(dst + c1) = v1;
    h += kGroups;
    load();
  }
}

template <typename T, int D, bool IL>
cudaError_t launch(const RopeArgs& a, cudaStream_t stream) {
  // (four tokens a block: 16384 take 54.3 us, 59 with two and 55 with eight; one where they would be too few for a block an SM: 400
  // of 40 heads 3.4 us; 1000 take 4.9 us with four, 5.8 with one)
  constexpr int kTok = 4;
  if (a.tokens > static_cast<long long>(kTok) * num_sms()) {
    rope_kernel<T, D, IL, kTok><<<static_cast<unsigned>((a.tokens + kTok - 1) / kTok), kThreads, 0, stream>>>(a);
  } else {
    rope_kernel<T, D, IL, 1><<<static_cast<unsigned>(a.tokens), kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const RopeArgs& a, int dim, bool il, cudaStream_t stream) {
  if (dim == 128) return il ? launch<T, 128, true>(a, stream) : launch<T, 128, false>(a, stream);
  return il ? launch<T, 64, true>(a, stream) : launch<T, 64, false>(a, stream);
}

}  // namespace

extern "C" oscar_status_t oscar_rope(const oscar_dims_t* dims, const oscar_rope_t* rope, int32_t type, int64_t num_tokens,
                                     const int32_t* positions, const void* q, int64_t q_stride, const void* k,
                                     int64_t k_stride, void* q_out, int64_t q_out_stride, void* k_out,
                                     int64_t k_out_stride, void* stream) {
  oscar_status_t st = check_dims(dims);
  if (st != OSCAR_OK) return st;
  st = check_rope(rope, dims);
  if (st != OSCAR_OK) return st;
  if (type != OSCAR_TYPE_BF16 && type != OSCAR_TYPE_FP16 && type != OSCAR_TYPE_FP32) return OSCAR_ERR_INVALID_ARG;
  if (num_tokens < 0 || num_tokens > 0x7fffffffLL) return OSCAR_ERR_INVALID_ARG;
  if (num_tokens == 0) return OSCAR_OK;
  if (!positions || (!q && !k) || !q != !q_out || !k != !k_out) return OSCAR_ERR_INVALID_ARG;
  const int elem = type == OSCAR_TYPE_FP32 ? 4 : 2;
  const RopeArgs a{{rope->turns, rope->rotary_dim, rope->magnitude},
                   positions,
                   {q, q_out, q_stride, q_out_stride, q ? dims->num_q_heads : 0},
                   {k, k_out, k_stride, k_out_stride, k ? dims->num_kv_heads : 0},
                   num_tokens};
  for (const Rows* r : {&a.q, &a.k}) {
    if (r->heads > 0 && (misaligned16(r->in) || misaligned16(r->out) || bad_stride(r->in_stride, r->heads, dims->head_dim, elem) ||
                         bad_stride(r->out_stride, r->heads, dims->head_dim, elem) ||
                         bad_in_place(r->in, r->in_stride, r->out, r->out_stride, num_tokens)))
      return OSCAR_ERR_INVALID_ARG;
  }
  const bool il = rope->interleaved != 0;
  cudaStream_t s = as_stream(stream);
  const cudaError_t e = type == OSCAR_TYPE_BF16   ? launch_type<__nv_bfloat16>(a, dims->head_dim, il, s)
                        : type == OSCAR_TYPE_FP16 ? launch_type<__half>(a, dims->head_dim, il, s)
                                                  : launch_type<float>(a, dims->head_dim, il, s);
  return e == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

extern "C" oscar_status_t oscar_rope_turns(int32_t rotary_dim, double base, const oscar_rope_scaling_t* scaling,
                                           uint64_t* turns, float* magnitude) {
  const double kPi = 3.14159265358979323846;
  // 1 / (2 pi), as a double and what it lacks: the fraction of a turn keeps more bits than a double has
  const double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
  const double kMostRadians = 1e6;  // per position (1 is usual): more has no use, and would leave the integers below
  if (!turns || !magnitude || rotary_dim <= 0 || !(base > 1.0) || !isfinite(base)) return OSCAR_ERR_INVALID_ARG;
  if (rotary_dim % 16 != 0 || rotary_dim > 128) return OSCAR_ERR_UNSUPPORTED;
  const int n = rotary_dim / 2;
  const int kind = scaling ? scaling->kind : OSCAR_ROPE_PLAIN;
  const double factor = scaling ? scaling->factor : 1.0, length = scaling ? scaling->original_max_position : 0;
  const double low = scaling ? scaling->low : 0.0, high = scaling ? scaling->high : 0.0;
  if (kind < OSCAR_ROPE_PLAIN || kind > OSCAR_ROPE_DIVISORS) return OSCAR_ERR_INVALID_ARG;
  if (kind != OSCAR_ROPE_PLAIN && kind != OSCAR_ROPE_DIVISORS && !(factor > 0.0 && isfinite(factor)))
    return OSCAR_ERR_INVALID_ARG;
  if ((kind == OSCAR_ROPE_YARN || kind == OSCAR_ROPE_BANDS) && !(length > 0 && low > 0.0 && high > low && isfinite(high)))
    return OSCAR_ERR_INVALID_ARG;
  if (kind == OSCAR_ROPE_DIVISORS) {
    if (!scaling->divisors) return OSCAR_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
      if (!(scaling->divisors[i] > 0.0 && isfinite(scaling->divisors[i]))) return OSCAR_ERR_INVALID_ARG;
  }
  if (kind == OSCAR_ROPE_NTK) base *= pow(factor, static_cast<double>(rotary_dim) / (rotary_dim - 2));
  if (!(base > 1.0) || !isfinite(base)) return OSCAR_ERR_INVALID_ARG;
  // the pair that turns `times` times within the original length
  auto pair_of = [&](double times) { return rotary_dim * log(length / (times * 2 * kPi)) / (2 * log(base)); };
  double from = 0.0, to = 0.0;
  if (kind == OSCAR_ROPE_YARN) {
    from = fmax(floor(pair_of(high)), 0.0);
    to = fmin(ceil(pair_of(low)), rotary_dim - 1.0);
    if (to < from + 0.001) to = from + 0.001;
  }
  for (int i = 0; i < n; ++i) {
    const double x = -2.0 * i / rotary_dim;
    double f = pow(base, x);
    const double lacks = fma(-x, rotary_dim, -2.0 * i) / rotary_dim * log(base);  // relative, from the exponent's rounding
    if (kind == OSCAR_ROPE_LINEAR) {
      f /= factor;
    } else if (kind == OSCAR_ROPE_DIVISORS) {
      f /= scaling->divisors[i];
    } else if (kind == OSCAR_ROPE_YARN) {
      const double slow = fmin(fmax((i - from) / (to - from), 0.0), 1.0);
      f = f / factor * slow + f * (1.0 - slow);
    } else if (kind == OSCAR_ROPE_BANDS) {
      const double fast = fmin(fmax((length * f / (2 * kPi) - low) / (high - low), 0.0), 1.0);
      f = f * fast + f / factor * (1.0 - fast);
    }
    if (!(f <= kMostRadians)) return OSCAR_ERR_INVALID_ARG;
    // f / (2 pi) modulo 1, in units of 2^-64
    const double p = f * kHi, rest = fma(f, kHi, -p) + f * kLo + p * lacks, frac = p - floor(p);
    turns[i] = static_cast<uint64_t>(ldexp(frac, 64)) + static_cast<uint64_t>(static_cast<int64_t>(ldexp(rest, 64)));
  }
  *magnitude = kind == OSCAR_ROPE_YARN && factor > 1.0 ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.0f;
  return OSCAR_OK;
}
