// Rotary positions: the rotation of a pair of channels by position * frequency, shared by oscar_rope and the append that
// rotates on the way.
//
// A frequency is held as a 64-bit fraction of a turn.  Its product with a position, modulo 2^64, is the angle modulo one
// turn, exact for the fraction that is held, so far positions are as good as near ones and no table over positions is read.  (The
// fraction itself comes from a power in double, up to 2^-52 of the frequency off: 2^-24 of a turn for the fastest pairs at position 2^31.)
// The nearest quarter turn is taken off in whole numbers; what is left, within an eighth of a turn, becomes fp32 from all 64 bits, so
// that cosine and sine are good to 2^-22 of themselves, the sines of slow pairs' first positions too.
#pragma once

#include <math.h>

#include "common.cuh"

namespace oscar {
namespace rope {

struct Rope {
  const uint64_t* turns;  // [rotary / 2]
  int rotary;
  float magnitude;
};

static inline oscar_status_t check_rope(const oscar_rope_t* r, const oscar_dims_t* d) {
  if (r == nullptr || r->turns == nullptr || (reinterpret_cast<uintptr_t>(r->turns) & 7u) != 0) return OSCAR_ERR_INVALID_ARG;
  if (r->rotary_dim <= 0 || r->rotary_dim > d->head_dim || (r->interleaved != 0 && r->interleaved != 1) ||
      !isfinite(r->magnitude))
    return OSCAR_ERR_INVALID_ARG;
  if (static_cast<int64_t>(d->num_q_heads) * d->head_dim > 0x7fffffffLL) return OSCAR_ERR_UNSUPPORTED;  // (a row's channels)
  return r->rotary_dim % 16 != 0 ? OSCAR_ERR_UNSUPPORTED : OSCAR_OK;
}

// Whether rows of `heads` heads with this many elements from one to the next can be read 16 bytes at a time.
static inline bool bad_stride(int64_t stride, int heads, int dim, int elem) {
  return stride < static_cast<int64_t>(heads) * dim || stride * elem % 16 != 0;
}

// Rows that go over rows still to be read.
static inline bool bad_in_place(const void* in, int64_t in_stride, const void* out, int64_t out_stride, int64_t rows) {
  return in == out && in_stride != out_stride && rows > 1;
}

// (cos, sin) of pos * frequency, times magnitude.
__device__ __forceinline__ float2 cos_sin(uint64_t turns, int pos, float magnitude) {
  const uint64_t whole = turns * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const uint64_t quarter = (whole + (1ull << 61)) >> 62;
  float s, c;
  sincospif(static_cast<float>(static_cast<int64_t>(whole - (quarter << 62))) * 0x1p-63f, &s, &c);
  const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;  // |cos|, |sin| of the whole angle, up to their signs
  const bool neg_x = quarter == 1 || quarter == 2, neg_y = quarter >= 2;
  return make_float2((neg_x ? -x : x) * magnitude, (neg_y ? -y : y) * magnitude);
}

// The pair (a, b) turned by (cos, sin).
__device__ __forceinline__ void turn(float& a, float& b, float2 cs) {
  const float x = fmaf(a, cs.x, -(b * cs.y)), y = fmaf(b, cs.x, a * cs.y);
  a = x;
  b = y;
}

// A row of D channels is worked on in units of 2 x E channels, two vectors each: the vectors of a half-layout unit hold the
// first and the second channels of E pairs, an interleaved unit's two vectors are neighbours and hold E whole pairs.
// Behind the rotated channels units are two neighbouring vectors in either layout.
template <int E, bool IL>
__device__ __forceinline__ int first_channel(int unit, int rotary) {
  return IL || unit * 2 * E >= rotary ? unit * 2 * E : unit * E;
}
template <int E, bool IL>
__device__ __forceinline__ int second_channel(int unit, int rotary) {
  return IL || unit * 2 * E >= rotary ? unit * 2 * E + E : rotary / 2 + unit * E;
}

// x[0 .. E) and x[E .. 2 E), the two vectors of a rotated unit; cs(j): the unit's pair j.
template <int E, bool IL, typename Cs>
__device__ __forceinline__ void turn_unit(float (&x)[2 * E], Cs cs) {
#pragma unroll
  for (int j = 0; j < E; ++j) {
    if (IL) turn(x[2 * j], x[2 * j + 1], cs(j));
    else turn(x[j], x[E + j], cs(j));
  }
}

}  // namespace rope
}  // namespace oscar
