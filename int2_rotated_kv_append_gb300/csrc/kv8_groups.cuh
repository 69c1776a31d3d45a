// Groups of sequences whose first pages are the same (oscar_kv8_decode_shared): the lists, as its kernels read them.
#pragma once

#include "kv8_attn.cuh"

namespace oscar {
namespace kv8 {

struct Groups {
  const int32_t* members;      // [num_members] sequences, group after group
  const int32_t* start;        // [num_groups + 1]
  const int32_t* prefix_lens;  // [num_groups]
  int num_members, num_groups, max_prefix;
};

// Of group g: first member, members, tokens of the prefix that are attended together (whole pages).  False: bad numbers.
__device__ __forceinline__ bool group_of(const Groups& s, int g, int& start, int& n, int& prefix) {
  start = __ldg(s.start + g);
  const int end = __ldg(s.start + g + 1);
  n = end - start;
  prefix = min(max(__ldg(s.prefix_lens + g), 0), s.max_prefix) / kPageSize * kPageSize;
  return start >= 0 && n >= 0 && end <= s.num_members && (g > 0 || start == 0);
}

// A member's sequence, in range: one that is not is flagged, and left without a result, where members' own parts are attended.
__device__ __forceinline__ int in_batch(int b, int batch) { return min(max(b, 0), batch - 1); }

// One warp: the prefix of member i's group; kBadLists, or kNoGroup where i is behind the last group's members.
constexpr int kBadLists = -1, kNoGroup = -2;
__device__ __forceinline__ int prefix_of_member(const Groups& s, int i, int lane) {
  int got = kNoGroup;
  for (int g0 = 0; g0 < s.num_groups; g0 += 32) {
    int start = 0, n = 0, prefix = 0;
    const bool fine = g0 + lane >= s.num_groups || group_of(s, g0 + lane, start, n, prefix);
    if (__any_sync(0xffffffffu, !fine)) return kBadLists;
    const uint32_t mine = __ballot_sync(0xffffffffu, i >= start && i < start + n);
    if (mine != 0) got = __shfl_sync(0xffffffffu, prefix, __ffs(mine) - 1);  // (the rest of the list is looked at as well)
  }
  return got;
}

}  // namespace kv8
}  // namespace oscar
