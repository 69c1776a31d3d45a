// Operations on the pages of a paged cache: copy, reserve, fork, free, trim, compact, and groups of sequences that share pages.
//
// A page's reference count is the allocator's whole state (0 = free), and free pages are taken
// lowest id first in the order of the requests: ranks by prefix sums, no atomics whose order
// matters.  Each operation is a planning kernel over counts and lengths and, where bytes move,
// a second kernel that copies pages and table rows, launched as its programmatic dependent.
// Planning is latency (a few dependent passes over 4 bytes per page: a token more for each of 64 sequences 3.4 us, a
// trim 2.3, a fork of 24 sequences 11 with the free before it); the copies are bound by 2 x page bytes (11.5 thousand
// pages of 32 KB moved: 124 us, 6.1 TB/s, 90% of a plain copy's rate).
#include "kv8.cuh"

namespace {

using namespace oscar;

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kChunk = 4 * kPlanThreads;  // counts per block pass: one int4 a thread

struct Pools {
  uint8_t* base[OSCAR_MAX_POOLS];
  long long bytes[OSCAR_MAX_POOLS];
  int n;
};

struct Tables {
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
  int batch, num_pages, max_pages;
};

__device__ __forceinline__ bool length_ok(const Tables& t, int L) { return L >= 0 && L <= t.max_pages * kPageSize; }
__device__ __forceinline__ int pages_of(int L) { return (L + kPageSize - 1) / kPageSize; }

// Exclusive prefix sum of v over the block's kPlanThreads threads; *total receives the sum.
// `part` is shared memory of kPlanWarps values.  Two barriers.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* part, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // part may still be read from the call before
  if (lane == 31) part[warp] = x;
  __syncthreads();
  T p = part[lane];  // kPlanWarps == 32
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, p, o);
    if (lane >= o) p += y;
  }
  *total = __shfl_sync(0xffffffffu, p, 31);
  const T before = __shfl_sync(0xffffffffu, p, (warp + 31) & 31);
  return x - v + (warp > 0 ? before : 0);
}

// The lowest free pages, at most `want` of them, into list[0 ..); returns how many there are.
__device__ int find_free(const int32_t* refs, int num_pages, int want, int32_t* list, int* part) {
  int found = 0;
  for (int c = 0; c < num_pages && found < want; c += kChunk) {
    const int i0 = c + threadIdx.x * 4;
    int f = 0;
    if (i0 + 3 < num_pages) {
      const int4 r = *reinterpret_cast<const int4*>(refs + i0);
      f = (r.x == 0) | (r.y == 0) << 1 | (r.z == 0) << 2 | (r.w == 0) << 3;
    } else {
      for (int e = 0; e < 4; ++e)
        if (i0 + e < num_pages && refs[i0 + e] == 0) f |= 1 << e;
    }
    int total;
    int at = found + block_scan(__popc(f), part, &total);
    for (int e = 0; e < 4; ++e)
      if (f >> e & 1) {
        if (at < want) list[at] = i0 + e;
        ++at;
      }
    found += total;
  }
  __syncthreads();
  return min(found, want);
}

// ---- copy --------------------------------------------------------------------------------

// Bytes [part/parts] of a page, by the threads of a block.
template <typename V>
__device__ __forceinline__ void copy_bytes(uint8_t* dst, const uint8_t* src, long long bytes, int part, int parts) {
  const long long n = bytes / static_cast<long long>(sizeof(V));
  const V* s = reinterpret_cast<const V*>(src);
  V* d = reinterpret_cast<V*>(dst);
  const long long step = static_cast<long long>(parts) * blockDim.x;
  long long i = static_cast<long long>(part) * blockDim.x + threadIdx.x;
  for (; i + 3 * step < n; i += 4 * step) {  // four loads in flight a thread
    const V a = s[i], b = s[i + step], c = s[i + 2 * step], e = s[i + 3 * step];
    d[i] = a;
    d[i + step] = b;
    d[i + 2 * step] = c;
    d[i + 3 * step] = e;
  }
  for (; i < n; i += step) d[i] = s[i];
}

__device__ __forceinline__ void copy_page(const Pools& pools, int src, int dst, int part, int parts) {
  for (int k = 0; k < pools.n; ++k) {
    const long long bytes = pools.bytes[k];
    const uint8_t* s = pools.base[k] + bytes * src;
    uint8_t* d = pools.base[k] + bytes * dst;
    if (bytes % 16 == 0) copy_bytes<uint4>(d, s, bytes, part, parts);
    else copy_bytes<uint32_t>(d, s, bytes, part, parts);
  }
}

__global__ void __launch_bounds__(256) copy_kernel(Pools pools, const int32_t* src, const int32_t* dst, int num_pages) {
  const int s = src[blockIdx.x], d = dst[blockIdx.x];
  if (s < 0 || d < 0) return;
  if (s >= num_pages || d >= num_pages) {
    if (threadIdx.x == 0) record_error(OSCAR_DEVERR_PAGE_ID);
    return;
  }
  if (s != d) copy_page(pools, s, d, blockIdx.y, gridDim.y);
}

// ---- free, trim ----------------------------------------------------------------------------

// Takes the page of a table entry out of the table and drops one reference to it.
__device__ __forceinline__ void release(const Tables& t, int32_t* entry) {
  if (*entry < 0) return;
  const int id = atomicExch(entry, -1);  // of two that release it, one finds the page
  if (id < 0) return;
  if (id >= t.num_pages) {
    record_error(OSCAR_DEVERR_PAGE_ID);
    return;
  }
  if (atomicSub(t.refs + id, 1) <= 0) {  // it was free already
    atomicAdd(t.refs + id, 1);
    record_error(OSCAR_DEVERR_PAGE_ID);
  }
}

__global__ void __launch_bounds__(512) free_kernel(Tables t, const int32_t* seqs) {
  const int s = seqs[blockIdx.x];
  if (s < 0 || s >= t.batch) {
    if (threadIdx.x == 0) record_error(OSCAR_DEVERR_POSITION);
    return;
  }
  const int L = t.lens[s];
  __syncthreads();
  if (!length_ok(t, L)) {
    if (threadIdx.x == 0) record_error(OSCAR_DEVERR_POSITION);
    return;
  }
  int32_t* row = t.table + static_cast<size_t>(s) * t.max_pages;
  for (int j = threadIdx.x; j < pages_of(L); j += blockDim.x) release(t, row + j);
  if (threadIdx.x == 0) t.lens[s] = 0;
}

__global__ void __launch_bounds__(256) trim_kernel(Tables t, int sink, int window) {
  const int b = blockIdx.y;
  const int L = t.lens[b];
  if (!length_ok(t, L)) {
    if (threadIdx.x == 0 && blockIdx.x == 0) record_error(OSCAR_DEVERR_POSITION);
    return;
  }
  const int lo = sink / kPageSize + (sink % kPageSize != 0), hi = L > window ? (L - window) / kPageSize : 0;
  int32_t* row = t.table + static_cast<size_t>(b) * t.max_pages;
  const int step = gridDim.x * blockDim.x;
  for (long long j = static_cast<long long>(lo) + blockIdx.x * blockDim.x + threadIdx.x; j < hi; j += step)
    release(t, row + j);
}

// ---- reserve ---------------------------------------------------------------------------------

__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(Tables t, const int32_t* new_tokens, int32_t* granted,
                                                               int32_t* free_list, int32_t* first) {
  __shared__ int part[kPlanWarps];
  __shared__ long long part64[kPlanWarps];
  // pages asked for: first[b] = those of the sequences before b, at most num_pages (beyond every
  // page: refused).  64 bits: 1024 requests of up to 2^27 pages.
  long long total = 0;
  for (int b0 = 0; b0 < t.batch; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    long long need = 0;
    if (b < t.batch) {
      const int L = t.lens[b], n = new_tokens[b];
      if (!length_ok(t, L) || n < 0 || n > t.max_pages * kPageSize - L) record_error(OSCAR_DEVERR_POSITION);
      else need = pages_of(L + n) - pages_of(L);
    }
    long long sum;
    const long long at = total + block_scan(need, part64, &sum);
    if (b < t.batch) first[b] = static_cast<int32_t>(min(at, static_cast<long long>(t.num_pages)));
    total += sum;
  }
  __syncthreads();
  const int want = static_cast<int>(min(total, static_cast<long long>(t.num_pages)));
  const int have = want > 0 ? find_free(t.refs, t.num_pages, want, free_list, part) : 0;
  __syncthreads();
  // one warp per sequence
  const int lane = threadIdx.x & 31;
  for (int b = threadIdx.x >> 5; b < t.batch; b += kPlanWarps) {
    const int L = t.lens[b], n = new_tokens[b];
    bool ok = length_ok(t, L) && n >= 0 && n <= t.max_pages * kPageSize - L;
    if (ok) {
      const int j0 = pages_of(L), need = pages_of(L + n) - j0, f = first[b];
      if (need > have - f) {
        ok = need == 0;
        if (!ok && lane == 0) record_error(OSCAR_DEVERR_NO_PAGES);
      }
      if (ok) {
        for (int i = lane; i < need; i += 32) {
          const int id = free_list[f + i];
          t.table[static_cast<size_t>(b) * t.max_pages + j0 + i] = id;
          t.refs[id] = 1;
        }
        __syncwarp();
        if (lane == 0) t.lens[b] = L + n;
      }
    }
    if (lane == 0 && granted != nullptr) granted[b] = ok;
  }
}

// ---- fork ------------------------------------------------------------------------------------

// What fork i does: the length, and the free page that takes the partial last one (-1: none).
struct ForkPlan {
  int32_t len;  // -1: refused
  int32_t page;
};

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(Tables t, const int32_t* src, const int32_t* dst,
                                                                 int n, int32_t* granted, int32_t* claim,
                                                                 int32_t* free_list, ForkPlan* plan) {
  __shared__ int part[kPlanWarps];
  for (int b = threadIdx.x; b < t.batch; b += kPlanThreads) claim[b] = 0x7fffffff;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads)
    if (dst[i] >= 0 && dst[i] < t.batch) atomicMin(claim + dst[i], i);  // the lowest fork of a dst counts
  __syncthreads();
  int total = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    int L = -1, need = 0;
    if (i < n) {
      const int s = src[i], d = dst[i];
      if (s >= 0 && s < t.batch && d >= 0 && d < t.batch && s != d && claim[d] == i && t.lens[d] == 0 &&
          length_ok(t, t.lens[s])) {
        L = t.lens[s];
        if (L % kPageSize != 0) {
          const int id = t.table[static_cast<size_t>(s) * t.max_pages + L / kPageSize];
          if (id >= t.num_pages) record_error(OSCAR_DEVERR_PAGE_ID);
          need = id >= 0 && id < t.num_pages;
        }
      } else {
        record_error(OSCAR_DEVERR_POSITION);
      }
    }
    int sum;
    const int at = total + block_scan(need, part, &sum);
    if (i < n) plan[i] = ForkPlan{L, need ? at : -1};
    total += sum;
  }
  __syncthreads();
  const int have = total > 0 ? find_free(t.refs, t.num_pages, min(total, t.num_pages), free_list, part) : 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    ForkPlan p = plan[i];
    if (p.page >= have) {
      record_error(OSCAR_DEVERR_NO_PAGES);
      p = ForkPlan{-1, -1};
    } else if (p.page >= 0) {
      p.page = free_list[p.page];
      t.refs[p.page] = 1;
    }
    plan[i] = p;
    if (granted != nullptr) granted[i] = p.len >= 0;
    if (p.len >= 0) t.lens[dst[i]] = p.len;  // every length was read above
  }
}

// Grid (forks, parts): each part takes a share of the table row and of the copied page.
__global__ void __launch_bounds__(256) fork_apply_kernel(Tables t, Pools pools, const int32_t* src, const int32_t* dst,
                                                         const ForkPlan* plan) {
  grid_dep_wait();
  const ForkPlan p = plan[blockIdx.x];
  if (p.len <= 0) return;
  const int32_t* from = t.table + static_cast<size_t>(src[blockIdx.x]) * t.max_pages;
  int32_t* to = t.table + static_cast<size_t>(dst[blockIdx.x]) * t.max_pages;
  const int full = p.len / kPageSize, last = p.len % kPageSize;
  for (int j = blockIdx.y * blockDim.x + threadIdx.x; j < full; j += gridDim.y * blockDim.x) {
    const int id = from[j];
    if (id >= 0 && id < t.num_pages) atomicAdd(t.refs + id, 1);
    else if (id >= 0) record_error(OSCAR_DEVERR_PAGE_ID);
    to[j] = id < t.num_pages ? id : -1;
  }
  if (last != 0) {
    if (blockIdx.y == 0 && threadIdx.x == 0) to[full] = p.page;
    if (p.page >= 0) copy_page(pools, from[full], p.page, blockIdx.y, gridDim.y);
  }
}

// ---- compact ---------------------------------------------------------------------------------

// Which of the four pages from i0 on are in use.
__device__ __forceinline__ int used_mask(const int32_t* refs, int i0, int num_pages) {
  int f = 0;
  if (i0 + 3 < num_pages) {
    const int4 r = *reinterpret_cast<const int4*>(refs + i0);
    f = (r.x > 0) | (r.y > 0) << 1 | (r.z > 0) << 2 | (r.w > 0) << 3;
  } else {
    for (int e = 0; e < 4; ++e)
      if (i0 + e < num_pages && refs[i0 + e] > 0) f |= 1 << e;
  }
  return f;
}

// Pools of up to kOwnChunks chunks: every planning block counts them all itself; with more, a counting kernel before it is
// quicker (nothing to move, one against two kernels: 2 chunks 5.9 and 6.9 us, 4: 7.5 and 8.3, 6: 8.6 and 9.0, 8: 10.0 and 9.7,
// 13: 13.0 and 11.5).
constexpr int kOwnChunks = 6;

// Pages in use per chunk of kChunk counts.
__global__ void __launch_bounds__(kPlanThreads) compact_count_kernel(const int32_t* refs, int num_pages,
                                                                     int32_t* counts) {
  const int f = used_mask(refs, blockIdx.x * kChunk + threadIdx.x * 4, num_pages);
  __shared__ int part[kPlanWarps];
  int total;
  block_scan(__popc(f), part, &total);
  if (threadIdx.x == 0) counts[blockIdx.x] = total;
}

// info[0] = pages in use, info[1] = pages that move.  from[r] / to[r]: the r-th used page with id >= used,
// the r-th free id below it; rank[id] = r for the pages that move.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const int32_t* refs, int num_pages,
                                                                    const int32_t* counts, int chunks, int32_t* from,
                                                                    int32_t* to, int32_t* rank, int32_t* info,
                                                                    int32_t* num_used) {
  grid_dep_wait();
  __shared__ int part[kPlanWarps];
  __shared__ int own[kOwnChunks];
  if (counts == nullptr) {
    if (threadIdx.x < kOwnChunks) own[threadIdx.x] = 0;
    __syncthreads();
    for (int c = 0; c < chunks; ++c) {
      const int n = __reduce_add_sync(0xffffffffu, __popc(used_mask(refs, c * kChunk + threadIdx.x * 4, num_pages)));
      if ((threadIdx.x & 31) == 0) atomicAdd(own + c, n);
    }
    __syncthreads();
    counts = own;
  }
  // used pages in all chunks, and in those before this one
  int all = 0, before = 0;
  for (int c0 = 0; c0 < chunks; c0 += kPlanThreads) {
    const int c = c0 + threadIdx.x;
    const int v = c < chunks ? counts[c] : 0;
    int s;
    block_scan(v, part, &s);
    all += s;
    block_scan(c < static_cast<int>(blockIdx.x) ? v : 0, part, &s);
    before += s;
  }
  const int i0 = blockIdx.x * kChunk + threadIdx.x * 4;
  const int f = used_mask(refs, i0, num_pages);
  int total;
  int used = before + block_scan(__popc(f), part, &total);  // used pages with a lower id than i0
  // used pages below id `all`: the chunk that holds it is counted again
  const int border = all / kChunk;
  int low = 0;
  for (int c0 = 0; c0 < border; c0 += kPlanThreads) {
    const int c = c0 + threadIdx.x;
    int s;
    block_scan(c < border ? counts[c] : 0, part, &s);
    low += s;
  }
  const int e0 = border * kChunk + threadIdx.x * 4;
  int g = used_mask(refs, e0, num_pages);
  if (e0 + 3 >= all) g &= all > e0 ? (1 << (all - e0)) - 1 : 0;
  block_scan(__popc(g), part, &total);
  low += total;
  for (int e = 0; e < 4; ++e) {
    const int id = i0 + e;
    if (id >= num_pages) break;
    const bool u = f >> e & 1;
    if (u && id >= all) {
      from[used - low] = id;
      rank[id] = used - low;
    }
    if (!u && id < all) to[id - used] = id;
    used += u;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    info[0] = all;
    info[1] = all - low;
    if (num_used != nullptr) *num_used = all;
  }
}

// The first `rows` blocks rewrite a row of the page table each; the others move pages.
__global__ void __launch_bounds__(256) compact_apply_kernel(Tables t, Pools pools, const int32_t* from,
                                                            const int32_t* to, const int32_t* rank,
                                                            const int32_t* info) {
  grid_dep_wait();
  const int used = info[0], moves = info[1];
  if (static_cast<int>(blockIdx.x) < t.batch) {
    const int L = t.lens[blockIdx.x];
    if (!length_ok(t, L)) {
      if (threadIdx.x == 0) record_error(OSCAR_DEVERR_POSITION);
      return;
    }
    int32_t* row = t.table + static_cast<size_t>(blockIdx.x) * t.max_pages;
    for (int j = threadIdx.x; j < pages_of(L); j += blockDim.x) {
      const int id = row[j];
      if (id < used) continue;
      if (id >= t.num_pages) {
        record_error(OSCAR_DEVERR_PAGE_ID);
        continue;
      }
      const int r = rank[id];
      if (r >= 0 && r < moves && from[r] == id) row[j] = to[r];
      else record_error(OSCAR_DEVERR_PAGE_ID);  // an entry whose page is free
    }
    return;
  }
  const int mover = blockIdx.x - t.batch, movers = gridDim.x - t.batch;
  for (int r = mover; r < moves; r += movers) {
    const int s = from[r], d = to[r];
    copy_page(pools, s, d, 0, 1);
    if (threadIdx.x == 0) {
      t.refs[d] = t.refs[s];
      t.refs[s] = 0;
    }
  }
}

// ---- host ------------------------------------------------------------------------------------

struct Layout {
  size_t claim, first, free_list, plan, counts, from, to, rank, info, total;
};

Layout layout(const oscar_dims_t* d, int batch, int forks) {
  Layout l{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align_up(bytes, 256);
    return at;
  };
  const size_t pages = static_cast<size_t>(d->num_pages) * 4;
  l.claim = take(static_cast<size_t>(batch) * 4);
  l.first = l.claim;
  l.free_list = take(pages);
  l.plan = take(static_cast<size_t>(forks) * sizeof(ForkPlan));
  l.counts = take((static_cast<size_t>(d->num_pages) + kChunk - 1) / kChunk * 4);
  l.from = l.free_list;
  l.to = take(pages);
  l.rank = take(pages);
  l.info = take(8);
  l.total = off;
  return l;
}

oscar_status_t check_pages(const oscar_dims_t* d, int batch, int num_pools, const oscar_page_pool_t* pools) {
  if (d == nullptr || d->num_pages <= 0 || d->max_pages_per_seq <= 0) return OSCAR_ERR_INVALID_ARG;
  if (d->page_size != kPageSize) return d->page_size <= 0 ? OSCAR_ERR_INVALID_ARG : OSCAR_ERR_UNSUPPORTED;
  if (batch < 0 || num_pools < 0 || num_pools > OSCAR_MAX_POOLS || (num_pools > 0 && pools == nullptr))
    return OSCAR_ERR_INVALID_ARG;
  for (int i = 0; i < num_pools; ++i)
    if (pools[i].base == nullptr || misaligned16(pools[i].base) || pools[i].page_bytes <= 0 ||
        pools[i].page_bytes % 4 != 0)
      return OSCAR_ERR_INVALID_ARG;
  if (d->num_pages > 0x7fffffff - 2 * kChunk || d->max_pages_per_seq > 0x7fffffff / kPageSize || batch > 65535)
    return OSCAR_ERR_UNSUPPORTED;
  return OSCAR_OK;
}

oscar_status_t check_workspace(const oscar_dims_t* d, int batch, int forks, const void* ws, size_t bytes) {
  if (ws == nullptr || reinterpret_cast<uintptr_t>(ws) % 256 != 0) return OSCAR_ERR_INVALID_ARG;
  return bytes < layout(d, batch, forks).total ? OSCAR_ERR_WORKSPACE : OSCAR_OK;
}

Pools make_pools(int n, const oscar_page_pool_t* pools) {
  Pools p{};
  p.n = n;
  for (int i = 0; i < n; ++i) {
    p.base[i] = static_cast<uint8_t*>(pools[i].base);
    p.bytes[i] = pools[i].page_bytes;
  }
  return p;
}

// Blocks of 256 threads that share one page: one per 16 KB.
int page_parts(const Pools& p) {
  long long bytes = 0;
  for (int i = 0; i < p.n; ++i) bytes += p.bytes[i];
  const long long parts = (bytes + 16383) / 16384;
  return static_cast<int>(parts < 1 ? 1 : parts > 64 ? 64 : parts);
}

oscar_status_t launched() { return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA; }

// ---- groups of sequences with the same first pages ------------------------------------------

constexpr int kNoMatch = 0x7fffffff;

// One block per sequence b: the lowest sequence whose first k pages are b's (b itself where there is none lower), and how many
// leading pages the two have in common.  A sequence with fewer than k full pages is its own.
__global__ void __launch_bounds__(256) groups_find_kernel(Tables t, int k, int32_t* leader, int32_t* depth) {
  __shared__ int found, differs;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  auto full_pages = [&](int a) {
    const int L = __ldg(t.lens + a);
    return length_ok(t, L) ? L / kPageSize : 0;
  };
  auto row = [&](int a) { return t.table + static_cast<size_t>(a) * t.max_pages; };
  const int full = full_pages(b);
  if (tid == 0 && !length_ok(t, __ldg(t.lens + b))) record_error(OSCAR_DEVERR_POSITION);
  const int32_t* mine = row(b);
  const int last = full >= k ? __ldg(mine + k - 1) : -1;
  if (tid == 0) found = differs = kNoMatch;
  __syncthreads();
  for (int a0 = 0; a0 < b && last >= 0; a0 += blockDim.x) {
    const int a = a0 + tid;
    bool hit = false;
    uint32_t maybe = __ballot_sync(0xffffffffu, a < b && full_pages(min(a, b)) >= k && __ldg(row(min(a, b)) + k - 1) == last);
    for (; maybe != 0; maybe &= maybe - 1) {  // a warp looks at its own, lowest first
      const int c = a - lane + __ffs(maybe) - 1;
      bool same = true;
      for (int j = lane; j < k && same; j += 32) {
        const int p = __ldg(mine + j);
        same = p >= 0 && p == __ldg(row(c) + j);
      }
      if (__all_sync(0xffffffffu, same)) {
        if (lane == 0) atomicMin(&found, c);
        hit = true;
        break;
      }
    }
    if (__syncthreads_or(hit)) break;
  }
  const int lead = found == kNoMatch ? b : found;
  if (tid == 0) leader[b] = lead;
  if (lead == b) {
    if (tid == 0) depth[b] = full;
    return;
  }
  const int32_t* theirs = row(lead);
  const int most = min(full, full_pages(lead));
  constexpr int kEach = 4;
  for (int j0 = k; j0 < most; j0 += kEach * 256) {
    int x[kEach], y[kEach], at = kNoMatch;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int j = min(j0 + e * 256 + tid, most - 1);
      x[e] = __ldg(mine + j);
      y[e] = __ldg(theirs + j);
    }
#pragma unroll
    for (int e = kEach - 1; e >= 0; --e)
      if (j0 + e * 256 + tid < most && (x[e] != y[e] || x[e] < 0)) at = j0 + e * 256 + tid;
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0 && at != kNoMatch) atomicMin(&differs, at);
    if (__syncthreads_or(at != kNoMatch)) break;
  }
  if (tid == 0) depth[b] = min(differs, most);
}

// One block: numbers the groups of two members or more in the order of their leaders, `room` - 1 of them at most, and lists
// their members; then all other sequences as one group without a prefix.
constexpr int kLeadersHere = 4096;
__global__ void __launch_bounds__(kPlanThreads) groups_list_kernel(int batch, int room, const int32_t* leaders, const int32_t* depth,
                                                                   int32_t* kind, int32_t* heads, int32_t* members,
                                                                   int32_t* start, int32_t* prefix) {
  __shared__ int part[kPlanWarps];
  __shared__ int32_t here[kLeadersHere];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_wait();
  for (int b = tid; b < batch; b += kPlanThreads) {
    if (batch <= kLeadersHere) here[b] = leaders[b];
    kind[b] = 0;
  }
  const int32_t* leader = batch <= kLeadersHere ? here : leaders;
  __syncthreads();
  for (int b = tid; b < batch; b += kPlanThreads)
    if (leader[b] != b) kind[leader[b]] = 1;  // leads others
  __syncthreads();
  int count = 0;
  for (int b0 = 0; b0 < batch; b0 += kPlanThreads) {
    const int b = b0 + tid;
    const int leads = b < batch && kind[b] == 1;
    int sum;
    const int rank = count + block_scan(leads, part, &sum);
    if (leads && rank < room - 1) {
      heads[rank] = b;
      kind[b] = 2;  // leads a group that is listed
    }
    count += sum;
  }
  count = min(count, room - 1);
  __syncthreads();
  // a warp per group: members, and the pages that all of them share
  for (int g = warp; g < count; g += kPlanWarps) {
    const int head = heads[g];
    int n = 0, least = kNoMatch;
    for (int b0 = head & ~31; b0 < batch; b0 += 32) {
      const int b = b0 + lane;
      const bool in = b < batch && leader[min(b, batch - 1)] == head;
      if (in) least = min(least, depth[b]);
      n += __popc(__ballot_sync(0xffffffffu, in));
    }
    least = __reduce_min_sync(0xffffffffu, least);
    if (lane == 0) {
      start[g + 1] = n;
      prefix[g] = least * kPageSize;
    }
  }
  __syncthreads();
  int before = 0;
  for (int g0 = 0; g0 < room; g0 += kPlanThreads) {
    const int g = g0 + tid;
    int sum;
    const int n = g < count ? start[g + 1] : 0;
    const int at = before + block_scan(n, part, &sum) + n;
    if (g < room) {
      start[g + 1] = g < count ? at : batch;
      if (g >= count) prefix[g] = 0;
    }
    before += sum;
  }
  if (tid == 0) start[0] = 0;
  __syncthreads();
  for (int g = warp; g < count; g += kPlanWarps) {
    const int head = heads[g];
    int at = start[g];
    const int end = start[g + 1];
    for (int b0 = head & ~31; at < end; b0 += 32) {
      const int b = b0 + lane;
      const bool in = b < batch && leader[min(b, batch - 1)] == head;
      const uint32_t all = __ballot_sync(0xffffffffu, in);
      if (in) members[at + __popc(all & ((1u << lane) - 1))] = b;
      at += __popc(all);
    }
  }
  int rest = before;
  for (int b0 = 0; b0 < batch; b0 += kPlanThreads) {
    const int b = b0 + tid;
    const int alone = b < batch && kind[leader[min(b, batch - 1)]] != 2;
    int sum;
    const int at = rest + block_scan(alone, part, &sum);
    if (alone) members[at] = b;
    rest += sum;
  }
}

size_t groups_bytes(int batch) { return 4 * align_up(static_cast<size_t>(batch) * sizeof(int32_t), 256) + 256; }

}  // namespace

extern "C" size_t oscar_pages_workspace_bytes(const oscar_dims_t* dims, int32_t batch, int32_t num_forks) {
  if (check_pages(dims, batch, 0, nullptr) != OSCAR_OK || num_forks < 0) return 0;
  return layout(dims, batch, num_forks).total;
}

extern "C" oscar_status_t oscar_pages_copy(const oscar_dims_t* dims, int32_t num_pools, const oscar_page_pool_t* pools,
                                           int32_t num_copies, const int32_t* src, const int32_t* dst, void* stream) {
  const oscar_status_t st = check_pages(dims, 0, num_pools, pools);
  if (st != OSCAR_OK) return st;
  if (num_copies < 0) return OSCAR_ERR_INVALID_ARG;
  if (num_copies == 0 || num_pools == 0) return OSCAR_OK;
  if (!src || !dst) return OSCAR_ERR_INVALID_ARG;
  const Pools p = make_pools(num_pools, pools);
  copy_kernel<<<dim3(num_copies, page_parts(p)), 256, 0, as_stream(stream)>>>(p, src, dst, dims->num_pages);
  return launched();
}

extern "C" oscar_status_t oscar_pages_reserve(const oscar_dims_t* dims, int32_t batch, const int32_t* new_tokens,
                                              int32_t* page_table, int32_t* seq_lens, int32_t* page_refs,
                                              int32_t* granted, void* workspace, size_t workspace_bytes,
                                              void* stream) {
  oscar_status_t st = check_pages(dims, batch, 0, nullptr);
  if (st != OSCAR_OK) return st;
  if (batch == 0) return OSCAR_OK;
  if (!new_tokens || !page_table || !seq_lens || !page_refs || misaligned16(page_refs)) return OSCAR_ERR_INVALID_ARG;
  st = check_workspace(dims, batch, 0, workspace, workspace_bytes);
  if (st != OSCAR_OK) return st;
  const Layout l = layout(dims, batch, 0);
  char* w = static_cast<char*>(workspace);
  const Tables t{page_table, seq_lens, page_refs, batch, dims->num_pages, dims->max_pages_per_seq};
  reserve_kernel<<<1, kPlanThreads, 0, as_stream(stream)>>>(t, new_tokens, granted,
                                                            reinterpret_cast<int32_t*>(w + l.free_list),
                                                            reinterpret_cast<int32_t*>(w + l.first));
  return launched();
}

extern "C" oscar_status_t oscar_pages_fork(const oscar_dims_t* dims, int32_t num_pools, const oscar_page_pool_t* pools,
                                           int32_t batch, int32_t num_forks, const int32_t* src_seq,
                                           const int32_t* dst_seq, int32_t* page_table, int32_t* seq_lens,
                                           int32_t* page_refs, int32_t* granted, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  oscar_status_t st = check_pages(dims, batch, num_pools, pools);
  if (st != OSCAR_OK) return st;
  if (num_forks < 0) return OSCAR_ERR_INVALID_ARG;
  if (num_forks == 0) return OSCAR_OK;
  if (batch == 0 || !src_seq || !dst_seq || !page_table || !seq_lens || !page_refs || misaligned16(page_refs))
    return OSCAR_ERR_INVALID_ARG;
  st = check_workspace(dims, batch, num_forks, workspace, workspace_bytes);
  if (st != OSCAR_OK) return st;
  const Layout l = layout(dims, batch, num_forks);
  char* w = static_cast<char*>(workspace);
  const Tables t{page_table, seq_lens, page_refs, batch, dims->num_pages, dims->max_pages_per_seq};
  const Pools p = make_pools(num_pools, pools);
  ForkPlan* plan = reinterpret_cast<ForkPlan*>(w + l.plan);
  fork_plan_kernel<<<1, kPlanThreads, 0, as_stream(stream)>>>(t, src_seq, dst_seq, num_forks, granted,
                                                              reinterpret_cast<int32_t*>(w + l.claim),
                                                              reinterpret_cast<int32_t*>(w + l.free_list), plan);
  if (cudaGetLastError() != cudaSuccess) return OSCAR_ERR_CUDA;
  return launch_pdl(fork_apply_kernel, dim3(num_forks, page_parts(p)), dim3(256), 0, as_stream(stream), t, p, src_seq,
                    dst_seq, static_cast<const ForkPlan*>(plan)) == cudaSuccess
             ? OSCAR_OK
             : OSCAR_ERR_CUDA;
}

extern "C" oscar_status_t oscar_pages_free(const oscar_dims_t* dims, int32_t batch, int32_t num_seqs,
                                           const int32_t* seqs, int32_t* page_table, int32_t* seq_lens,
                                           int32_t* page_refs, void* stream) {
  const oscar_status_t st = check_pages(dims, batch, 0, nullptr);
  if (st != OSCAR_OK) return st;
  if (num_seqs < 0) return OSCAR_ERR_INVALID_ARG;
  if (num_seqs == 0) return OSCAR_OK;
  if (batch == 0 || !seqs || !page_table || !seq_lens || !page_refs) return OSCAR_ERR_INVALID_ARG;
  const Tables t{page_table, seq_lens, page_refs, batch, dims->num_pages, dims->max_pages_per_seq};
  free_kernel<<<num_seqs, 512, 0, as_stream(stream)>>>(t, seqs);
  return launched();
}

extern "C" oscar_status_t oscar_pages_trim(const oscar_dims_t* dims, int32_t batch, int32_t sink_len,
                                           int32_t window_len, int32_t* page_table, const int32_t* seq_lens,
                                           int32_t* page_refs, void* stream) {
  const oscar_status_t st = check_pages(dims, batch, 0, nullptr);
  if (st != OSCAR_OK) return st;
  if (sink_len < 0 || window_len < 1) return OSCAR_ERR_INVALID_ARG;
  if (batch == 0) return OSCAR_OK;
  if (!page_table || !seq_lens || !page_refs) return OSCAR_ERR_INVALID_ARG;
  const Tables t{page_table, const_cast<int32_t*>(seq_lens), page_refs, batch, dims->num_pages,
                 dims->max_pages_per_seq};
  const int gx = dims->max_pages_per_seq / 1024 + 1;
  trim_kernel<<<dim3(gx < 16 ? gx : 16, batch), 256, 0, as_stream(stream)>>>(t, sink_len, window_len);
  return launched();
}

extern "C" oscar_status_t oscar_pages_compact(const oscar_dims_t* dims, int32_t num_pools,
                                              const oscar_page_pool_t* pools, int32_t batch, int32_t* page_table,
                                              const int32_t* seq_lens, int32_t* page_refs, int32_t* num_used,
                                              void* workspace, size_t workspace_bytes, void* stream) {
  oscar_status_t st = check_pages(dims, batch, num_pools, pools);
  if (st != OSCAR_OK) return st;
  if (!page_refs || misaligned16(page_refs) || (batch > 0 && (!page_table || !seq_lens))) return OSCAR_ERR_INVALID_ARG;
  st = check_workspace(dims, batch, 0, workspace, workspace_bytes);
  if (st != OSCAR_OK) return st;
  const Layout l = layout(dims, batch, 0);
  char* w = static_cast<char*>(workspace);
  auto words = [&](size_t off) { return reinterpret_cast<int32_t*>(w + off); };
  const Tables t{page_table, const_cast<int32_t*>(seq_lens), page_refs, batch, dims->num_pages,
                 dims->max_pages_per_seq};
  const Pools p = make_pools(num_pools, pools);
  cudaStream_t s = as_stream(stream);
  const int chunks = (dims->num_pages + kChunk - 1) / kChunk;
  const int32_t* refs = page_refs;
  const bool own = chunks <= kOwnChunks;
  if (!own) {
    compact_count_kernel<<<chunks, kPlanThreads, 0, s>>>(refs, dims->num_pages, words(l.counts));
    if (cudaGetLastError() != cudaSuccess) return OSCAR_ERR_CUDA;
  }
  cudaError_t e = launch_pdl(compact_plan_kernel, dim3(chunks), dim3(kPlanThreads), 0, s, refs, dims->num_pages,
                             static_cast<const int32_t*>(own ? nullptr : words(l.counts)), chunks, words(l.from), words(l.to),
                             words(l.rank), words(l.info), num_used);
  if (e != cudaSuccess) return OSCAR_ERR_CUDA;
  const int movers = 8 * num_sms();
  e = launch_pdl(compact_apply_kernel, dim3(batch + movers), dim3(256), 0, s, t, p,
                 static_cast<const int32_t*>(words(l.from)), static_cast<const int32_t*>(words(l.to)),
                 static_cast<const int32_t*>(words(l.rank)), static_cast<const int32_t*>(words(l.info)));
  return e == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

extern "C" size_t oscar_pages_groups_workspace_bytes(const oscar_dims_t* dims, int32_t batch) {
  return check_pages(dims, batch, 0, nullptr) == OSCAR_OK ? groups_bytes(batch) : 0;
}

extern "C" oscar_status_t oscar_pages_groups(const oscar_dims_t* dims, int32_t batch, int32_t min_pages, int32_t max_groups,
                                             const int32_t* page_table, const int32_t* seq_lens, int32_t* members,
                                             int32_t* group_start, int32_t* prefix_lens, void* workspace,
                                             size_t workspace_bytes, void* stream) {
  const oscar_status_t st = check_pages(dims, batch, 0, nullptr);
  if (st != OSCAR_OK) return st;
  if (min_pages < 1 || max_groups < 1) return OSCAR_ERR_INVALID_ARG;
  if (batch == 0) return OSCAR_OK;
  if (!page_table || !seq_lens || !members || !group_start || !prefix_lens || !workspace ||
      reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
    return OSCAR_ERR_INVALID_ARG;
  if (workspace_bytes < groups_bytes(batch)) return OSCAR_ERR_WORKSPACE;
  const Tables t{const_cast<int32_t*>(page_table), const_cast<int32_t*>(seq_lens), nullptr, batch, dims->num_pages,
                 dims->max_pages_per_seq};
  const size_t each = align_up(static_cast<size_t>(batch) * sizeof(int32_t), 256);
  auto words = [&](int i) { return reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + i * each); };
  groups_find_kernel<<<batch, 256, 0, as_stream(stream)>>>(t, min_pages, words(0), words(1));
  if (cudaGetLastError() != cudaSuccess) return OSCAR_ERR_CUDA;
  const cudaError_t e = launch_pdl(groups_list_kernel, dim3(1), dim3(kPlanThreads), 0, as_stream(stream), batch,
                                   max_groups, static_cast<const int32_t*>(words(0)), static_cast<const int32_t*>(words(1)),
                                   words(2), words(3), members, group_start, prefix_lens);
  return e == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

oscar_status_t oscar_internal_pages_errors(uint32_t* flags, int reset) {
  return oscar::read_unit_errors(flags, reset) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}
