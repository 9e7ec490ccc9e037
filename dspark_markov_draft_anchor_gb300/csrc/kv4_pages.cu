// kv4_pages.cu -- the pages of a cache (dspark_pages_* of include/dspark_kv4.h):
// trimming, forking and growing page tables with reference counts, compacting
// a pool, copying pages' data.
//
// The bookkeeping works on a few thousand integers and is bound by latency:
// each call is one launch (two for compact), with no host in the loop.  What
// needs an order over the whole pool (the lowest free pages, the k-th live
// page) is done by one CTA whose warps own consecutive ranges of the
// reference counts: every warp counts its range, the 32 counts are scanned,
// and a second pass hands out ranks.  Results do not depend on the order in
// which threads run.
// Measured: trim, fork, grow and copy for 8 requests of 4 branches 11 us in a
// graph, 21 us as four calls (the host's part bounds those); a pool of 256 slots
// of 1 to 5 k tokens compacted, with the data of 4 layers moved (1.75 GB read and
// written), 300 us, 5.8 TB/s of a copy's 6.7.
#include "kv4.cuh"

namespace dspark {
namespace kv4 {
namespace {

constexpr int kWarpsPerBlock = 8;
constexpr unsigned kFull = 0xFFFFFFFFu;

struct Pool {
  int32_t num_pages, page_size, max_slots, max_pages;
  int32_t* refs;
  int32_t* table;
  int64_t table_stride;
  int32_t* lens;
};

__device__ __forceinline__ int32_t pages_of(const Pool& p, int32_t len) {
  if (len <= 0) return 0;
  const int32_t n = static_cast<int32_t>((static_cast<int64_t>(len) + p.page_size - 1) / p.page_size);
  return min(n, p.max_pages);
}

__device__ __forceinline__ bool has_slot(const Pool& p, int32_t slot) { return slot >= 0 && slot < p.max_slots; }
__device__ __forceinline__ bool has_page(const Pool& p, int32_t page) { return page >= 0 && page < p.num_pages; }

// One warp per slot.
__global__ void __launch_bounds__(32 * kWarpsPerBlock)
    trim_kernel(Pool p, int32_t n, const int32_t* __restrict__ slots, const int32_t* __restrict__ new_len) {
  const int32_t i = blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (i >= n) return;
  const int32_t slot = slots[i], to = new_len[i];
  if (!has_slot(p, slot)) return;
  const int32_t len = p.lens[slot];
  if (to < 0 || to >= len) return;
  int32_t* row = p.table + slot * p.table_stride;
  const int32_t end = pages_of(p, len);
  for (int32_t j = pages_of(p, to) + lane; j < end; j += 32) {
    const int32_t page = row[j];
    if (has_page(p, page)) atomicSub(&p.refs[page], 1);
    row[j] = -1;
  }
  __syncwarp();
  if (lane == 0) p.lens[slot] = to;
}

// One warp per pair.
__global__ void __launch_bounds__(32 * kWarpsPerBlock)
    fork_kernel(Pool p, int32_t n, const int32_t* __restrict__ src, const int32_t* __restrict__ dst) {
  const int32_t i = blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (i >= n) return;
  const int32_t a = src[i], b = dst[i];
  if (!has_slot(p, a) || !has_slot(p, b) || a == b) return;
  const int32_t len = p.lens[a];
  const int32_t held = pages_of(p, p.lens[b]), now = pages_of(p, len);
  const int32_t* from = p.table + a * p.table_stride;
  int32_t* to = p.table + b * p.table_stride;
  for (int32_t j = lane; j < max(held, now); j += 32) {
    const int32_t old = j < held ? to[j] : -1, page = j < now ? from[j] : -1;
    if (has_page(p, old)) atomicSub(&p.refs[old], 1);
    if (has_page(p, page)) atomicAdd(&p.refs[page], 1);
    to[j] = page;
  }
  __syncwarp();
  if (lane == 0) p.lens[b] = max(len, 0);
}

// ---------------------------------------------------------------------------
// One CTA over the whole pool
// ---------------------------------------------------------------------------
constexpr int kPoolThreads = 1024;
constexpr int kPoolWarps = kPoolThreads / 32;

// The range of reference counts that a warp owns: a multiple of 128, so that
// its lanes read aligned groups of four.
struct Range {
  int32_t lo, hi;
};
__device__ __forceinline__ Range warp_range(int32_t num_pages, int warp) {
  const int32_t per = ((num_pages + kPoolWarps - 1) / kPoolWarps + 127) / 128 * 128;
  const int64_t lo = static_cast<int64_t>(per) * warp;
  Range r;
  r.lo = static_cast<int32_t>(lo < num_pages ? lo : num_pages);
  r.hi = static_cast<int32_t>(lo + per < num_pages ? lo + per : num_pages);
  return r;
}

// refs[at .. at + 3], -1 behind the pool's end (neither free nor live).
template <bool kVec>
__device__ __forceinline__ int4 load_refs(const int32_t* refs, int32_t at, int32_t end) {
  if (kVec && at + 4 <= end) return *reinterpret_cast<const int4*>(refs + at);
  int4 r = make_int4(-1, -1, -1, -1);
  if (at < end) r.x = refs[at];
  if (at + 1 < end) r.y = refs[at + 1];
  if (at + 2 < end) r.z = refs[at + 2];
  if (at + 3 < end) r.w = refs[at + 3];
  return r;
}

template <typename Pred>
__device__ __forceinline__ uint32_t mask4(const int4& r, Pred pred) {
  return (pred(r.x) ? 1u : 0u) | (pred(r.y) ? 2u : 0u) | (pred(r.z) ? 4u : 0u) | (pred(r.w) ? 8u : 0u);
}

struct IsFree {
  __device__ __forceinline__ bool operator()(int32_t r) const { return r == 0; }
};
struct IsLive {
  __device__ __forceinline__ bool operator()(int32_t r) const { return r > 0; }
};

// How many of refs[lo .. hi) hold, over the warp; several loads in flight.
template <bool kVec, typename Pred>
__device__ __forceinline__ int32_t count_range(const int32_t* refs, Range r, Pred pred) {
  const int lane = threadIdx.x & 31;
  int32_t n = 0;
  for (int32_t at = r.lo + 4 * lane; at < r.hi; at += 128 * 4) {
#pragma unroll
    for (int u = 0; u < 4; ++u) n += __popc(mask4(load_refs<kVec>(refs, at + 128 * u, r.hi), pred));
  }
  return __reduce_add_sync(kFull, n);
}

// An inclusive sum over the warp.
__device__ __forceinline__ int32_t sum_warp(int32_t v) {
  return scan_warp(v, [](int32_t a, int32_t b) { return a + b; });
}

// A sum that stays at the type's largest value (for numbers of pages, so that
// wanting more than 2^31 pages is still more than are free).
__device__ __forceinline__ int32_t add_sat(int32_t a, int32_t b) {
  const uint32_t s = static_cast<uint32_t>(a) + static_cast<uint32_t>(b);
  return s > 0x7FFFFFFFu ? 0x7FFFFFFF : static_cast<int32_t>(s);
}

constexpr int kPerThread = DSPARK_PAGES_MAX_SLOTS / kPoolThreads;

__host__ __device__ __forceinline__ int hash_size(int32_t n) {
  int h = 64;
  while (h < 2 * n) h <<= 1;
  return h;
}

// Shared memory of grow_kernel.
__host__ __device__ __forceinline__ int grow_smem(int32_t n) { return hash_size(n) * 12 + n * 16 + 256; }

template <bool kVec>
__global__ void __launch_bounds__(kPoolThreads)
    grow_kernel(Pool p, int32_t n, const int32_t* __restrict__ slots, const int32_t* __restrict__ add,
                int32_t* __restrict__ copy_src, int32_t* __restrict__ copy_dst, int32_t* __restrict__ granted) {
  extern __shared__ int32_t sm[];
  const int hs = hash_size(n);
  int32_t* key = sm;          // page ids of partly filled last pages, -1 empty
  int32_t* holders = key + hs;  // listed slots on that page, with tokens to come that fit their tables
  int32_t* final_i = holders + hs;  // the last of them
  int32_t* before = final_i + hs;   // pages wanted before an item
  int32_t* item_slot = before + n;
  int32_t* item_have = item_slot + n;
  int32_t* item_flags = item_have + n;  // 1: takes a copy first, 2: granted, 4: keeps a page that others leave
  int32_t* scan = item_flags + n;       // [kPoolWarps]
  int32_t* scan2 = scan + kPoolWarps;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  for (int i = tid; i < hs; i += kPoolThreads) key[i] = -1, holders[i] = 0, final_i[i] = -1;
  const Range range = warp_range(p.num_pages, warp);
  const int32_t my_free = count_range<kVec>(p.refs, range, IsFree{});
  __syncthreads();

  // each thread's consecutive items
  const int per = (n + kPoolThreads - 1) / kPoolThreads;
  int32_t cur[kPerThread], more[kPerThread], last[kPerThread], fresh[kPerThread], where[kPerThread];
  const auto fits = [&](int u) {
    return more[u] >= 0 && static_cast<int64_t>(cur[u]) + more[u] <= static_cast<int64_t>(p.max_pages) * p.page_size;
  };
#pragma unroll
  for (int u = 0; u < kPerThread; ++u) {
    const int i = tid * per + u;
    cur[u] = 0, more[u] = 0, last[u] = -1, fresh[u] = 0, where[u] = -1;
    if (u >= per || i >= n) continue;
    const int32_t slot = slots[i];
    const bool ok = has_slot(p, slot);
    item_slot[i] = ok ? slot : -1;
    copy_src[i] = -1;
    copy_dst[i] = -1;
    more[u] = add[i];
    if (!ok) more[u] = -1;
    cur[u] = ok ? max(p.lens[slot], 0) : 0;
    const int32_t have = pages_of(p, cur[u]);
    item_have[i] = have;
    if (more[u] > 0) {
      const int64_t total = (static_cast<int64_t>(cur[u]) + more[u] + p.page_size - 1) / p.page_size;
      const int64_t f = total - have;
      fresh[u] = static_cast<int32_t>(f < 0 ? 0 : f);
      if (cur[u] % p.page_size != 0 && have > 0) {
        last[u] = p.table[slot * p.table_stride + have - 1];
        if (!has_page(p, last[u])) last[u] = -1;
      }
    }
    if (last[u] >= 0 && fits(u)) {
      uint32_t h = (static_cast<uint32_t>(last[u]) * 2654435761u) & (hs - 1);
      for (int t = 0; t < hs; ++t) {  // at most n of hs >= 2 n places are taken
        const int32_t was = atomicCAS(&key[h], -1, last[u]);
        if (was == -1 || was == last[u]) break;
        h = (h + 1) & (hs - 1);
      }
      where[u] = static_cast<int32_t>(h);
      atomicAdd(&holders[h], 1);
      atomicMax(&final_i[h], i);
    }
  }
  if (lane == 0) scan2[warp] = my_free;
  __syncthreads();

  // pages wanted by each item, and before it
  int32_t want[kPerThread], sum = 0;
#pragma unroll
  for (int u = 0; u < kPerThread; ++u) {
    const int i = tid * per + u;
    want[u] = 0;
    if (u >= per || i >= n) continue;
    bool copy = false, keep = false;
    if (last[u] >= 0) {
      const int32_t refs = p.refs[last[u]];
      keep = refs > 1 && where[u] >= 0 && holders[where[u]] == refs && final_i[where[u]] == i;
      copy = refs > 1 && !keep;
    }
    item_flags[i] = (copy ? 1 : 0) | (keep ? 4 : 0);
    want[u] = add_sat(fresh[u], copy ? 1 : 0);
    sum = add_sat(sum, want[u]);
  }
  const int32_t upto = scan_warp(sum, add_sat);
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
  if (warp == 0) {
    scan[lane] = scan_warp(scan[lane], add_sat);
  } else if (warp == 1) {
    scan2[lane] = sum_warp(scan2[lane]);
  }
  __syncthreads();
  const int32_t free_total = scan2[kPoolWarps - 1], want_total = scan[kPoolWarps - 1];
  // exclusive: what the lanes before hold, after what the warps before hold
  int32_t excl = __shfl_up_sync(kFull, upto, 1);
  if (lane == 0) excl = 0;
  int32_t at = add_sat(warp > 0 ? scan[warp - 1] : 0, excl);
#pragma unroll
  for (int u = 0; u < kPerThread; ++u) {
    const int i = tid * per + u;
    if (u >= per || i >= n) continue;
    before[i] = at;
    at = add_sat(at, want[u]);
    const bool ok = fits(u) && (want[u] == 0 || at <= free_total);
    if (ok) item_flags[i] |= 2;
    else if (where[u] >= 0) holders[where[u]] = -1;  // it stays on its page
  }
  __syncthreads();
  // A page that one of its holders stays on is kept by none of them: the keeper, who has the largest sum of pages
  // wanted among them, could not have a copy either.
#pragma unroll
  for (int u = 0; u < kPerThread; ++u) {
    const int i = tid * per + u;
    if (u >= per || i >= n) continue;
    int32_t flags = item_flags[i];
    if ((flags & 4) && holders[where[u]] < 0) item_flags[i] = flags &= ~2;
    const bool ok = flags & 2;
    granted[i] = ok ? 1 : 0;
    if (ok) p.lens[item_slot[i]] = cur[u] + more[u];
    if (ok && (flags & 1)) copy_src[i] = last[u];
  }
  __syncthreads();

  // the r-th free page goes to the item whose wanted pages hold number r
  const int32_t limit = min(want_total, free_total);
  int32_t rank = warp > 0 ? scan2[warp - 1] : 0;
  for (int32_t base = range.lo; base < range.hi && rank < limit; base += 128) {
    const uint32_t m = mask4(load_refs<kVec>(p.refs, base + 4 * lane, range.hi), IsFree{});
    const int32_t c = __popc(m), incl = sum_warp(c);
    int32_t r = rank + incl - c;
    rank += __shfl_sync(kFull, incl, 31);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (!(m >> e & 1)) continue;
      if (r < limit) {
        int lo = 0, hi = n;  // the last item with before <= r
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (before[mid] <= r) lo = mid;
          else hi = mid;
        }
        const int32_t flags = item_flags[lo];
        if (flags & 2) {
          const int32_t page = base + 4 * lane + e;
          const int32_t nth = r - before[lo] - (flags & 1);
          if (nth < 0) copy_dst[lo] = page;
          p.table[item_slot[lo] * p.table_stride + item_have[lo] + nth] = page;
          p.refs[page] = 1;
        }
      }
      ++r;
    }
  }
  __syncthreads();
  // pages that were given up for a copy
#pragma unroll
  for (int u = 0; u < kPerThread; ++u) {
    const int i = tid * per + u;
    if (u < per && i < n && (item_flags[i] & 3) == 3) atomicSub(&p.refs[last[u]], 1);
  }
}

// Ranks of the live pages: map, the moves, refs_out.
template <bool kVec>
__global__ void __launch_bounds__(kPoolThreads)
    compact_kernel(Pool p, int32_t* refs_out, int32_t* __restrict__ map, int32_t* __restrict__ move_src,
                   int32_t* __restrict__ move_dst, int32_t* __restrict__ count) {
  __shared__ int32_t scan[kPoolWarps];
  __shared__ int32_t live_below;  // live pages among ids 0 .. L - 1
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Range range = warp_range(p.num_pages, warp);
  const int32_t mine = count_range<kVec>(p.refs, range, IsLive{});
  if (lane == 0) scan[warp] = mine;
  if (tid == 0) live_below = p.num_pages;  // L == num_pages: every page lives
  __syncthreads();
  if (warp == 0) scan[lane] = sum_warp(scan[lane]);
  __syncthreads();
  const int32_t total = scan[kPoolWarps - 1];  // L
  const int32_t first = warp > 0 ? scan[warp - 1] : 0;
  if (range.lo <= total && total < range.hi) {
    Range r;
    r.lo = range.lo;
    r.hi = total;
    const int32_t below = first + count_range<kVec>(p.refs, r, IsLive{});
    if (lane == 0) live_below = below;
  }
  __syncthreads();
  const int32_t below = live_below;
  const int32_t moves = total - min(below, total);
  if (tid == 0) count[0] = moves;
  int32_t rank = first;
  for (int32_t base = range.lo; base < range.hi; base += 128) {
    const int32_t at = base + 4 * lane;
    const int4 v = load_refs<kVec>(p.refs, at, range.hi);
    const uint32_t m = mask4(v, IsLive{});
    const int32_t c = __popc(m), incl = sum_warp(c);
    int32_t r = rank + incl - c;
    rank += __shfl_sync(kFull, incl, 31);
    const int32_t ref[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int32_t id = at + e;
      if (id >= range.hi) break;
      const bool live = m >> e & 1;
      if (id < total) {
        map[id] = live ? id : -1;
        if (!live) move_dst[id - r] = id;
        refs_out[id] = live ? ref[e] : 0;
      } else {
        map[id] = -1;
        if (live) move_src[r - below] = id;
      }
      r += live ? 1 : 0;
    }
  }
  __syncthreads();
  for (int32_t k = tid; k < moves; k += kPoolThreads) {
    const int32_t a = move_src[k], b = move_dst[k];
    map[a] = b;
    refs_out[b] = p.refs[a];
  }
  __syncthreads();
  for (int32_t i = tid; i < p.num_pages; i += kPoolThreads) {
    if (i >= total) refs_out[i] = 0;
    if (i >= moves) move_src[i] = -1, move_dst[i] = -1;
  }
}

__global__ void __launch_bounds__(256)
    renumber_kernel(Pool p, const int32_t* __restrict__ map, int32_t* table_out) {
  const int64_t n = static_cast<int64_t>(p.max_slots) * p.max_pages;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t slot = i / p.max_pages;
    const int64_t at = slot * p.table_stride + (i - slot * p.max_pages);
    const int32_t page = p.table[at];
    table_out[at] = has_page(p, page) ? map[page] : page;
  }
}

// ---------------------------------------------------------------------------
// Page data
// ---------------------------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int64_t kCopyChunk = 16 * kCopyThreads * kCopyUnroll;  // bytes of a work item

__global__ void __launch_bounds__(kCopyThreads)
    copy_kernel(uint8_t* __restrict__ data, int32_t num_pages, int64_t page_bytes, int64_t page_stride, int32_t layers,
                int64_t layer_stride, int32_t n, const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
                const int32_t* __restrict__ count) {
  if (count) n = min(n, *count);
  const int64_t chunks = (page_bytes + kCopyChunk - 1) / kCopyChunk;
  const int64_t items = chunks * layers * n;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t chunk = it % chunks, rest = it / chunks;
    const int32_t layer = static_cast<int32_t>(rest % layers);
    const int32_t pair = static_cast<int32_t>(rest / layers);
    const int32_t a = src[pair], b = dst[pair];
    if (a < 0 || b < 0 || a >= num_pages || b >= num_pages || a == b) continue;
    uint8_t* base = data + layer * layer_stride + chunk * kCopyChunk;
    const uint4* from = reinterpret_cast<const uint4*>(base + a * page_stride);
    uint4* to = reinterpret_cast<uint4*>(base + b * page_stride);
    const int64_t left = page_bytes - chunk * kCopyChunk;
    const int words = static_cast<int>((left < kCopyChunk ? left : kCopyChunk) / 16);
    uint4 v[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
      const int w = threadIdx.x + u * kCopyThreads;
      if (w < words) v[u] = __ldcs(from + w);
    }
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
      const int w = threadIdx.x + u * kCopyThreads;
      if (w < words) __stcs(to + w, v[u]);
    }
  }
}

int make_pool(const dspark_page_pool* p, Pool* out) {
  if (!p || p->num_pages < 0 || p->num_pages > (1 << 30) || p->page_size < 1 || p->max_slots < 0 || p->max_pages < 0 ||
      p->table_stride < p->max_pages)
    return DSPARK_ERR_INVALID_ARG;
  if ((p->num_pages > 0 && !p->refs) || (p->max_slots > 0 && (!p->lens || (p->max_pages > 0 && !p->table))))
    return DSPARK_ERR_INVALID_ARG;
  if (!aligned(p->refs, 4) || !aligned(p->table, 4) || !aligned(p->lens, 4)) return DSPARK_ERR_MISALIGNED;
  *out = Pool{p->num_pages, p->page_size, p->max_slots, p->max_pages, p->refs, p->table, p->table_stride, p->lens};
  return DSPARK_OK;
}

// A list of n slots; *go: there is something to do.
int check_list(const dspark_page_pool* pool, int32_t n, const int32_t* a, const int32_t* b, Pool* p, bool* go) {
  const int rc = make_pool(pool, p);
  if (rc != DSPARK_OK) return rc;
  if (n < 0) return DSPARK_ERR_INVALID_ARG;
  if (n > DSPARK_PAGES_MAX_SLOTS) return DSPARK_ERR_TOO_MANY_ROWS;
  *go = n > 0;
  if (n > 0 && (!a || !b)) return DSPARK_ERR_INVALID_ARG;
  if (!aligned(a, 4) || !aligned(b, 4)) return DSPARK_ERR_MISALIGNED;
  return DSPARK_OK;
}

int launched() { return cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA; }

SmemAttr g_grow_attr[2];

}  // namespace
}  // namespace kv4
}  // namespace dspark

extern "C" {

int dspark_pages_trim(const dspark_page_pool* pool, int32_t n, const int32_t* slots, const int32_t* new_len,
                      cudaStream_t stream) {
  using namespace dspark::kv4;
  Pool p;
  bool go = false;
  const int rc = check_list(pool, n, slots, new_len, &p, &go);
  if (rc != DSPARK_OK || !go) return rc;
  trim_kernel<<<(n + kWarpsPerBlock - 1) / kWarpsPerBlock, 32 * kWarpsPerBlock, 0, stream>>>(p, n, slots, new_len);
  return launched();
}

int dspark_pages_fork(const dspark_page_pool* pool, int32_t n, const int32_t* src, const int32_t* dst,
                      cudaStream_t stream) {
  using namespace dspark::kv4;
  Pool p;
  bool go = false;
  const int rc = check_list(pool, n, src, dst, &p, &go);
  if (rc != DSPARK_OK || !go) return rc;
  fork_kernel<<<(n + kWarpsPerBlock - 1) / kWarpsPerBlock, 32 * kWarpsPerBlock, 0, stream>>>(p, n, src, dst);
  return launched();
}

int dspark_pages_grow(const dspark_page_pool* pool, int32_t n, const int32_t* slots, const int32_t* add,
                      int32_t* copy_src, int32_t* copy_dst, int32_t* granted, cudaStream_t stream) {
  using namespace dspark::kv4;
  Pool p;
  bool go = false;
  const int rc = check_list(pool, n, slots, add, &p, &go);
  if (rc != DSPARK_OK || !go) return rc;
  if (!copy_src || !copy_dst || !granted) return DSPARK_ERR_INVALID_ARG;
  if (!aligned(copy_src, 4) || !aligned(copy_dst, 4) || !aligned(granted, 4)) return DSPARK_ERR_MISALIGNED;
  const bool vec = aligned(p.refs, 16);
  const auto kernel = vec ? grow_kernel<true> : grow_kernel<false>;
  if (!smem_attr_ready(g_grow_attr[vec], kernel, grow_smem(DSPARK_PAGES_MAX_SLOTS))) return DSPARK_ERR_CUDA;
  kernel<<<1, kPoolThreads, grow_smem(n), stream>>>(p, n, slots, add, copy_src, copy_dst, granted);
  return launched();
}

int dspark_pages_compact(const dspark_page_pool* pool, int32_t* table_out, int32_t* refs_out, int32_t* map,
                         int32_t* move_src, int32_t* move_dst, int32_t* count, cudaStream_t stream) {
  using namespace dspark::kv4;
  Pool p;
  const int rc = make_pool(pool, &p);
  if (rc != DSPARK_OK) return rc;
  if (!count || (p.num_pages > 0 && (!refs_out || !map || !move_src || !move_dst)) ||
      (p.max_slots > 0 && p.max_pages > 0 && !table_out))
    return DSPARK_ERR_INVALID_ARG;
  if (!aligned(table_out, 4) || !aligned(refs_out, 4) || !aligned(map, 4) || !aligned(move_src, 4) ||
      !aligned(move_dst, 4) || !aligned(count, 4))
    return DSPARK_ERR_MISALIGNED;
  const auto kernel = aligned(p.refs, 16) ? compact_kernel<true> : compact_kernel<false>;
  kernel<<<1, kPoolThreads, 0, stream>>>(p, refs_out, map, move_src, move_dst, count);
  const int64_t entries = static_cast<int64_t>(p.max_slots) * p.max_pages;
  if (entries > 0) {
    const int64_t blocks = (entries + 255) / 256;
    renumber_kernel<<<static_cast<unsigned>(blocks < 1216 ? blocks : 1216), 256, 0, stream>>>(p, map, table_out);
  }
  return launched();
}

int dspark_pages_copy(void* data, int32_t num_pages, int64_t page_bytes, int64_t page_stride, int32_t layers,
                      int64_t layer_stride, int32_t n, const int32_t* src, const int32_t* dst, const int32_t* count,
                      cudaStream_t stream) {
  using namespace dspark::kv4;
  if (num_pages < 0 || page_bytes < 0 || page_stride < page_bytes || layers < 0 || n < 0 ||
      (layers > 1 && layer_stride < 0))
    return DSPARK_ERR_INVALID_ARG;
  if (n == 0 || layers == 0 || page_bytes == 0 || num_pages == 0) return DSPARK_OK;
  if (!data || !src || !dst) return DSPARK_ERR_INVALID_ARG;
  if (!aligned(data, 16) || page_bytes % 16 != 0 || page_stride % 16 != 0 || layer_stride % 16 != 0 ||
      !aligned(src, 4) || !aligned(dst, 4) || !aligned(count, 4))
    return DSPARK_ERR_MISALIGNED;
  const int64_t chunks = (page_bytes + kCopyChunk - 1) / kCopyChunk;
  const int64_t most = 152 * 8;
  const int64_t items = n < most ? chunks * layers * n : most;
  copy_kernel<<<static_cast<unsigned>(items < most ? items : most), kCopyThreads, 0, stream>>>(
      static_cast<uint8_t*>(data), num_pages, page_bytes, page_stride, layers, layer_stride, n, src, dst, count);
  return launched();
}

}  // extern "C"
