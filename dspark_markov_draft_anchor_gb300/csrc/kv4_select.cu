// kv4_select.cu -- the bounds of pages' keys, and the pages that a row attends to
// (dspark_kv4_bound_pages, dspark_kv4_select of include/dspark_kv4.h).
//
// For a query q and a key k within a page's bounds, <q, k> is at most
//   sum_d max(q_d lo_d, q_d hi_d) = sum_d (min(q_d, 0) lo_d + max(q_d, 0) hi_d),
// which is linear in the query's two parts: a head's group of queries adds its
// parts first, and a page costs one product of 2 D elements whatever the group.
// Both sides are int8, so that the sum is exact (below 2^23) and which pages are
// taken does not depend on its order.
//
// A call reads each page's bounds once (272 bytes a page and head at 128
// dimensions, 1/34 of the page's own bytes at 64 tokens): 32 rows over 16 to 64 k
// tokens, 40 MB, 18 us, 2.3 TB/s.  That is a third of the memory's rate: what bounds a
// call, over long caches and short ones, is its launches and each one's chain of
// dependent loads (request, slot, length, page, bounds); 11 us for one row over 128 k
// tokens, 4.5 MB.
#include "kv4.cuh"

namespace dspark {
namespace kv4 {
namespace {

template <int kDim>
constexpr int kBoundBytes = 2 * kDim + 16;

__device__ __forceinline__ uint32_t min_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float half_of(uint32_t two, int i) {
  return __half2float(__ushort_as_half(static_cast<uint16_t>(i ? two >> 16 : two)));
}

// ---- bounds -----------------------------------------------------------------
// A row stands for its page where the next row is in another page or there is none.

// The page that row `row` of request i stands for, or -1, and how many tokens it
// holds.
__device__ __forceinline__ int32_t page_of(const Cache& c, const Batch& s, int32_t i, int32_t row, int32_t& held) {
  if (i < 0) return -1;
  const Request r = load_request(s, i);
  const int32_t j = row - r.start, pos = r.len - r.rows + j;
  if (j < 0 || j >= r.rows || pos < 0 || (j != r.rows - 1 && (pos + 1) % c.page_size != 0)) return -1;
  const int32_t id = r.pages[pos >> c.page_shift];
  held = (pos & (c.page_size - 1)) + 1;
  return id < c.num_pages ? id : -1;
}

// The smallest and largest key elements of a page's tokens first, first + step, ..
// below `held`, by a warp: a lane has 32 dimensions of every kTokens-th of them, and
// ends with those of lane % kLanes, as FP16, over all.
template <int kDim>
struct Extremes {
  static constexpr int kLanes = kDim / 32;     // of a token: 16 bytes of codes each
  static constexpr int kTokens = 32 / kLanes;  // at a time
  uint32_t lo[16], hi[16];

  template <int kDepth>  // loads of a lane in flight
  __device__ __forceinline__ void take(const Cache& c, int32_t page, int32_t head, int32_t first, int32_t step,
                                       int32_t held) {
    using R = Record<kDim>;
    const int lane = threadIdx.x & 31;
    const uint8_t* rec = c.data + static_cast<int64_t>(page) * c.page_stride +
                         static_cast<int64_t>(head) * R::bytes(c.page_size);
    const uint8_t* codes = rec + R::codes(c.page_size, 0) + (lane % kLanes) * 16;
    const uint8_t* scales = rec + R::scales(c.page_size, 0) + (lane % kLanes) * 2;
#pragma unroll
    for (int i = 0; i < 16; ++i) lo[i] = 0x7C007C00u, hi[i] = 0xFC00FC00u;  // +inf, -inf
    for (int32_t t0 = first + lane / kLanes; t0 < held; t0 += kDepth * step) {
      uint4 w[kDepth];
      uint32_t two[kDepth];
#pragma unroll
      for (int u = 0; u < kDepth; ++u) {  // tokens behind the last: the first one's again
        const int32_t t = t0 + u * step < held ? t0 + u * step : t0;
        w[u] = *reinterpret_cast<const uint4*>(codes + t * R::kCodeBytes);
        two[u] = *reinterpret_cast<const uint16_t*>(scales + t * R::kScaleBytes);
      }
#pragma unroll
      for (int u = 0; u < kDepth; ++u) {
        const uint32_t s2 = scales_to_f16(two[u]);
        const uint32_t by[2] = {__byte_perm(s2, s2, 0x1010), __byte_perm(s2, s2, 0x3232)};
        const uint32_t word[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t x[4];
          e2m1x8_to_f16(word[i], x);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t y = mul_f16x2(x[e], by[i / 2]);
            lo[4 * i + e] = min_f16x2(lo[4 * i + e], y);
            hi[4 * i + e] = max_f16x2(hi[4 * i + e], y);
          }
        }
      }
    }
#pragma unroll
    for (int d = kLanes; d < 32; d <<= 1)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        lo[i] = min_f16x2(lo[i], __shfl_xor_sync(0xFFFFFFFFu, lo[i], d));
        hi[i] = max_f16x2(hi[i], __shfl_xor_sync(0xFFFFFFFFu, hi[i], d));
      }
  }
  // All of them in order, lo, then hi.
  __device__ __forceinline__ void leave(uint32_t (&ends)[kDim]) const {
    const int lane = threadIdx.x & 31;
    if (lane >= kLanes) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      ends[lane * 16 + i] = lo[i];
      ends[kDim / 2 + lane * 16 + i] = hi[i];
    }
  }
};

// The fraction of `top`, of 127, that x is, as a byte.
__device__ __forceinline__ uint32_t fraction(float x, float top) {
  return top > 0.0f ? static_cast<uint32_t>(__float2int_rn(__fdiv_rn(__fmul_rn(127.0f, x), top))) & 0xFFu : 0u;
}

// Many rows: a CTA takes up to 32, its warps those pages' heads in turn.
constexpr int kBoundWarps = 8;
template <int kDim>
__global__ void __launch_bounds__(32 * kBoundWarps)
    bound_kernel(Cache c, Batch s, uint8_t* bounds, int64_t bounds_stride, int32_t rows_of_cta) {
  __shared__ int32_t ids[32], tokens[32], count;
  __shared__ __align__(16) uint32_t ends[kBoundWarps][kDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 0) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * rows_of_cta + lane;
    int32_t id = -1, held = 0;
    if (lane < rows_of_cta && row < s.total_rows)
      id = page_of(c, s, find_request(s, static_cast<int32_t>(row)), static_cast<int32_t>(row), held);
    const uint32_t some = __ballot_sync(0xFFFFFFFFu, id >= 0);
    if (id >= 0) {
      const int at = __popc(some & ((1u << lane) - 1));
      ids[at] = id;
      tokens[at] = held;
    }
    if (lane == 0) count = __popc(some);
  }
  __syncthreads();
  using E = Extremes<kDim>;
  const int32_t items = count * c.kv_heads;
  for (int32_t item = warp; item < items; item += kBoundWarps) {
    const int32_t at = item / c.kv_heads, head = item - at * c.kv_heads;
    E x;
    x.template take<4>(c, ids[at], head, 0, E::kTokens, tokens[at]);
    uint32_t top2 = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top2 = max_f16x2(top2, max_f16x2(x.lo[i] & 0x7FFF7FFFu, x.hi[i] & 0x7FFF7FFFu));
#pragma unroll
    for (int d = 1; d < E::kLanes; d <<= 1) top2 = max_f16x2(top2, __shfl_xor_sync(0xFFFFFFFFu, top2, d));
    const float top = fmaxf(half_of(top2, 0), half_of(top2, 1));
    __syncwarp();
    x.leave(ends[warp]);
    __syncwarp();
    // a lane's share of the 2 D ends: 4 words of 2 (8 values) at 128 dimensions, 2 at 64
    constexpr int kWords = kDim / 32;
    uint8_t* out = bounds + static_cast<int64_t>(ids[at]) * bounds_stride +
                   static_cast<int64_t>(head) * kBoundBytes<kDim>;
#pragma unroll
    for (int i = 0; i < kWords / 2; ++i) {
      uint32_t v = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v |= fraction(half_of(ends[warp][lane * kWords + 2 * i + e / 2], e & 1), top) << (8 * e);
      reinterpret_cast<uint32_t*>(out)[lane * (kWords / 2) + i] = v;
    }
    if (lane < 4) reinterpret_cast<uint32_t*>(out + 2 * kDim)[lane] = lane == 0 ? __float_as_uint(top) : 0u;
  }
}

// Few rows: a CTA a row and head, whose warps share the page's tokens.  One row of 8
// heads of 128 dimensions in a page of 64: 3.4 us, with the kernel above 5.6.
constexpr int kOneWarps = 4;
template <int kDim>
__global__ void __launch_bounds__(32 * kOneWarps)
    bound_one_kernel(Cache c, Batch s, uint8_t* bounds, int64_t bounds_stride) {
  __shared__ __align__(16) uint32_t ends[kOneWarps][kDim];
  __shared__ uint32_t tops[kOneWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t row = static_cast<int32_t>(blockIdx.x / c.kv_heads), head = blockIdx.x % c.kv_heads;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int32_t held = 0;
  const int32_t page = page_of(c, s, find_request_warp(s, row), row, held);
  if (page < 0) return;  // the whole CTA
  using E = Extremes<kDim>;
  E x;
  x.template take<2>(c, page, head, warp * E::kTokens, kOneWarps * E::kTokens, held);
  x.leave(ends[warp]);
  __syncthreads();
  uint32_t two = 0, top2 = 0;  // a word of the 2 D ends
  if (tid < kDim) {
    two = ends[0][tid];
#pragma unroll
    for (int w = 1; w < kOneWarps; ++w)
      two = tid < kDim / 2 ? min_f16x2(two, ends[w][tid]) : max_f16x2(two, ends[w][tid]);
    top2 = max(two & 0x7FFFu, two >> 16 & 0x7FFFu);  // magnitudes in the order of their bits
  }
  top2 = __reduce_max_sync(0xFFFFFFFFu, top2);
  if (lane == 0) tops[warp] = top2;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kOneWarps; ++w) top2 = max(top2, tops[w]);
  const float top = half_of(top2, 0);
  uint8_t* out = bounds + static_cast<int64_t>(page) * bounds_stride + static_cast<int64_t>(head) * kBoundBytes<kDim>;
  if (tid < kDim)
    reinterpret_cast<uint16_t*>(out)[tid] =
        static_cast<uint16_t>(fraction(half_of(two, 0), top) | fraction(half_of(two, 1), top) << 8);
  if (tid < 4) reinterpret_cast<uint32_t*>(out + 2 * kDim)[tid] = tid == 0 ? __float_as_uint(top) : 0u;
}

// ---- selection --------------------------------------------------------------
struct Select {
  Cache c;
  Batch s;
  const uint8_t* bounds;
  int64_t bounds_stride;
  const uint16_t* q;
  int64_t q_row, q_head;
  int32_t group;
  int32_t vec;  // 16-byte loads of q
  int32_t first, last, top;
  int32_t* pages;
  int32_t* lens;
  uint8_t* parts;   // workspace: [rows][heads][2 D]
  uint32_t* keys;   // workspace: [rows][heads][stride]
  int64_t stride;   // max_pages, to a multiple of 4
};

// Scores in an order of whole numbers (-0 as +0, NaN the largest): 0 is a page that is
// not there, the largest number one that is taken in any case, which no score reaches.
constexpr uint32_t kAbsent = 0u, kForced = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t key_of(float score) {
  const uint32_t u = __float_as_uint(score + 0.0f);
  if (isnan(score)) return kForced - 1;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Of a row, so that 31 bits count a group's queries 8 at a time behind its last one, too.
constexpr int32_t kMostQueryHeads = 1 << 30;

// The int8 parts of a row's queries of one head, by a warp: a lane's dimensions are
// 4 lane .. (128) or 2 lane .. (64).
template <int kDim, bool kBf16>
__device__ __forceinline__ void make_parts(const Select& p, int64_t row, int32_t head, uint8_t* out) {
  constexpr int kN = kDim / 32, kDepth = 8;
  const int lane = threadIdx.x & 31;
  const bool flip = p.c.k_scale && p.c.k_scale[head] < 0.0f;
  const uint16_t* q = p.q + row * p.q_row + static_cast<int64_t>(head) * p.group * p.q_head + lane * kN;
  float lo[kN], hi[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) lo[i] = hi[i] = 0.0f;
  for (int32_t m0 = 0; m0 < p.group; m0 += kDepth) {
    uint32_t w[kDepth][kN / 2];
#pragma unroll
    for (int u = 0; u < kDepth; ++u) {
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) w[u][i] = 0u;
      if (m0 + u >= p.group) continue;
      const uint16_t* from = q + (m0 + u) * p.q_head;
      if (p.vec) {
        if (kN == 4) {
          const uint2 v = *reinterpret_cast<const uint2*>(from);
          w[u][0] = v.x, w[u][kN / 2 - 1] = v.y;
        } else {
          w[u][0] = *reinterpret_cast<const uint32_t*>(from);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) w[u][i] = from[2 * i] | (static_cast<uint32_t>(from[2 * i + 1]) << 16);
      }
    }
#pragma unroll
    for (int u = 0; u < kDepth; ++u)
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const uint32_t bits = i & 1 ? w[u][i / 2] >> 16 : w[u][i / 2] & 0xFFFFu;
        float x = kBf16 ? __uint_as_float(bits << 16) : half_of(bits, 0);
        x = isnan(x) ? 0.0f : fminf(fmaxf(x, -0x1p100f), 0x1p100f);
        if (flip) x = -x;
        lo[i] += fminf(x, 0.0f);
        hi[i] += fmaxf(x, 0.0f);
      }
  }
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < kN; ++i) top = fmaxf(top, fmaxf(-lo[i], hi[i]));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  uint32_t a = 0, b = 0;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int u = top > 0.0f ? __float2int_rn(__fdiv_rn(__fmul_rn(127.0f, lo[i]), top)) : 0;
    const int v = top > 0.0f ? __float2int_rn(__fdiv_rn(__fmul_rn(127.0f, hi[i]), top)) : 0;
    a |= static_cast<uint32_t>(u & 0xFF) << (8 * i);
    b |= static_cast<uint32_t>(v & 0xFF) << (8 * i);
  }
  out += lane * kN;
  if (kN == 4) {
    *reinterpret_cast<uint32_t*>(out) = a;
    *reinterpret_cast<uint32_t*>(out + kDim) = b;
  } else {
    *reinterpret_cast<uint16_t*>(out) = static_cast<uint16_t>(a);
    *reinterpret_cast<uint16_t*>(out + kDim) = static_cast<uint16_t>(b);
  }
}

constexpr int kPartWarps = 4;
template <int kDim, bool kBf16>
__global__ void __launch_bounds__(32 * kPartWarps) parts_kernel(const __grid_constant__ Select p) {
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kPartWarps + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (item >= static_cast<int64_t>(p.s.total_rows) * p.c.kv_heads) return;
  const int64_t row = item / p.c.kv_heads;
  make_parts<kDim, kBf16>(p, row, static_cast<int32_t>(item - row * p.c.kv_heads), p.parts + item * (2 * kDim));
}

// Scores of a request's pages by one head's queries of up to 16 rows: an item of
// the line (request, 16 rows, some pages, head), which the warps take in turn.  A
// warp's lanes ask for 16 bytes of the pages' bounds each, so that a load
// instruction covers whole records, and meet them with the same 16 bytes of a row's
// parts; the sums over a record's lanes are folded over the records, so that each
// lane ends with one page's.  The items and the first bounds are looked up while the
// parts are made.
constexpr int kScoreThreads = 128;
constexpr int kScorePages = 16;  // of a warp
constexpr int kScoreRows = 16;
constexpr int kScoreCtas = 6;   // of an SM: with 4, 7, 8 and 32 or 8 pages a warp 32 rows take 18 to 23 us for 18

struct Items {
  int32_t row_parts, page_parts;
};
__device__ __forceinline__ Items items_of(const Select& p, const Request& r) {
  Items x{0, 0};
  const int32_t pages = (r.len + p.c.page_size - 1) / p.c.page_size;  // of the last row
  if (r.rows == 0 || pages <= p.top) return x;
  x.row_parts = (r.rows - 1) / kScoreRows + 1;
  x.page_parts = (pages - 1) / kScorePages + 1;
  return x;
}

// prefix[i]: items of the requests before i, by the whole CTA.
__device__ __forceinline__ void plan_items(const Select& p, int64_t* prefix) {
  constexpr int kWarps = kScoreThreads / 32;
  __shared__ int64_t sums[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t per = (p.s.batch + kScoreThreads - 1) / kScoreThreads;
  const int32_t lo = min(tid * per, p.s.batch), hi = min(lo + per, p.s.batch);
  int64_t sum = 0;
  for (int32_t i = lo; i < hi; ++i) {
    const Items x = items_of(p, load_request(p.s, i));
    prefix[i] = sum;
    sum += static_cast<int64_t>(x.row_parts) * x.page_parts * p.c.kv_heads;
  }
  int64_t upto = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  int64_t before = upto - sum;
  for (int w = 0; w < warp; ++w) before += sums[w];
  for (int32_t i = lo; i < hi; ++i) prefix[i] += before;
  if (tid == kScoreThreads - 1) prefix[p.s.batch] = before + sum;
  __syncthreads();
}

// A warp's pages: their bounds' pieces, and the products with a row's parts.
template <int kDim>
struct Scorer {
  static constexpr int kLanes = 2 * kDim / 16;   // of a record
  static constexpr int kTogether = 32 / kLanes;  // records of a load
  static constexpr int kLoads = kScorePages / kTogether;  // of a lane
  static constexpr int kSame = kLanes / kLoads;           // lanes that end with one page's sum
  int piece, sub;
  int mine;  // the record that this lane ends with
  uint4 w[kLoads];
  float m;
  int32_t id;  // of record `mine`, -1 if it is not there

  __device__ __forceinline__ Scorer() {
    const int lane = threadIdx.x & 31;
    piece = lane % kLanes, sub = lane / kLanes;
    mine = piece / kSame * kTogether + sub;
  }
  // Asks for the bounds of pages table[0 .. n - 1] of a head.
  __device__ __forceinline__ void load(const Select& p, int32_t head, const int32_t* table, int32_t n) {
    id = mine < n ? table[mine] : -1;
    if (id >= p.c.num_pages) id = -1;
    const uint8_t* bounds = p.bounds + static_cast<int64_t>(head) * kBoundBytes<kDim>;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int32_t of = __shfl_sync(0xFFFFFFFFu, id, sub * kLanes + j * kSame);
      w[j] = make_uint4(0u, 0u, 0u, 0u);
      if (of >= 0) w[j] = reinterpret_cast<const uint4*>(bounds + static_cast<int64_t>(of) * p.bounds_stride)[piece];
    }
    m = 0.0f;
    if (id >= 0) m = *reinterpret_cast<const float*>(bounds + static_cast<int64_t>(id) * p.bounds_stride + 2 * kDim);
  }
  // The key of page `mine`, by a row's parts' piece; right in lanes with has().
  __device__ __forceinline__ bool has() const { return piece % kSame == 0; }
  __device__ __forceinline__ uint32_t key(uint4 q) const {
    int v[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      v[u] = __dp4a(static_cast<int>(w[u].x), static_cast<int>(q.x), 0);
      v[u] = __dp4a(static_cast<int>(w[u].y), static_cast<int>(q.y), v[u]);
      v[u] = __dp4a(static_cast<int>(w[u].z), static_cast<int>(q.z), v[u]);
      v[u] = __dp4a(static_cast<int>(w[u].w), static_cast<int>(q.w), v[u]);
    }
#pragma unroll
    for (int half = kLoads / 2; half > 0; half >>= 1) {
      const bool upper = piece & half * kSame;
#pragma unroll
      for (int u = 0; u < half; ++u) {
        const int keep = upper ? v[u + half] : v[u], give = upper ? v[u] : v[u + half];
        v[u] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, half * kSame);
      }
    }
#pragma unroll
    for (int d = kSame / 2; d > 0; d >>= 1) v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], d);
    return id >= 0 ? key_of(__fmul_rn(m, static_cast<float>(v[0]))) : kAbsent;
  }
};

template <int kDim>
__global__ void __launch_bounds__(kScoreThreads, kScoreCtas) score_kernel(const __grid_constant__ Select p) {
  constexpr int kDepth = 4;  // rows whose parts are in flight together
  extern __shared__ int64_t prefix[];
  const int warp = threadIdx.x >> 5;
  Scorer<kDim> scorer;
  plan_items(p, prefix);
  bool waited = false;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * (kScoreThreads / 32) + warp; item < prefix[p.s.batch];
       item += gridDim.x * (kScoreThreads / 32)) {
    int32_t i = 0, behind = p.s.batch;  // prefix[i] <= item < prefix[behind]
    while (behind - i > 1) {
      const int32_t mid = (i + behind) >> 1;
      if (prefix[mid] <= item) i = mid;
      else behind = mid;
    }
    const Request r = load_request(p.s, i);
    const Items x = items_of(p, r);
    const int64_t in = item - prefix[i], part = in / p.c.kv_heads;
    const int32_t head = static_cast<int32_t>(in - part * p.c.kv_heads);
    const int32_t row0 = static_cast<int32_t>(part / x.page_parts) * kScoreRows;
    const int32_t page0 = static_cast<int32_t>(part % x.page_parts) * kScorePages;
    const int32_t rows = min(r.rows - row0, kScoreRows);
    const int32_t pos0 = r.len - r.rows + row0;  // of the first row
    const int32_t end = pos0 + rows > 0 ? (pos0 + rows - 1) / p.c.page_size + 1 : 0;  // pages that the last row sees
    if (page0 >= end) continue;

    scorer.load(p, head, r.pages + page0, end - page0);
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
    waited = true;
    const int64_t list0 = static_cast<int64_t>(r.start + row0) * p.c.kv_heads + head;
    for (int j0 = 0; j0 < rows; j0 += kDepth) {
      uint4 q[kDepth];
#pragma unroll
      for (int u = 0; u < kDepth; ++u)
        if (j0 + u < rows)
          q[u] = *reinterpret_cast<const uint4*>(
              p.parts + (list0 + static_cast<int64_t>(j0 + u) * p.c.kv_heads) * (2 * kDim) + 16 * scorer.piece);
#pragma unroll
      for (int g = 0; g < kDepth; ++g) {
        const int j = j0 + g;
        if (j >= rows) break;
        const uint32_t key = scorer.key(q[g]);
        const int32_t pos = pos0 + j, page = page0 + scorer.mine;
        if (scorer.has() && pos >= 0 && page <= pos / p.c.page_size)
          p.keys[(list0 + static_cast<int64_t>(j) * p.c.kv_heads) * p.stride + page] = key;
      }
    }
  }
  if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The list of a row and head, by a CTA.  What it looks up before it waits was
// written before the scores' kernel began, which waited for it.  Up to 2048 pages, a
// thread has up to 16 pages in a row, with their keys and ids in registers.  The
// smallest key that is taken is built bit by bit from the highest one in which the
// keys differ: one count of those at or above it a bit, until exactly as many are
// as are wanted (about 12 bits, where sorting by bytes takes 4 passes over bins that
// most keys share).
constexpr int kListThreads = 128;
constexpr int kListWarps = kListThreads / 32;
constexpr int kOwn = 16;          // pages of a thread
constexpr int kListKeys = 12288;  // of a longer list, held in shared memory

// The sum over the CTA of two numbers below 2^16, and that of the threads before.
__device__ __forceinline__ void scan_cta(uint32_t v, uint32_t* sums, uint32_t& before, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t upto = scan_warp(static_cast<int32_t>(v), [](int32_t a, int32_t b) { return a + b; });
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  before = upto - v, total = 0;
#pragma unroll
  for (int w = 0; w < kListWarps; ++w) {
    before += w < warp ? sums[w] : 0;
    total += sums[w];
  }
}

// More pages than threads hold: the `want`-th largest key by its bytes, the highest
// first, then the pages in order, each warp a run of them.
__device__ __noinline__ void list_long(const Select& p, const uint32_t* keys, const int32_t* table, int32_t n,
                                       int32_t* out) {
  extern __shared__ uint32_t kept[];
  __shared__ uint32_t bins[256];
  __shared__ int32_t warp_above[kListWarps], warp_equal[kListWarps];
  __shared__ uint32_t chosen;
  __shared__ int32_t left;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool fits = n <= kListKeys;
  const auto fetch = [&](int32_t k) { return k < p.first || k >= n - p.last ? kForced : keys[k]; };
  if (fits)
    for (int32_t k = tid; k < n; k += kListThreads) kept[k] = fetch(k);
  const auto key = [&](int32_t k) { return fits ? kept[k] : fetch(k); };
  uint32_t prefix = 0, mask = 0;
  int32_t want = p.top;  // of the keys that begin with the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int b = tid; b < 256; b += kListThreads) bins[b] = 0;
    __syncthreads();
    for (int32_t k = tid; k < n; k += kListThreads) {
      const uint32_t u = key(k);
      if ((u & mask) == prefix) atomicAdd(&bins[u >> shift & 255u], 1u);
    }
    __syncthreads();
    if (warp == 0) {  // lane's bins, from the highest: 255 - 8 lane ..
      int32_t sum = 0;
      for (int b = 0; b < 8; ++b) sum += bins[255 - 8 * lane - b];
      const int32_t upto = scan_warp(sum, [](int32_t a, int32_t b) { return a + b; });
      const uint32_t here = __ballot_sync(0xFFFFFFFFu, upto >= want);
      if (lane == __ffs(here) - 1) {
        int32_t rest = want - (upto - sum);
        int b = 255 - 8 * lane;
        while (rest > static_cast<int32_t>(bins[b])) rest -= bins[b--];
        chosen = b;
        left = rest;
      }
    }
    __syncthreads();
    prefix |= chosen << shift;
    mask |= 255u << shift;
    want = left;
  }
  const int32_t run = (n + kListWarps - 1) / kListWarps, lo = min(warp * run, n), hi = min(lo + run, n);
  int32_t above = 0, equal = 0;
  for (int32_t k = lo + lane; k < hi; k += 32) {
    const uint32_t u = key(k);
    above += u > prefix, equal += u == prefix;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    above += __shfl_xor_sync(0xFFFFFFFFu, above, d);
    equal += __shfl_xor_sync(0xFFFFFFFFu, equal, d);
  }
  if (lane == 0) warp_above[warp] = above, warp_equal[warp] = equal;
  __syncthreads();
  int32_t at = 0, equals = 0;  // listed before, and how many of those before are equal
  for (int w = 0; w < warp; ++w) at += warp_above[w], equals += warp_equal[w];
  at += min(equals, want);
  for (int32_t base = lo; base < hi; base += 32) {
    const int32_t k = base + lane;
    const uint32_t u = k < hi ? key(k) : 0u;
    const uint32_t same = __ballot_sync(0xFFFFFFFFu, k < hi && u == prefix);
    const bool take = k < hi && (u > prefix || (u == prefix && equals + __popc(same & ((1u << lane) - 1)) < want));
    const uint32_t taken = __ballot_sync(0xFFFFFFFFu, take);
    if (take) out[at + __popc(taken & ((1u << lane) - 1))] = table[k];
    at += __popc(taken);
    equals += __popc(same);
  }
}

// A row of the batch: its request's page table, how many pages it sees, and the
// tokens of the pages that it gets (-1: no request has it).
struct Seen {
  const int32_t* table;
  int32_t pages, tokens;
};
__device__ __forceinline__ Seen look_up(const Select& p, int32_t row) {
  Seen x{p.s.table, 0, -1};
  const int32_t i = find_request_warp(p.s, row);
  if (i < 0) return x;
  const Request r = load_request(p.s, i);
  const int32_t j = row - r.start, pos = r.len - r.rows + j;
  x.tokens = 0;
  if (j < 0 || j >= r.rows || pos < 0) return x;
  x.pages = pos / p.c.page_size + 1;
  x.tokens = (min(x.pages, p.top) - 1) * p.c.page_size + pos % p.c.page_size + 1;
  x.table = r.pages;
  return x;
}
__device__ __forceinline__ void list_all(const Select& p, const Seen& x, int32_t* out) {
  const uint32_t top = p.top, n = x.pages;  // unsigned: a place behind the last may be 2^31 or more
  for (uint32_t k = threadIdx.x; k < top; k += kListThreads) out[k] = k < n ? x.table[k] : -1;
}

// Of n > top pages: thread t has `own` (at most kOwn) from own t on, with ids `ids`;
// their keys are at `from` (16-byte aligned, to a multiple of 4).
template <int kOwn>
__device__ __forceinline__ void list_short(const Select& p, const uint32_t* from, int32_t n, int32_t own,
                                           const int32_t (&ids)[kOwn], int32_t* out) {
  __shared__ uint32_t sums[2][kListWarps], ends[2][kListWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t k0 = tid * own;
  uint32_t key[kOwn];  // 0 behind the last page, as what is absent: never above what is taken
  uint32_t all = ~0u, any = 0u;  // bits that all keys have, that any has; without the pages taken in any case
#pragma unroll
  for (int j = 0; j < kOwn; j += 4) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (j < own && k0 + j < n) v = *reinterpret_cast<const uint4*>(from + k0 + j);
    key[j] = v.x, key[j + 1] = v.y, key[j + 2] = v.z, key[j + 3] = v.w;
  }
#pragma unroll
  for (int j = 0; j < kOwn; ++j) {
    const int32_t k = k0 + j;
    if (j >= own || k >= n) key[j] = kAbsent;
    else if (k < p.first || k >= n - p.last) key[j] = kForced;
    else all &= key[j], any |= key[j];
  }
  all = __reduce_and_sync(0xFFFFFFFFu, all);
  any = __reduce_or_sync(0xFFFFFFFFu, any);
  if (lane == 0) ends[0][warp] = all, ends[1][warp] = any;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kListWarps; ++w) all &= ends[0][w], any |= ends[1][w];
  // the largest `least` that as many keys as are wanted reach; the pages taken in any case reach all
  uint32_t least = 0u;
  bool exact = false;
  const uint32_t differ = all ^ any;
  const int high = differ != 0 ? 31 - __clz(differ) : -1;
  if (high < 31) least = any >> (high + 1) << (high + 1);
  for (int bit = high, turn = 0; bit >= 0 && !exact; --bit, turn ^= 1) {
    const uint32_t trial = least | 1u << bit;
    int32_t reach = 0;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) reach += key[j] >= trial;
    reach = __reduce_add_sync(0xFFFFFFFFu, reach);
    if (lane == 0) sums[turn][warp] = reach;
    __syncthreads();
    reach = 0;
#pragma unroll
    for (int w = 0; w < kListWarps; ++w) reach += sums[turn][w];
    if (reach >= p.top) least = trial, exact = reach == p.top;
  }
  // the pages above it, and of those equal to it the first
  uint32_t mine = 0;
#pragma unroll
  for (int j = 0; j < kOwn; ++j)
    if (j < own && k0 + j < n) mine += key[j] > least ? 1u : key[j] == least ? 1u << 16 : 0u;
  uint32_t before, total;
  __syncthreads();  // the last counts have been read
  scan_cta(mine, sums[0], before, total);
  const int32_t want = p.top - static_cast<int32_t>(total & 0xFFFFu);  // of the equal ones
  int32_t equals = before >> 16, at = (before & 0xFFFFu) + min(equals, want);
#pragma unroll
  for (int j = 0; j < kOwn; ++j)
    if (j < own && k0 + j < n && (key[j] > least || (key[j] == least && equals++ < want))) out[at++] = ids[j];
}

// Pages of a thread, to a multiple of 4.
__device__ __forceinline__ int32_t own_pages(int32_t n) { return ((n + kListThreads - 1) / kListThreads + 3) / 4 * 4; }

__global__ void __launch_bounds__(kListThreads) list_kernel(const __grid_constant__ Select p) {
  const int32_t row = static_cast<int32_t>(blockIdx.x / p.c.kv_heads), head = blockIdx.x % p.c.kv_heads;
  const Seen x = look_up(p, row);
  const int32_t n = x.pages;
  const bool whole = n <= p.top, many = n > kOwn * kListThreads;
  const int32_t own = many ? 0 : own_pages(n), k0 = threadIdx.x * own;
  int32_t ids[kOwn];
  if (!whole && !many) {
#pragma unroll
    for (int j = 0; j < kOwn; ++j) ids[j] = j < own && k0 + j < n ? x.table[k0 + j] : -1;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (head == 0 && threadIdx.x == 0) p.lens[row] = x.tokens;
  int32_t* out = p.pages + static_cast<int64_t>(blockIdx.x) * p.top;
  if (whole) return list_all(p, x, out);
  const uint32_t* from = p.keys + static_cast<int64_t>(blockIdx.x) * p.stride;
  if (many) return list_long(p, from, x.table, n, out);
  list_short<kOwn>(p, from, n, own, ids, out);
}

// All of it in one launch, a CTA a row and head (a list), or for few lists of many
// pages a cluster of CTAs, which bring their keys together in the first one's shared
// memory.  Rows of one request read its bounds each for itself, and a CTA's few warps
// read all of a table, so that many pages are better spread over three launches,
// where up to 16 rows share what is read; unless lists of their own bounds fill the SMs.
//
// Lengths are on the device, so tables' width, lists and rows choose.  Measured with 8
// heads of 128 dimensions, bounds from memory (what other layers read comes between a
// layer's calls), requests as long as the tables, us of three launches / one / clusters:
//   pages                 128             256             320             400             640            1000
//   rows, one a request
//   4 (32 lists)     11.2/ 9.2/ 8.9  12.1/13.0/ 9.5  12.2/15.0/ 9.7  12.3/17.7/ 9.7  13.3/23.8/12.0  13.9/33.7/12.3
//   8                11.5/ 9.3/ 9.9  12.5/13.3/10.9  12.7/15.0/11.2  13.0/18.0/11.4  14.3/24.2/13.7  17.7/33.9/14.4
//   10               11.8/ 9.4/11.0  12.7/13.2/12.1  13.0/15.1/12.4  13.4/18.0/12.6  14.9/24.1/15.7  18.3/34.2/16.4
//   12               12.0/ 9.5/13.3  13.0/13.4/14.5  13.4/15.3/14.9  13.7/18.2/15.2  17.5/24.2/19.0  19.0/34.2/20.4
//   32               13.5/10.5       17.7/14.5       18.3/16.5       19.3/19.5       24.2/26.1       31.8/36.7
//   64               18.4/12.4       23.6/17.0       25.0/19.3       28.2/22.6       37.0/30.0       49.6/41.0
//   rows, six a request
//   48 (384 lists)   14.5/10.9       15.8/14.2       16.0/15.8       16.7/18.2       18.7/24.0       23.5/33.4
//   96               16.9/15.0       19.4/21.5       20.3/24.1       21.5/28.0       26.7/36.7       32.8/52.1
//   384              39.8/38.3       50.5/56.2       53.7/63.9       58.7/75.3       75.5/ 101       97.9/ 142
// Where requests are shorter than the tables one launch gains: lengths of a quarter of
// the width to all, 96 rows of six 18.9/18.3 at 320 pages, 20.5/22.4 at 512, 21.6/24.8
// at 640, lengths from 0 on 19.4/15.9, 20.9/20.5, 21.6/23.9; and where the bounds are
// still in the L2: 8 rows 10.6/ 9.6/10.4 at 256, 11.3/11.9/11.0 at 400; 48 of six over
// a quarter to all 14.4/12.1 at 320, 15.7/16.8 at 640.  Over all of these lengths, from
// memory and from the L2, 3 to 40 rows a request, one launch takes 0.93 of the three's
// time at 400 pages, 1.00 at 512, 1.02 at 563, 1.09 at 640.  Clusters end where their
// threads hold 16 keys each, as the list's kernel does: at 2048 pages 8 lists 13.2/15.0
// from memory and 11.5/11.4 from the L2, 64 lists 22.7/19.8 and 18.5/17.4.
constexpr int kPickPages = 128;            // one launch, however many lists
constexpr int kPickSingle = 320;           // where each row is a request's only one, the same
constexpr int kPickMost = 1024;            // and this with kPickFull lists and half as many as pages
constexpr int64_t kPickFull = 256;
constexpr int kPickShared = 576;           // where it is not, with less to read than
constexpr int64_t kPickReads = 1 << 20;    //   these records by all lists and, above kPickSingle pages,
constexpr int64_t kPickRecords = 1 << 16;  //   these of all tables
constexpr int kCluster = 8;
constexpr int kClusterPages = 2048;
constexpr int64_t kClusterLists = 80;      // of more than kClusterFewPages pages
constexpr int kClusterFewPages = 256;
constexpr int64_t kClusterFewLists = 32;   // of more than kPickPages

template <int kDim, bool kBf16, int kCtas>
__global__ void __launch_bounds__(kListThreads, 5) pick_kernel(const __grid_constant__ Select p) {
  constexpr int kPages = kCtas == 1 ? kPickMost : kClusterPages;
  constexpr int kStep = kCtas * kListWarps * kScorePages;
  __shared__ __align__(16) uint32_t keys[kPages];
  __shared__ __align__(16) uint8_t parts[2 * kDim];
  const int tid = threadIdx.x, warp = tid >> 5;
  const int rank = kCtas == 1 ? 0 : blockIdx.x % kCtas;
  const int32_t list = blockIdx.x / kCtas, row = list / p.c.kv_heads, head = list % p.c.kv_heads;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Seen x = look_up(p, row);
  const int32_t n = x.pages;
  if (head == 0 && rank == 0 && tid == 0) p.lens[row] = x.tokens;
  int32_t* out = p.pages + static_cast<int64_t>(list) * p.top;
  if (n <= p.top) {
    if (rank == 0) list_all(p, x, out);
    return;
  }
  if (kCtas > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int32_t first = (rank * kListWarps + warp) * kScorePages;
  Scorer<kDim> scorer;
  scorer.load(p, head, x.table + first, n - first);
  if (warp == kListWarps - 1) make_parts<kDim, kBf16>(p, row, head, parts);
  __syncthreads();
  if (kCtas > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // all of the cluster have begun
  const uint32_t to = ptx::dsmem_addr(keys, 0);
  const uint4 q = *reinterpret_cast<const uint4*>(&parts[16 * scorer.piece]);
  for (int32_t page0 = first; page0 < n; page0 += kStep) {
    const Scorer<kDim> now = scorer;
    if (page0 + kStep < n) scorer.load(p, head, x.table + page0 + kStep, n - page0 - kStep);
    const uint32_t key = now.key(q);
    if (now.has() && page0 + now.mine < n) {
      if (kCtas == 1) keys[page0 + now.mine] = key;
      else asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to + 4 * (page0 + now.mine)), "r"(key) : "memory");
    }
  }
  constexpr int kMost = kPages / kListThreads < 8 ? 8 : kPages / kListThreads;  // own_pages(kPages)
  static_assert(kMost * kListThreads >= kPages, "a thread's pages");
  const int32_t own = own_pages(n), k0 = tid * own;
  int32_t ids[kMost];
  if (rank == 0) {
#pragma unroll
    for (int j = 0; j < kMost; ++j) ids[j] = j < own && k0 + j < n ? x.table[k0 + j] : -1;
  }
  if (kCtas == 1) __syncthreads();
  else ptx::cluster_sync();
  if (rank == 0) list_short<kMost>(p, keys, n, own, ids, out);
}

template <typename Kernel>
cudaError_t launch_cluster(Kernel kernel, unsigned lists, cudaStream_t stream, const Select& p) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(lists * kCluster);
  cfg.blockDim = dim3(kListThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCluster, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

SmemAttr g_list_attr;

int64_t key_stride(const Batch& s) { return (static_cast<int64_t>(s.max_pages) + 3) / 4 * 4; }

int check_bounds(const Cache& c, int32_t dim, const void* bounds, int64_t stride) {
  if (stride < static_cast<int64_t>(c.kv_heads) * (2 * dim + 16) || (!bounds && c.num_pages > 0))
    return DSPARK_ERR_INVALID_ARG;
  return aligned(bounds, 16) && stride % 16 == 0 ? DSPARK_OK : DSPARK_ERR_MISALIGNED;
}

int check_selection(const dspark_kv4_selection* x) {
  if (!x || x->rows < 0 || x->top < 1 || (x->rows > 0 && (!x->pages || !x->lens))) return DSPARK_ERR_INVALID_ARG;
  return aligned(x->pages, 4) && aligned(x->lens, 4) ? DSPARK_OK : DSPARK_ERR_MISALIGNED;
}

enum class Launches { kThree, kOne, kClusters };
Launches choose_launches(const Batch& s, int64_t lists, int32_t heads) {
  const int32_t pages = s.max_pages;
  if (pages <= kClusterPages && pages > kPickPages &&
      lists <= (pages > kClusterFewPages ? kClusterLists : kClusterFewLists))
    return Launches::kClusters;
  if (pages <= kPickPages) return Launches::kOne;
  if (s.total_rows <= s.batch)
    return pages <= kPickSingle || (pages <= kPickMost && lists >= kPickFull && 2 * lists >= pages) ? Launches::kOne
                                                                                                     : Launches::kThree;
  const bool few = pages <= kPickSingle || static_cast<int64_t>(s.batch) * heads * pages <= kPickRecords;
  return pages <= kPickShared && lists * pages <= kPickReads && few ? Launches::kOne : Launches::kThree;
}

}  // namespace
}  // namespace kv4
}  // namespace dspark

extern "C" {

int dspark_kv4_bound_pages(const dspark_kv4_cache* cache, const dspark_kv4_batch* batch, void* bounds,
                           int64_t bounds_stride, cudaStream_t stream) {
  using namespace dspark::kv4;
  Cache c;
  Batch s;
  int rc = make_cache(cache, &c);
  if (rc == DSPARK_OK) rc = make_batch(batch, c, &s);
  if (rc == DSPARK_OK) rc = check_bounds(c, cache->head_dim, bounds, bounds_stride);
  if (rc != DSPARK_OK) return rc;
  if (s.batch == 0 || s.total_rows == 0 || c.num_pages == 0) return DSPARK_OK;
  const auto to = static_cast<uint8_t*>(bounds);
  const bool wide = cache->head_dim == 128;
  int32_t rows = s.total_rows / (152 * 4);
  cudaError_t e;
  if (rows < 1) {
    e = launch_behind(wide ? bound_one_kernel<128> : bound_one_kernel<64>,
                      dim3(static_cast<unsigned>(s.total_rows) * c.kv_heads), 32 * kOneWarps, 0, stream, c, s, to,
                      bounds_stride);
  } else {
    rows = rows > 32 ? 32 : rows;
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(s.total_rows) + rows - 1) / rows);
    e = launch_behind(wide ? bound_kernel<128> : bound_kernel<64>, dim3(grid), 32 * kBoundWarps, 0, stream, c, s, to,
                      bounds_stride, rows);
  }
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

size_t dspark_kv4_select_workspace_bytes(const dspark_kv4_cache* cache, const dspark_kv4_batch* batch,
                                         const dspark_kv4_selection* selection) {
  using namespace dspark::kv4;
  Cache c;
  Batch s;
  if (make_cache(cache, &c) != DSPARK_OK || make_batch(batch, c, &s) != DSPARK_OK ||
      check_selection(selection) != DSPARK_OK)
    return 0;
  const int64_t lists = static_cast<int64_t>(s.total_rows) * c.kv_heads;
  const int64_t bytes = s.max_pages > selection->top ? key_stride(s) * 4 + 2 * cache->head_dim : 0;
  return static_cast<size_t>(lists) * bytes + 256;  // never empty
}

int dspark_kv4_select(const dspark_kv4_cache* cache, const dspark_kv4_batch* batch, const void* bounds,
                      int64_t bounds_stride, const dspark_kv4_selection* selection, const dspark_kv4_select_args* args,
                      cudaStream_t stream) {
  using namespace dspark::kv4;
  Select p{};
  int rc = make_cache(cache, &p.c);
  if (rc == DSPARK_OK) rc = make_batch(batch, p.c, &p.s);
  if (rc == DSPARK_OK) rc = check_bounds(p.c, cache->head_dim, bounds, bounds_stride);
  if (rc == DSPARK_OK) rc = check_selection(selection);
  if (rc != DSPARK_OK) return rc;
  if (!args || (args->dtype != DSPARK_DTYPE_BF16 && args->dtype != DSPARK_DTYPE_F16)) return DSPARK_ERR_INVALID_ARG;
  if (args->q_heads < 1 || args->q_heads > kMostQueryHeads || args->q_heads % p.c.kv_heads != 0 || args->q_row < 0 ||
      args->q_head < 0)
    return DSPARK_ERR_INVALID_ARG;
  if (args->first < 0 || args->last < 1 || args->first > selection->top - args->last) return DSPARK_ERR_INVALID_ARG;
  if (selection->rows != p.s.total_rows) return DSPARK_ERR_INVALID_ARG;
  const int64_t lists = static_cast<int64_t>(p.s.total_rows) * p.c.kv_heads;
  if (lists > 0x7FFFFFFF || static_cast<int64_t>(p.s.total_rows) * args->q_heads > 0x7FFFFFFF)
    return DSPARK_ERR_INVALID_ARG;
  if (p.s.total_rows == 0) return DSPARK_OK;
  if (p.s.batch == 0) {  // rows of no request
    const size_t ids = static_cast<size_t>(lists) * selection->top;
    return cudaMemsetAsync(selection->lens, 0xFF, sizeof(int32_t) * p.s.total_rows, stream) == cudaSuccess &&
                   cudaMemsetAsync(selection->pages, 0xFF, sizeof(int32_t) * ids, stream) == cudaSuccess
               ? DSPARK_OK
               : DSPARK_ERR_CUDA;
  }
  if (!args->q || !args->workspace ||
      args->workspace_bytes < dspark_kv4_select_workspace_bytes(cache, batch, selection))
    return DSPARK_ERR_INVALID_ARG;
  if (!aligned(args->q, 2) || !aligned(args->workspace, 256)) return DSPARK_ERR_MISALIGNED;
  p.bounds = static_cast<const uint8_t*>(bounds);
  p.bounds_stride = bounds_stride;
  p.q = static_cast<const uint16_t*>(args->q);
  p.q_row = args->q_row, p.q_head = args->q_head;
  p.group = args->q_heads / p.c.kv_heads;
  p.vec = aligned(args->q, 16) && args->q_row % 8 == 0 && args->q_head % 8 == 0;
  p.first = args->first, p.last = args->last, p.top = selection->top;
  p.pages = selection->pages, p.lens = selection->lens;
  p.keys = static_cast<uint32_t*>(args->workspace);
  p.stride = key_stride(p.s);
  p.parts = static_cast<uint8_t*>(args->workspace) + lists * p.stride * 4;
  const bool wide = cache->head_dim == 128, bf16 = args->dtype == DSPARK_DTYPE_BF16;
  const dim3 grid(static_cast<unsigned>(lists));
  const Launches launches = choose_launches(p.s, lists, p.c.kv_heads);
  cudaError_t e = cudaSuccess;
  if (p.s.max_pages <= p.top) {  // nothing to choose from
    list_kernel<<<grid, kListThreads, 0, stream>>>(p);
    e = cudaGetLastError();
  } else if (launches == Launches::kClusters) {
    const auto pick = wide ? (bf16 ? pick_kernel<128, true, kCluster> : pick_kernel<128, false, kCluster>)
                           : (bf16 ? pick_kernel<64, true, kCluster> : pick_kernel<64, false, kCluster>);
    e = launch_cluster(pick, static_cast<unsigned>(lists), stream, p);
  } else if (launches == Launches::kOne) {
    const auto pick = wide ? (bf16 ? pick_kernel<128, true, 1> : pick_kernel<128, false, 1>)
                           : (bf16 ? pick_kernel<64, true, 1> : pick_kernel<64, false, 1>);
    e = launch_behind(pick, grid, kListThreads, 0, stream, p);
  } else {
    const int32_t most = p.s.max_pages < kListKeys ? p.s.max_pages : kListKeys;
    const int list_smem = p.s.max_pages > kOwn * kListThreads ? most * 4 : 0;
    if (list_smem > 0 && !smem_attr_ready(g_list_attr, list_kernel, kListKeys * 4)) return DSPARK_ERR_CUDA;
    const auto parts = wide ? (bf16 ? parts_kernel<128, true> : parts_kernel<128, false>)
                            : (bf16 ? parts_kernel<64, true> : parts_kernel<64, false>);
    e = launch_behind(parts, dim3(static_cast<unsigned>((lists + kPartWarps - 1) / kPartWarps)), 32 * kPartWarps, 0,
                      stream, p);
    // as many items as the batch could have, or what fills the SMs
    const int64_t page_parts = (static_cast<int64_t>(p.s.max_pages) + kScorePages - 1) / kScorePages;
    const int64_t items = (p.s.total_rows / kScoreRows + static_cast<int64_t>(p.s.batch)) * page_parts * p.c.kv_heads;
    const int64_t ctas = (items + kScoreThreads / 32 - 1) / (kScoreThreads / 32);
    const unsigned score_grid = static_cast<unsigned>(ctas < 152 * kScoreCtas ? ctas : 152 * kScoreCtas);
    const int smem = (p.s.batch + 1) * static_cast<int>(sizeof(int64_t));
    if (e == cudaSuccess)
      e = launch_behind(wide ? score_kernel<128> : score_kernel<64>, dim3(score_grid), kScoreThreads, smem, stream, p);
    if (e == cudaSuccess) e = launch_behind(list_kernel, grid, kListThreads, list_smem, stream, p);
  }
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

}  // extern "C"
