// kv4_attn.cuh -- what the attention kernels over the paged 4-bit cache share
// (kv4_rows.cu, kv4_attention.cu): parameters, the division of the work, and
// the layout of the workspace.
//
// A unit is one tile of a request's query rows (row r of a request's tile
// grid is query r / group, head r % group of the key/value head's group) with
// one key/value head; it reads a run of 64-token blocks of the request's
// cache.  The units' blocks are numbered through (request, tile, head, block)
// and every CTA takes an equal run of them, so that the work is even whatever
// the lengths are; a unit that is cut by a run's end leaves partial sums in
// the workspace, which a second kernel joins in order.
#pragma once

#include "kv4.cuh"

namespace dspark {
namespace kv4 {

constexpr int kBlock = 64;  // tokens of a block
constexpr int kMaxGrid = 256;  // CTAs that may leave partial sums
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNone = -1e30f;  // the running maximum of a row that saw nothing

struct Attn {
  Cache c;
  Batch s;
  const uint16_t* q;
  int64_t q_row, q_head;
  uint16_t* out;
  int64_t out_row, out_head;
  float* lse;
  int32_t heads;  // key/value heads
  int32_t group;
  int32_t window;
  int32_t bf16;
  int32_t q_vec;    // 16-byte loads of q
  int32_t out_vec;  // 16-byte stores of out
  float scale_log2;  // scale * log2(e)
  int32_t* prefix;   // workspace: [batch + 1] blocks before each request
  float* partials;   // workspace: [2 * grid] slots
};

// Shared by both kernels: rows of a tile, blocks of a unit.
struct Tile {
  int32_t lo, hi;    // blocks
  int32_t p0, p1;    // positions of its first and last query
};

// Tile `t` of `kRows` rows of request r.
template <int kRows>
__device__ __forceinline__ Tile make_tile(const Attn& a, const Request& r, int32_t t) {
  Tile x;
  const int32_t rows = r.rows * a.group;
  const int32_t first = t * kRows, last = min(first + kRows, rows) - 1;
  x.p0 = r.len - r.rows + first / a.group;
  x.p1 = r.len - r.rows + last / a.group;
  if (x.p1 < 0) {
    x.lo = x.hi = 0;
    return x;
  }
  x.hi = x.p1 / kBlock + 1;
  x.lo = a.window > 0 ? max(0, x.p0 - a.window + 1) / kBlock : 0;
  return x;
}

template <int kRows>
__device__ __forceinline__ int32_t num_tiles(const Attn& a, const Request& r) {
  return static_cast<int32_t>((static_cast<int64_t>(r.rows) * a.group + kRows - 1) / kRows);
}

// Blocks of all units of request r.
template <int kRows>
__device__ __forceinline__ int32_t request_blocks(const Attn& a, const Request& r) {
  int64_t n = 0;
  if (r.len <= 0) return 0;
  const int32_t tiles = num_tiles<kRows>(a, r);
  for (int32_t t = 0; t < tiles; ++t) {
    const Tile x = make_tile<kRows>(a, r, t);
    n += x.hi - x.lo;
  }
  n *= a.heads;
  return static_cast<int32_t>(n < 0x7FFFFFFF ? n : 0x7FFFFFFF);
}

// Blocks of a CTA's run: at least `least`, so that a small call does not pay
// for joining more parts than its blocks are worth.
__device__ __forceinline__ int32_t run_length(int32_t total, int grid, int32_t least) {
  const int32_t n = total / grid + (total % grid != 0 ? 1 : 0);
  return max(n, least);
}

// Walks the units of a run of blocks.
template <int kRows>
struct Walk {
  const Attn& a;
  const int32_t* prefix;
  int32_t b, tile, tiles, head;
  Tile x;
  Request r;

  __device__ __forceinline__ Walk(const Attn& a_, const int32_t* prefix_) : a(a_), prefix(prefix_) {}

  // To the unit with block number `at`; returns its offset in the unit.
  __device__ __forceinline__ int32_t seek(int32_t at) {
    int32_t lo = 0, hi = a.s.batch;
    while (hi - lo > 1) {
      const int32_t mid = (lo + hi) >> 1;
      if (prefix[mid] <= at) lo = mid;
      else hi = mid;
    }
    b = lo;
    r = load_request(a.s, b);
    tiles = num_tiles<kRows>(a, r);
    int32_t rem = at - prefix[b];
    for (tile = 0; tile < tiles; ++tile) {
      x = make_tile<kRows>(a, r, tile);
      const int32_t n = (x.hi - x.lo) * a.heads;
      if (rem < n) {
        head = rem / (x.hi - x.lo);
        return rem - head * (x.hi - x.lo);
      }
      rem -= n;
    }
    return 0;
  }

  // To the next unit that has blocks; there is one.
  __device__ __forceinline__ void next() {
    if (++head < a.heads) return;
    head = 0;
    for (;;) {
      if (++tile >= tiles) {
        do {
          ++b;
        } while (b + 1 < a.s.batch && prefix[b + 1] == prefix[b]);
        r = load_request(a.s, b);
        tiles = num_tiles<kRows>(a, r);
        tile = 0;
      }
      x = make_tile<kRows>(a, r, tile);
      if (x.hi > x.lo || (b + 1 >= a.s.batch && tile + 1 >= tiles)) return;
    }
  }
};

// The prefix sums of the requests' blocks, by a whole CTA of kThreads threads
// into shared memory ([batch + 1]); CTA 0 leaves them in the workspace.
template <int kRows, int kThreads>
__device__ __forceinline__ void plan(const Attn& a, int32_t* prefix, int32_t* scratch /* [kThreads / 32 + 1] */) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t per = (a.s.batch + kThreads - 1) / kThreads;
  const int32_t lo = min(tid * per, a.s.batch), hi = min(lo + per, a.s.batch);
  int32_t sum = 0;
  for (int32_t i = lo; i < hi; ++i) {
    const int32_t n = request_blocks<kRows>(a, load_request(a.s, i));
    prefix[i] = n;
    sum += n;
  }
  int32_t incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t u = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += u;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  int32_t at = incl - sum;
  for (int w = 0; w < warp; ++w) at += scratch[w];
  for (int32_t i = lo; i < hi; ++i) {
    const int32_t n = prefix[i];
    prefix[i] = at;
    if (blockIdx.x == 0) a.prefix[i] = at;
    at += n;
  }
  if (tid == kThreads - 1) {
    prefix[a.s.batch] = at;
    if (blockIdx.x == 0) a.prefix[a.s.batch] = at;
  }
  __syncthreads();
}

// Workspace: the prefix sums, then slots of kRows rows: the unnormalised sums
// [kRows][kDim], the maxima [kRows] and the totals [kRows] (log2 units).
__host__ __device__ __forceinline__ int64_t workspace_header(int32_t batch) {
  return (static_cast<int64_t>(batch + 1) * 4 + 255) / 256 * 256;
}
template <int kRows, int kDim>
__host__ __device__ __forceinline__ constexpr int64_t slot_floats() {
  return kRows * (kDim + 2);
}

__device__ __forceinline__ uint32_t pack_out(bool bf16, float lo, float hi) {
  return bf16 ? ptx::cvt_bf16x2(lo, hi) : cvt_f16x2(lo, hi);
}

constexpr int kRowsTile = 16;  // the most rows of a tile of the small kernel
cudaError_t launch_rows(const Attn& a, int dim, int32_t max_rows, int grid, cudaStream_t stream);

}  // namespace kv4
}  // namespace dspark
