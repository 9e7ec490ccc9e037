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
constexpr int kMaxGrid = 160;  // CTAs that may leave partial sums
// Registers a thread that the attention kernels of 512 threads are launched
// with, all of an SM's: one CTA runs on an SM, and may take all of its tensor
// memory.  Their warpgroups' shares come out of these.
constexpr int kLaunchRegs = 128;
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNone = -1e30f;  // the running maximum of a row that saw nothing

// A unit that starts in a run and does not end there, for the kernel that joins
// its parts: how many runs it spans (0: none is cut, -1: the call is too long),
// the request's first row, the tile's first row and how many it has, the
// key/value head.
struct alignas(16) Cut {
  int32_t parts, start, first, rows, head, pad[3];
};

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
  int32_t window;   // below the tokens that a request can have; 0: none
  int32_t bf16;
  int32_t q_vec;    // 16-byte loads of q
  int32_t out_vec;  // 16-byte stores of out
  int32_t many_tiles;  // requests may have more than one tile of rows
  float scale_log2;  // scale * log2(e)
  Cut* cuts;         // workspace: [kMaxGrid] the unit that each run's end cuts
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
  const int32_t first = t * kRows, last = first + min(rows - first, kRows) - 1;
  x.p0 = r.len - r.rows + first / a.group;
  x.p1 = r.len - r.rows + last / a.group;
  if (x.p1 < 0) {
    x.lo = x.hi = 0;
    return x;
  }
  x.hi = x.p1 / kBlock + 1;
  x.lo = a.window > 0 ? max(0, max(0, x.p0) - a.window + 1) / kBlock : 0;  // p0 may be far below 0
  return x;
}

template <int kRows>
__device__ __forceinline__ int32_t num_tiles(const Attn& a, const Request& r) {
  return static_cast<int32_t>((static_cast<int64_t>(r.rows) * a.group + kRows - 1) / kRows);
}

// What the start and the end of a unit (queries, sums, results) take, in blocks.
// The runs are cut along a line on which each unit has as many positions in front
// of its blocks' ones, so that a CTA with many short units gets fewer blocks.
// Measured, with 0 / 3 / 5 / 7 / 10 positions for the larger tiles: 48
// verifications of 6 rows over 1 to 8 k tokens 147 / 136 / 131 / 126 / 125 us, 23
// requests of 0 to 133 rows over up to 3001 tokens 54 / 45 / 44 / 45 / 46; with 0 /
// 2 / 4 / 5 / 8 for the smaller ones: 64 single tokens over 4 to 16 k tokens 145 /
// 142 / 139 / 139 / 138, one over 2 k 12.3 / 12.1 / 10.0 / 10.1 / 10.9.
template <int kRows>
__host__ __device__ constexpr int32_t unit_lead() {
  return kRows >= 128 ? 7 : 5;
}

// Positions are counted in 31 bits, with room behind the last one for a unit's
// lead.  The host takes tiles large enough that a call's cannot be more
// (kv4_attention.cu); where none is, sums stay at kTooMany, and a call whose line
// is that long gives NaN.
constexpr int32_t kTooMany = 0x7FFFFF00;
__device__ __forceinline__ int32_t add_positions(int32_t a, int32_t b) {
  return static_cast<int32_t>(min(static_cast<uint32_t>(a) + static_cast<uint32_t>(b), static_cast<uint32_t>(kTooMany)));
}

// Positions of tile t's units of request r, all heads (0 behind its tiles).
template <int kRows>
__device__ __forceinline__ int32_t tile_positions(const Attn& a, const Request& r, int32_t t, int32_t tiles) {
  if (t >= tiles || r.len <= 0) return 0;
  const Tile x = make_tile<kRows>(a, r, t);
  if (x.hi <= x.lo) return 0;
  const uint32_t unit = x.hi - x.lo + unit_lead<kRows>(), heads = a.heads;
  return __umulhi(unit, heads) != 0 ? kTooMany : static_cast<int32_t>(min(unit * heads, static_cast<uint32_t>(kTooMany)));
}

__device__ __forceinline__ int32_t scan_positions(int32_t v) { return scan_warp(v, add_positions); }

// Positions of a CTA's run: more than a unit's lead, so that each run has a
// block.
template <int kRows>
__device__ __forceinline__ int32_t run_length(int32_t total, int grid) {
  const int32_t n = total / grid + (total % grid != 0 ? 1 : 0);
  return max(n, unit_lead<kRows>() + 1);
}

// Walks the units of a run.
template <int kRows>
struct Walk {
  static constexpr int32_t kLead = unit_lead<kRows>();
  const Attn& a;
  const int32_t* prefix;
  int32_t b, tile, tiles, head;
  int32_t lead;  // positions from where seek went to the unit's first block, or 0
  Tile x;
  Request r;

  __device__ __forceinline__ Walk(const Attn& a_, const int32_t* prefix_) : a(a_), prefix(prefix_) {}

  // To the unit with position `at`; returns how many of its blocks lie before.
  // The whole warp searches, a tile a lane.
  __device__ __forceinline__ int32_t seek(int32_t at) {
    const int lane = threadIdx.x & 31;
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
    for (int32_t base = 0; base < tiles; base += 32) {
      const int32_t n = tile_positions<kRows>(a, r, base + lane, tiles), upto = scan_positions(n);
      const uint32_t here = __ballot_sync(0xFFFFFFFFu, rem < upto);
      if (here != 0) {
        const int l = __ffs(here) - 1;
        rem -= __shfl_sync(0xFFFFFFFFu, upto - n, l);
        tile = base + l;
        x = make_tile<kRows>(a, r, tile);
        head = rem / (x.hi - x.lo + kLead);
        const int32_t in_unit = rem - head * (x.hi - x.lo + kLead);
        lead = max(kLead - in_unit, 0);
        return max(in_unit - kLead, 0);
      }
      rem -= __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    tile = 0, head = 0, lead = 0;  // not reached: `at` is below the number of positions
    x = make_tile<kRows>(a, r, 0);
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

// The prefix sums of the requests' positions, by a whole CTA of kThreads threads
// into shared memory ([batch + 1]).  A request of one tile takes a thread, one
// of many a warp.
template <int kRows, int kThreads>
__device__ __forceinline__ void plan(const Attn& a, int32_t* prefix, int32_t* scratch /* [kThreads / 32 + 1] */) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t per = (a.s.batch + kThreads - 1) / kThreads;
  const int32_t lo = min(tid * per, a.s.batch), hi = min(lo + per, a.s.batch);
  if (a.many_tiles) {
    for (int32_t i = warp; i < a.s.batch; i += kThreads / 32) {
      const Request r = load_request(a.s, i);
      const int32_t tiles = num_tiles<kRows>(a, r);
      int32_t n = 0;
      for (int32_t t = lane; t < tiles; t += 32) n = add_positions(n, tile_positions<kRows>(a, r, t, tiles));
      n = __shfl_sync(0xFFFFFFFFu, scan_positions(n), 31);
      if (lane == 0) prefix[i] = n;
    }
    __syncthreads();
  } else {
    for (int32_t i = lo; i < hi; ++i) {
      const Request r = load_request(a.s, i);
      const int32_t tiles = num_tiles<kRows>(a, r);
      int32_t n = 0;
      for (int32_t t = 0; t < tiles; ++t) n = add_positions(n, tile_positions<kRows>(a, r, t, tiles));
      prefix[i] = n;  // read again by this thread
    }
  }
  int32_t sum = 0;
  for (int32_t i = lo; i < hi; ++i) sum = add_positions(sum, prefix[i]);
  const int32_t incl = scan_positions(sum);
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  int32_t at = __shfl_up_sync(0xFFFFFFFFu, incl, 1);  // what the lanes before hold, then the warps before
  if (lane == 0) at = 0;
  for (int w = 0; w < warp; ++w) at = add_positions(at, scratch[w]);
  for (int32_t i = lo; i < hi; ++i) {
    const int32_t n = prefix[i];
    prefix[i] = at;
    at = add_positions(at, n);
  }
  if (tid == kThreads - 1) prefix[a.s.batch] = at;
  __syncthreads();
}

// Workspace: the cuts, then two slots a CTA, of kRows rows: the unnormalised sums
// [kRows][kDim], the maxima [kRows] and the totals [kRows] (log2 units).
template <int kRows, int kDim>
__host__ __device__ __forceinline__ constexpr int64_t slot_floats() {
  return kRows * (kDim + 2);
}
constexpr int64_t kCutBytes = kMaxGrid * sizeof(Cut);
static_assert(kCutBytes % 256 == 0, "slots start on 256 bytes");

// Says for CTA blockIdx.x which unit its run's end cuts: the last one of the run,
// at `walk`, of which `left` blocks lie behind the run (0: none is cut, or the
// unit did not start here).
template <typename Walk>
__device__ __forceinline__ void leave_cut(const Attn& a, const Walk& walk, int32_t left, int32_t run, int32_t first,
                                          int32_t rows) {
  Cut c{};
  c.parts = left > 0 ? 2 + (left - 1) / run : 0;
  c.start = walk.r.start;
  c.first = first;
  c.rows = rows;
  c.head = walk.head;
  a.cuts[blockIdx.x] = c;
}
__device__ __forceinline__ void leave_no_cut(const Attn& a, int32_t total) {
  if (threadIdx.x == 0) a.cuts[blockIdx.x].parts = total == kTooMany ? -1 : 0;
}

// ---- waits, copies ----------------------------------------------------------
constexpr uint32_t kPolls = 1u << 20;
// Weights are 2^(x - m + kShift) and the maximum m moves only when a row
// exceeds it by kSlack: at most 2^13 in FP16, and nothing above 2^-30 of the
// row's largest weight is lost to FP16's smallest number.
constexpr float kShift = 5.0f;
constexpr float kSlack = 8.0f;

// Waits for up to three barriers.  Every lane polls all of them (a phase is
// seen by those who have waited for it), and the polls are in flight together:
// one costs about 100 cycles even where the phase is over.  The answer is the
// warp's: false after too many polls, here or in another warp of the CTA.  A
// phase that is not wanted (the same for the whole warp) counts as over.
struct Phase {
  uint64_t* bar;
  uint32_t parity;
  uint32_t wanted;
  __device__ __forceinline__ Phase(uint64_t* b, uint32_t number, bool want = true)
      : bar(b), parity(number & 1), wanted(want ? 1u : 0u) {}
};
template <typename Poll>
__device__ __forceinline__ bool wait_until(Poll poll, volatile int32_t* gave_up) {
  for (uint32_t i = 0; i < kPolls; ++i) {
    if (__all_sync(0xFFFFFFFFu, poll())) return true;
    if ((i & 63u) == 63u && __any_sync(0xFFFFFFFFu, *gave_up != 0)) return false;
  }
  *gave_up = 1;
  return false;
}
__device__ __forceinline__ bool wait_for(const Phase& a, const Phase& b, const Phase& c, volatile int32_t* gave_up) {
  const uint32_t want = a.wanted | b.wanted << 1 | c.wanted << 2;
  return wait_until(
      [&] { return (ptx::mbar_try_wait3(a.bar, a.parity, b.bar, b.parity, c.bar, c.parity) & want) == want; }, gave_up);
}
__device__ __forceinline__ bool wait_for(const Phase& a, const Phase& b, volatile int32_t* gave_up) {
  const uint32_t want = a.wanted | b.wanted << 1;
  return wait_until([&] { return (ptx::mbar_try_wait2(a.bar, a.parity, b.bar, b.parity) & want) == want; }, gave_up);
}
__device__ __forceinline__ bool wait_for(const Phase& a, volatile int32_t* gave_up) {
  return wait_until([&] { return ptx::mbar_try_wait(a.bar, a.parity); }, gave_up);
}

// Where the parts of a block's records are in a ring stage: records of up to
// 64 tokens lie there side by side, whole; of larger pages a 64-token part of
// each section.
struct Stage {
  int tokens, shift;  // of a record's part, and its log2
};
__device__ __forceinline__ Stage make_stage(const Cache& c) {
  return Stage{min(c.page_size, kBlock), c.page_size < kBlock ? c.page_shift : 6};
}

// A producer warp (number `self` of kProducers): brings its blocks of the run
// begin .. end - 1 into the ring, a stage each.  masks[stage] gets which of
// the block's pages are there, and kLastBlock with the run's last one; the
// copies complete on full[stage].
constexpr uint32_t kLastBlock = 1u << 31;
template <int kDim, int kRows, int kStages, int kProducers>
__device__ __forceinline__ void produce(const Attn& a, const int32_t* prefix, int32_t begin, int32_t end, int self,
                                        uint8_t* ring, uint64_t* full, uint64_t* empty, uint32_t* masks,
                                        int32_t* gave_up) {
  const int lane = threadIdx.x & 31;
  constexpr int kStageBytes = kBlock * (kDim + kDim / 8);
  Walk<kRows> walk(a, prefix);
  int32_t skip = walk.seek(begin);
  int32_t behind = self;  // blocks before this warp's next one, from the unit's first on
  int stage = self;       // of that block
  uint32_t lap = 0;
  const int record = Record<kDim>::bytes(a.c.page_size);
  const bool whole = a.c.page_size <= kBlock;
  const int per_block = whole ? kBlock / make_stage(a.c).tokens : 1;  // pages of a block
  const int copies = whole ? per_block : 4;
  bool ok = true;
  for (int32_t at = begin + walk.lead; at < end;) {  // to the end even where a wait gave up: the cut is left there
    const int32_t blk0 = walk.x.lo + skip;
    const int32_t n = min(walk.x.hi - blk0, end - at);
    const bool last = at + n + walk.kLead >= end;  // unit of the run
    const int64_t last_page = (walk.r.len - 1) >> a.c.page_shift;
    int64_t first = 0;   // page number of lane 0's id
    int32_t ids = -1;
    int64_t next = -1;   // first page number behind the ids
    if (self == 0) {  // the unit's queries on their way while its blocks wait in the ring
      const int32_t first_row = walk.tile * kRows, rows = min(walk.r.rows * a.group - first_row, kRows);
      for (int32_t r = lane; r < rows; r += 32) {
        const int32_t i = (first_row + r) / a.group;
        const uint16_t* q = a.q + (walk.r.start + i) * a.q_row + (walk.head * a.group + first_row + r - i * a.group) * a.q_head;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
        if (kDim == 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 64));
      }
      __syncwarp();
    }
    for (; ok && behind < n; behind += kProducers) {
      const int32_t blk = blk0 + behind;
      const int64_t page0 = (static_cast<int64_t>(blk) * kBlock) >> a.c.page_shift;
      if (page0 >= next) {
        first = page0;
        ids = first + lane <= last_page ? walk.r.pages[first + lane] : -1;
        if (ids >= a.c.num_pages) ids = -1;
        next = first + 32;
      }
      if (lap > 0) ok = wait_for(Phase(&empty[stage], lap - 1), gave_up);
      if (!ok) break;
      const int which = whole ? lane : 0;
      const int32_t id = __shfl_sync(0xFFFFFFFFu, ids, static_cast<int>(page0 - first) + (which & (per_block - 1)));
      const bool mine = lane < copies && id >= 0;
      const uint32_t valid = __ballot_sync(0xFFFFFFFFu, mine);
      const int bytes = whole ? __popc(valid) * record : (valid ? kStageBytes : 0);
      if (lane == 0) {
        masks[stage] = (whole ? valid : (valid ? 1u : 0u)) | (last && behind == n - 1 ? kLastBlock : 0u);
        ptx::mbar_arrive_expect_tx(&full[stage], bytes);
      }
      __syncwarp();
      if (mine) {
        const uint8_t* src = a.c.data + static_cast<int64_t>(id) * a.c.page_stride +
                             static_cast<int64_t>(walk.head) * record;
        uint8_t* dst = ring + stage * kStageBytes;
        if (whole) {
          ptx::bulk_load(dst + lane * record, src, record, &full[stage]);
        } else {
          // a 64-token part of the record's four sections
          const int row0 = (blk * kBlock) & (a.c.page_size - 1);
          using R = Record<kDim>;
          const int w = lane & 1;
          if (lane < 2)
            ptx::bulk_load(dst + R::codes(kBlock, w), src + R::codes(a.c.page_size, w) + row0 * R::kCodeBytes,
                           kBlock * R::kCodeBytes, &full[stage]);
          else
            ptx::bulk_load(dst + R::scales(kBlock, w), src + R::scales(a.c.page_size, w) + row0 * R::kScaleBytes,
                           kBlock * R::kScaleBytes, &full[stage]);
        }
      }
      stage += kProducers;
      if (stage >= kStages) stage -= kStages, ++lap;
    }
    behind -= n;
    at += n + walk.kLead;
    if (last && self == 0 && lane == 0) {
      const int32_t first_row = walk.tile * kRows;
      leave_cut(a, walk, skip > 0 ? 0 : walk.x.hi - walk.x.lo - n, end - begin, first_row,
                min(walk.r.rows * a.group - first_row, kRows));
    }
    skip = 0;
    if (at < end) walk.next();
  }
  if (!ok) {  // this warp's copies in flight land before the CTA's memory goes
    for (int i = self; i < kStages; i += kProducers) {
      const uint32_t laps = lap + (i < stage ? 1 : 0);  // copies into stage i so far
      for (uint32_t t = 0;
           t < kPolls && laps > 0 && !ptx::mbar_try_wait(&full[i], (laps - 1) & 1); ++t) {
      }
    }
  }
}

// kN consecutive 16-bit values of a query row, raw, as words of two.
template <int kN>
__device__ __forceinline__ void load_raw(const Attn& a, const uint16_t* p, bool there, uint32_t (&w)[kN / 2]) {
#pragma unroll
  for (int i = 0; i < kN / 2; ++i) w[i] = 0u;
  if (!there) return;
  if (a.q_vec) {
#pragma unroll
    for (int i = 0; i < kN / 8; ++i) {
      const uint4 x = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) w[i] = p[2 * i] | (static_cast<uint32_t>(p[2 * i + 1]) << 16);
  }
}

// The largest magnitude among BF16 words, as its bits.
template <int kN>
__device__ __forceinline__ uint32_t largest(const uint32_t (&w)[kN]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kN; ++i) top = max(top, max(w[i] & 0x7FFFu, w[i] >> 16 & 0x7FFFu));
  return top;
}

// BF16 queries enter the products as FP16 of q 2^e, with the row's largest
// magnitude (bits `top`) in [2^14, 2^15); zeros, infinities and NaN as they
// are.  The shift is held to what 2^e and 2^-e can be as normal numbers.
__device__ __forceinline__ int query_shift(uint32_t top) {
  const int exponent = static_cast<int>(top >> 7);
  const int e = exponent == 0 || exponent == 255 ? 0 : 14 - (exponent - 127);
  return min(max(e, -120), 120);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
template <int kN>
__device__ __forceinline__ void shift_queries(uint32_t (&w)[kN], float up) {
#pragma unroll
  for (int i = 0; i < kN; ++i)
    w[i] = cvt_f16x2(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xFFFF0000u) * up);
}

__device__ __forceinline__ uint32_t pack_out(bool bf16, float lo, float hi) {
  return bf16 ? ptx::cvt_bf16x2(lo, hi) : cvt_f16x2(lo, hi);
}

// Launchers, by the rows of a tile: 8 or 16, and 128 or 256.
cudaError_t launch_rows(const Attn& a, int dim, int32_t tile, int grid, cudaStream_t stream);   // kv4_rows.cu
cudaError_t launch_tiles(const Attn& a, int dim, int32_t tile, int grid, cudaStream_t stream);  // kv4_tiles.cu

}  // namespace kv4
}  // namespace dspark
