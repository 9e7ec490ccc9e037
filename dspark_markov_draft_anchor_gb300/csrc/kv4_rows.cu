// kv4_rows.cu -- attention of few rows over the paged 4-bit cache: the kernel
// for tiles of up to 16 rows (single tokens and short verifications), and the
// kernel that joins partial sums.
//
// out_r = sum_t p_rt v_t / sum_t p_rt, p_rt = 2^(x_rt - m_r), x = scale log2(e) <q_r, k_t>.
// Few rows over a long cache: the cache's bytes bound it (144 bytes a token
// and head at 128 dimensions, for 16 x 512 multiply-adds).  So each byte is
// brought in once, by bulk copies of whole page records into a ring that a
// producer warp keeps full, and is turned into FP16 operands in registers:
// a thread's share of a key row is the B fragment of mma.m16n8k16 as it lies
// (the order of the dimensions under a dot product is free, so each thread
// takes consecutive ones), and the values' codes of two tokens are interleaved
// by two logic operations a word before the conversion, which gives the pairs
// along tokens that the second product wants.  Per token and head a warp
// spends 2 matrix instructions (4 cycles of an SM's tensor pipe), about 6
// conversions and 4 multiplications; the memory takes 6.2 cycles.
#include "kv4_attn.cuh"

namespace dspark {
namespace kv4 {
namespace {

constexpr int kTeams = 3;            // teams of four warps take blocks in turn
constexpr int kWarps = 4 * kTeams;   // consumers
constexpr int kConsumers = 32 * kWarps;
constexpr int kThreadsRows = kConsumers + 128;  // and the producer's warpgroup, of which one warp works
// Registers a thread: the block is launched with 128; 3 x 128 x 152 + 128 x 56 = 512 x 128.
constexpr int kProducerRegs = 56;
constexpr int kConsumerRegs = 152;
constexpr int kLeast = kTeams;       // blocks of a run
constexpr uint32_t kPolls = 1u << 22;
// Weights are 2^(x - m + kShift) and the maximum m moves only when a row
// exceeds it by kSlack: at most 2^13 in FP16, and nothing above 2^-30 of the
// row's largest weight is lost to FP16's smallest number.
constexpr float kShift = 5.0f;
constexpr float kSlack = 8.0f;

template <int kDim>
struct Shape {
  static constexpr int kStages = kDim == 128 ? 10 : 18;
  static constexpr int kStageBytes = kBlock * (kDim + kDim / 8);
  static constexpr int kTiles = kDim / 8;      // n-tiles of the second product
  static constexpr int kSteps = kDim / 16;     // k-steps of the first
  static constexpr int kLane = kDim / 8;       // consecutive dimensions of a thread (second product)
  static constexpr int kGroupStride = kLane + 1;  // padded, in the merge buffer
  static constexpr int kRowStride = 8 * kGroupStride + 1;
  static constexpr int kMergeBytes = kWarps * kRowsTile * kRowStride * 4;
  // ring, merge buffer, maxima and totals, barriers and page masks, prefix sums
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kStats = kRing + kMergeBytes;
  static constexpr int kBars = kStats + 4 * kWarps * kRowsTile * 4;  // two of each, for turns
  static constexpr int kMasks = kBars + 2 * kStages * 8;
  static constexpr int kMisc = kMasks + kStages * 4;
  static constexpr int kPrefix = kMisc + (kThreadsRows / 32 + 3) * 4;
  static int smem(int32_t batch) { return kPrefix + (batch + 1) * 4; }
};

__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, volatile int32_t* gave_up) {
  for (uint32_t i = 0; i < kPolls; ++i) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 63u && *gave_up) return false;
  }
  *gave_up = 1;
  return false;
}

// Column n of an 8-token score tile is token n ^ (n >> 2 & 1): with it the
// shared-memory reads of keys and of values are both free of avoidable bank
// conflicts at 64 and at 32 bytes a token.
__device__ __forceinline__ int token_of(int n) { return n ^ (n >> 2 & 1); }

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// kN consecutive 16-bit values of a query row as FP16 words, scaled by 2^e
// for BF16 (e from the row's largest magnitude over the quad).  Returns 2^-e.
template <int kN>
__device__ __forceinline__ float load_query(const Attn& a, const uint16_t* p, bool there, uint32_t (&w)[kN / 2]) {
#pragma unroll
  for (int i = 0; i < kN / 2; ++i) w[i] = 0u;
  if (there) {
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
  if (!a.bf16) return 1.0f;
  uint32_t top = 0;  // the largest magnitude's bits
#pragma unroll
  for (int i = 0; i < kN / 2; ++i) top = max(top, max(w[i] & 0x7FFFu, w[i] >> 16 & 0x7FFFu));
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
  // to [2^14, 2^15); zeros, infinities and NaN as they are.  The shift is held
  // to what 2^e and 2^-e can be as normal numbers.
  const int exponent = static_cast<int>(top >> 7);
  int e = exponent == 0 || exponent == 255 ? 0 : 14 - (exponent - 127);
  e = min(max(e, -120), 120);
  const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
  for (int i = 0; i < kN / 2; ++i) {
    const float lo = __uint_as_float(w[i] << 16) * up, hi = __uint_as_float(w[i] & 0xFFFF0000u) * up;
    w[i] = cvt_f16x2(lo, hi);
  }
  return __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

template <int kDim>
__global__ void __launch_bounds__(kThreadsRows, 1) rows_kernel(const __grid_constant__ Attn a) {
  using S = Shape<kDim>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBars);
  uint64_t* empty = full + S::kStages;
  uint32_t* masks = reinterpret_cast<uint32_t*>(smem + S::kMasks);
  int32_t* misc = reinterpret_cast<int32_t*>(smem + S::kMisc);
  int32_t* gave_up = misc + kThreadsRows / 32 + 1;
  int32_t* prefix = reinterpret_cast<int32_t*>(smem + S::kPrefix);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      ptx::mbar_init(&full[i], 1);
      ptx::mbar_init(&empty[i], 4);
    }
    ptx::fence_mbar_init();
    *gave_up = 0;
  }
  plan<kRowsTile, kThreadsRows>(a, prefix, misc);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int32_t total = prefix[a.s.batch];
  const int32_t run = run_length(total, gridDim.x, kLeast);
  const int64_t begin64 = static_cast<int64_t>(run) * blockIdx.x;
  if (begin64 >= total) return;
  const int32_t begin = static_cast<int32_t>(begin64);
  const int32_t end = static_cast<int32_t>(begin64 + run < total ? begin64 + run : total);

  // records of up to 64 tokens lie side by side in a stage
  const int sub = min(a.c.page_size, kBlock);  // tokens of a record's part in a stage
  const int sub_shift = a.c.page_size < kBlock ? a.c.page_shift : 6;
  const uint32_t ring = ptx::smem_addr(smem);

  int32_t count = 0;  // blocks of this run so far

  if (warp >= kWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    if (warp > kWarps) return;
    Walk<kRowsTile> walk(a, prefix);
    int32_t skip = walk.seek(begin);
    // ---- producer ----------------------------------------------------------
    const int record = Record<kDim>::bytes(a.c.page_size);
    const bool whole = a.c.page_size <= kBlock;
    const int per_block = whole ? kBlock / sub : 1;  // pages of a block
    const int copies = whole ? per_block : 4;
    bool ok = true;
    for (int32_t at = begin; at < end && ok;) {
      int32_t blk = walk.x.lo + skip;
      const int32_t n = min(walk.x.hi - blk, end - at);
      const int64_t last_page = (walk.r.len - 1) >> a.c.page_shift;
      int64_t first = 0;   // page number of lane 0's id
      int32_t ids = -1;
      int64_t next = -1;   // first page number behind the ids
      for (int32_t i = 0; i < n && ok; ++i, ++blk, ++count) {
        const int64_t page0 = (static_cast<int64_t>(blk) * kBlock) >> a.c.page_shift;
        if (page0 >= next) {
          first = page0;
          ids = first + lane <= last_page ? walk.r.pages[first + lane] : -1;
          if (ids >= a.c.num_pages) ids = -1;
          next = first + 32;
        }
        const int stage = count % S::kStages;
        if (count >= S::kStages) ok = wait_bounded(&empty[stage], (count / S::kStages - 1) & 1, gave_up);
        if (!ok) break;
        const int which = whole ? lane : 0;
        const int32_t id = __shfl_sync(0xFFFFFFFFu, ids, static_cast<int>(page0 - first) + (which & (per_block - 1)));
        const bool mine = lane < copies && id >= 0;
        const uint32_t valid = __ballot_sync(0xFFFFFFFFu, mine);
        const int bytes = whole ? __popc(valid) * record : (valid ? S::kStageBytes : 0);
        if (lane == 0) {
          masks[stage] = whole ? valid : (valid ? 1u : 0u);
          ptx::mbar_arrive_expect_tx(&full[stage], bytes);
        }
        __syncwarp();
        if (mine) {
          const uint8_t* src = a.c.data + static_cast<int64_t>(id) * a.c.page_stride +
                               static_cast<int64_t>(walk.head) * record;
          uint8_t* dst = smem + stage * S::kStageBytes;
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
      }
      at += n;
      skip = 0;
      if (at < end) walk.next();
    }
    if (!ok) {  // copies in flight land before the CTA's memory goes
      for (int32_t i = max(0, count - S::kStages); i < count; ++i)
        for (uint32_t t = 0; t < kPolls && !ptx::mbar_try_wait(&full[i % S::kStages], (i / S::kStages) & 1); ++t) {
        }
    }
    return;
  }

  // ---- consumers -----------------------------------------------------------
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
  Walk<kRowsTile> walk(a, prefix);
  int32_t skip = walk.seek(begin);
  const int g = lane >> 2, t = lane & 3;
  const int team = warp >> 2, part = (warp & 3) * 16;  // 16 tokens of a block
  using R = Record<kDim>;
  const uint32_t rec = ring + (part >> sub_shift) * (sub * (kDim + kDim / 8));
  const int row0 = part & (sub - 1);
  const uint32_t k_codes = rec + R::codes(sub, 0) + row0 * R::kCodeBytes;
  const uint32_t v_codes = rec + R::codes(sub, 1) + row0 * R::kCodeBytes;
  const uint32_t k_scales = rec + R::scales(sub, 0) + row0 * R::kScaleBytes;
  const uint32_t v_scales = rec + R::scales(sub, 1) + row0 * R::kScaleBytes;
  const int my_sub = part >> sub_shift;
  const uint32_t all_valid = (1u << (kBlock >> sub_shift)) - 1;
  float* merge = reinterpret_cast<float*>(smem + S::kRing);
  bool failed = false;
  int turn = 0;

  for (int32_t at = begin; at < end;) {
    const int32_t blk0 = walk.x.lo + skip;
    const int32_t n = min(walk.x.hi - blk0, end - at);
    const int32_t rows = walk.r.rows * a.group;  // of the request's tile grid
    const int32_t first_row = walk.tile * kRowsTile;
    const int32_t valid_rows = min(rows - first_row, kRowsTile);
    const int32_t pos0 = walk.r.len - walk.r.rows;

    // this thread's rows: g and g + 8 of the tile
    uint32_t qa[S::kSteps][4];
    float factor[2];
    int32_t limit[2];
    const float gk = a.c.k_scale ? a.c.k_scale[walk.head] : 1.0f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int32_t row = first_row + g + 8 * e;
      const bool there = g + 8 * e < valid_rows;
      const int32_t i = there ? row / a.group : 0;
      const int32_t h = walk.head * a.group + (there ? row - i * a.group : 0);
      uint32_t w[kDim / 8];  // kDim / 4 values
      const float down = load_query<kDim / 4>(
          a, a.q + (walk.r.start + i) * a.q_row + h * a.q_head + t * (kDim / 4), there, w);
#pragma unroll
      for (int j = 0; j < S::kSteps; ++j) qa[j][e] = w[2 * j], qa[j][2 + e] = w[2 * j + 1];
      factor[e] = a.scale_log2 * gk * down;
      limit[e] = there ? pos0 + i : 0x7FFFFFFF;
    }

    float o[S::kTiles][4];
#pragma unroll
    for (int j = 0; j < S::kTiles; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
    float m[2] = {kNone, kNone}, l[2] = {0.0f, 0.0f};
    bool any = false;

    // the team's blocks of this unit
    const int32_t first_mine = (team - count % kTeams + kTeams) % kTeams;
    for (int32_t i = first_mine; i < n; i += kTeams) {
      const int32_t blk = blk0 + i, number = count + i;
      const int stage = number % S::kStages;
      any = true;
      if (!failed && !wait_bounded(&full[stage], (number / S::kStages) & 1, gave_up)) failed = true;
      if (failed) continue;  // the producer stops by itself
      const uint32_t base = stage * S::kStageBytes;
      const uint32_t valid = masks[stage];

      // scores of 16 tokens
      float x[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.0f;
        const int tok = 8 * nt + token_of(g);
        uint32_t w[kDim / 32], s[2];
        if (kDim == 128) {
          const uint4 v = ptx::lds_v4(base + k_codes + tok * R::kCodeBytes + 16 * t);
          w[0] = v.x, w[1] = v.y, w[kDim / 32 - 2] = v.z, w[kDim / 32 - 1] = v.w;
          const uint32_t s2 = scales_to_f16(lds16(base + k_scales + tok * R::kScaleBytes + 2 * t));
          s[0] = __byte_perm(s2, s2, 0x1010), s[1] = __byte_perm(s2, s2, 0x3232);
        } else {
          const uint2 v = lds64(base + k_codes + tok * R::kCodeBytes + 8 * t);
          w[0] = v.x, w[1] = v.y;
          const uint32_t one = lds8(base + k_scales + tok * R::kScaleBytes + t);
          s[0] = s[1] = scales_to_f16(one * 0x0101u);
        }
#pragma unroll
        for (int j = 0; j < kDim / 32; ++j) {
          uint32_t b[4];
          e2m1x8_to_f16(w[j], b);
#pragma unroll
          for (int u = 0; u < 4; ++u) b[u] = mul_f16x2(b[u], s[j / 2 & 1]);
          mma_16816(x[nt], qa[2 * j], b[0], b[1]);
          mma_16816(x[nt], qa[2 * j + 1], b[2], b[3]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int u = 0; u < 4; ++u) x[nt][u] *= factor[u >> 1];

      const int32_t tok0 = blk * kBlock + part;
      const bool cut = blk * kBlock + kBlock - 1 > walk.x.p0 ||
                       (a.window > 0 && blk * kBlock <= walk.x.p1 - a.window) || valid != all_valid;
      if (cut) {
        const bool here = valid >> my_sub & 1;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int32_t tok = tok0 + 8 * nt + token_of(2 * t + (u & 1));
            const int32_t p = limit[u >> 1];
            const bool seen = here && tok <= p && tok < walk.r.len && (a.window <= 0 || tok > p - a.window);
            if (!seen) x[nt][u] = -INFINITY;
          }
      }

      // the running maximum
      float top[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        top[e] = fmaxf(fmaxf(x[0][2 * e], x[0][2 * e + 1]), fmaxf(x[1][2 * e], x[1][2 * e + 1]));
      if (__any_sync(0xFFFFFFFFu, top[0] > m[0] + kSlack || top[1] > m[1] + kSlack)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = top[e];
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
          v = fmaxf(v, m[e]);
          const float down = ex2(m[e] - v);
          m[e] = v;
          l[e] *= down;
#pragma unroll
          for (int j = 0; j < S::kTiles; ++j) o[j][2 * e] *= down, o[j][2 * e + 1] *= down;
        }
      }
      uint32_t pa[4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float p0 = ex2(x[nt][2 * e] - (m[e] - kShift)), p1 = ex2(x[nt][2 * e + 1] - (m[e] - kShift));
          l[e] += p0 + p1;
          pa[2 * nt + e] = cvt_f16x2(p0, p1);
        }

      // values: tokens a, b (columns 2t, 2t + 1) and c, d eight further
      const int ta = token_of(2 * t), tb = token_of(2 * t + 1);
      const uint32_t vs = base + v_scales + (kDim == 128 ? g : g >> 1);
      const uint32_t s_ab = scales_to_f16(lds8(vs + ta * R::kScaleBytes) | lds8(vs + tb * R::kScaleBytes) << 8);
      const uint32_t s_cd =
          scales_to_f16(lds8(vs + (8 + ta) * R::kScaleBytes) | lds8(vs + (8 + tb) * R::kScaleBytes) << 8);
      uint32_t wa[kDim / 64], wb[kDim / 64], wc[kDim / 64], wd[kDim / 64];
      const uint32_t vc = base + v_codes + g * (kDim / 16);
      if (kDim == 128) {
        const uint2 v0 = lds64(vc + ta * R::kCodeBytes), v1 = lds64(vc + tb * R::kCodeBytes);
        const uint2 v2 = lds64(vc + (8 + ta) * R::kCodeBytes), v3 = lds64(vc + (8 + tb) * R::kCodeBytes);
        wa[0] = v0.x, wb[0] = v1.x, wc[0] = v2.x, wd[0] = v3.x;
        wa[kDim / 64 - 1] = v0.y, wb[kDim / 64 - 1] = v1.y, wc[kDim / 64 - 1] = v2.y, wd[kDim / 64 - 1] = v3.y;
      } else {
        wa[0] = lds32(vc + ta * R::kCodeBytes), wb[0] = lds32(vc + tb * R::kCodeBytes);
        wc[0] = lds32(vc + (8 + ta) * R::kCodeBytes), wd[0] = lds32(vc + (8 + tb) * R::kCodeBytes);
      }
#pragma unroll
      for (int w = 0; w < kDim / 64; ++w) {
        constexpr uint32_t kLow = 0x0F0F0F0Fu;
        uint32_t even0[4], odd0[4], even1[4], odd1[4];
        e2m1x8_to_f16((wa[w] & kLow) | (wb[w] << 4 & ~kLow), even0);
        e2m1x8_to_f16((wa[w] >> 4 & kLow) | (wb[w] & ~kLow), odd0);
        e2m1x8_to_f16((wc[w] & kLow) | (wd[w] << 4 & ~kLow), even1);
        e2m1x8_to_f16((wc[w] >> 4 & kLow) | (wd[w] & ~kLow), odd1);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          mma_16816(o[8 * w + 2 * u], pa, mul_f16x2(even0[u], s_ab), mul_f16x2(even1[u], s_cd));
          mma_16816(o[8 * w + 2 * u + 1], pa, mul_f16x2(odd0[u], s_ab), mul_f16x2(odd1[u], s_cd));
        }
      }
      // the stage may be filled again: these were generic reads, the copy is not
      __syncwarp();
      if (lane == 0) {
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&empty[stage]);
      }
    }
    count += n;

    // ---- join the warps' parts ---------------------------------------------
    // The statistics are read until the rows are written; the next unit's go
    // to the other pair, and its sums only after its first barrier.
    float* st_max = reinterpret_cast<float*>(smem + S::kStats) + turn * 2 * kWarps * kRowsTile;
    float* st_sum = st_max + kWarps * kRowsTile;
    turn ^= 1;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 1);
      l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 2);
      if (failed) l[e] = NAN;
      if (t == 0) {
        st_max[warp * kRowsTile + g + 8 * e] = any ? m[e] : -INFINITY;
        st_sum[warp * kRowsTile + g + 8 * e] = l[e];
      }
    }
    ptx::named_bar_sync(1, kConsumers);
    if (any) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = kNone;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, st_max[w * kRowsTile + g + 8 * e]);
        const float down = ex2(m[e] - top);
        float* row = merge + (warp * kRowsTile + g + 8 * e) * S::kRowStride + 2 * t * S::kGroupStride;
#pragma unroll
        for (int j = 0; j < S::kTiles; ++j) {
          row[j] = o[j][2 * e] * down;
          row[S::kGroupStride + j] = o[j][2 * e + 1] * down;
        }
      }
    }
    ptx::named_bar_sync(1, kConsumers);
    // unit whole in this run: its rows are done; else a slot of the workspace
    const bool whole_unit = skip == 0 && n == walk.x.hi - walk.x.lo;
    const float gv = a.c.v_scale ? a.c.v_scale[walk.head] : 1.0f;
    float* slot = a.partials + (2 * static_cast<int64_t>(blockIdx.x) + (skip > 0 ? 0 : 1)) *
                                   slot_floats<kRowsTile, kDim>();
    for (int32_t it = tid; it < valid_rows * (kDim / 8); it += kConsumers) {
      const int32_t row = it / (kDim / 8), d0 = it % (kDim / 8) * 8;
      float top = kNone, sum = 0.0f, y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, st_max[w * kRowsTile + row]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = st_max[w * kRowsTile + row];
        if (mw == -INFINITY) continue;  // no blocks
        sum += st_sum[w * kRowsTile + row] * ex2(mw - top);
        const float* from = merge + (w * kRowsTile + row) * S::kRowStride + d0 / S::kLane * S::kGroupStride;
#pragma unroll
        for (int u = 0; u < 8; ++u) y[u] += from[d0 % S::kLane + u];
      }
      if (whole_unit) {
        const int32_t i = (first_row + row) / a.group;
        const int32_t h = walk.head * a.group + (first_row + row - i * a.group);
        const float by = sum == 0.0f ? 0.0f : gv / sum;
        uint16_t* out = a.out + (walk.r.start + i) * a.out_row + h * a.out_head + d0;
        uint32_t w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = pack_out(a.bf16, y[2 * u] * by, y[2 * u + 1] * by);
        if (a.out_vec) {
          *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u) out[2 * u] = w[u] & 0xFFFFu, out[2 * u + 1] = w[u] >> 16;
        }
        if (a.lse && d0 == 0)
          a.lse[static_cast<int64_t>(walk.r.start + i) * (a.heads * a.group) + h] =
              sum == 0.0f ? -INFINITY : (top - kShift + log2f(sum)) * kLn2;
      } else {
        float4* p = reinterpret_cast<float4*>(slot + row * kDim + d0);
        p[0] = make_float4(y[0], y[1], y[2], y[3]);
        p[1] = make_float4(y[4], y[5], y[6], y[7]);
        if (d0 == 0) slot[kRowsTile * kDim + row] = top, slot[kRowsTile * (kDim + 1) + row] = sum;
      }
    }
    at += n;
    skip = 0;
    if (at < end) walk.next();
  }
}

// Joins a unit's parts: one warp for each row and head.  Rows whose unit has
// no blocks are written here too.
constexpr int kJoinWarps = 8;

template <int kDim>
__global__ void __launch_bounds__(32 * kJoinWarps) join_rows_kernel(const __grid_constant__ Attn a, int grid) {
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);
  const int32_t q_heads = a.heads * a.group;
  const int64_t row64 = item / q_heads;
  if (row64 >= a.s.total_rows) return;
  const int32_t row = static_cast<int32_t>(row64), h = static_cast<int32_t>(item - row64 * q_heads);
  const int32_t b = find_request(a.s, row);
  if (b < 0) return;
  const Request r = load_request(a.s, b);
  const int32_t i = row - r.start;
  if (i < 0 || i >= r.rows) return;
  const int32_t head = h / a.group, in_grid = i * a.group + (h - head * a.group);
  const int32_t tile = in_grid / kRowsTile, in_tile = in_grid % kRowsTile;
  Tile x{0, 0, 0, 0};
  int32_t before = 0;
  if (r.len > 0) {
    for (int32_t t = 0; t < tile; ++t) {
      x = make_tile<kRowsTile>(a, r, t);
      before += (x.hi - x.lo) * a.heads;
    }
    x = make_tile<kRowsTile>(a, r, tile);
  }
  const int32_t n = x.hi - x.lo;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float y[kDim / 32];
#pragma unroll
  for (int u = 0; u < kDim / 32; ++u) y[u] = 0.0f;
  float sum = 0.0f, top = kNone;
  if (n > 0) {
    const int32_t run = run_length(a.prefix[a.s.batch], grid, kLeast);
    const int32_t u0 = a.prefix[b] + before + head * n;
    const int32_t c0 = u0 / run, c1 = (u0 + n - 1) / run;
    if (c0 == c1) return;  // whole in one run
    const auto slot_of = [&](int32_t c) {
      return a.partials + (2 * static_cast<int64_t>(c) + (c == c0 && static_cast<int64_t>(run) * c <= u0 ? 1 : 0)) *
                              slot_floats<kRowsTile, kDim>();
    };
    for (int32_t c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, slot_of(c)[kRowsTile * kDim + in_tile]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    for (int32_t c = c0; c <= c1; ++c) {
      const float* p = slot_of(c);
      const float w = ex2(p[kRowsTile * kDim + in_tile] - top);
      sum += p[kRowsTile * (kDim + 1) + in_tile] * w;
#pragma unroll
      for (int u = 0; u < kDim / 32; ++u) y[u] += p[in_tile * kDim + lane * (kDim / 32) + u] * w;
    }
  }
  const float gv = a.c.v_scale ? a.c.v_scale[head] : 1.0f;
  const float by = sum == 0.0f ? 0.0f : gv / sum;
  uint16_t* out = a.out + static_cast<int64_t>(row) * a.out_row + h * a.out_head + lane * (kDim / 32);
#pragma unroll
  for (int u = 0; u < kDim / 32; u += 2) {
    const uint32_t w = pack_out(a.bf16, y[u] * by, y[u + 1] * by);
    out[u] = w & 0xFFFFu, out[u + 1] = w >> 16;
  }
  if (a.lse && lane == 0)
    a.lse[static_cast<int64_t>(row) * q_heads + h] = sum == 0.0f ? -INFINITY : (top - kShift + log2f(sum)) * kLn2;
}

SmemAttr g_rows_attr[2];

template <int kDim>
cudaError_t launch_dim(const Attn& a, int grid, cudaStream_t stream) {
  const int smem = Shape<kDim>::smem(a.s.batch);
  if (!smem_attr_ready(g_rows_attr[kDim == 128], rows_kernel<kDim>, Shape<kDim>::smem(DSPARK_KV4_MAX_BATCH)))
    return cudaErrorInvalidValue;
  rows_kernel<kDim><<<grid, kThreadsRows, smem, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t items = static_cast<int64_t>(a.s.total_rows) * a.heads * a.group;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((items + kJoinWarps - 1) / kJoinWarps));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_rows_kernel<kDim>, a, grid);
}

}  // namespace

cudaError_t launch_rows(const Attn& a, int dim, int grid, cudaStream_t stream) {
  return dim == 128 ? launch_dim<128>(a, grid, stream) : launch_dim<64>(a, grid, stream);
}

}  // namespace kv4
}  // namespace dspark
