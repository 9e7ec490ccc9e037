// kv4_rows.cu -- attention of few rows over the paged 4-bit cache: the kernel
// for tiles of 8 or 16 rows (single tokens and short verifications).
//
// out_r = sum_t p_rt v_t / sum_t p_rt, p_rt = 2^(x_rt - m_r), x = scale log2(e) <q_r, k_t>.
// Few rows over a long cache: the cache's bytes bound it (144 bytes a token
// and head at 128 dimensions, for 8 x 512 multiply-adds).  So each byte is
// brought in once, by bulk copies of whole page records into a ring that a
// producer warp keeps full, and is turned into FP16 operands in registers.
// The tokens are the M side of both products (mma.m16n8k16: 16 tokens by 8
// rows, then 16 dimensions by 8 rows), so that 8 rows waste nothing:
//   S^T = K Q^T   a thread's share of a key row is the A fragment as it lies
//                 (the order of the dimensions under a dot product is free, so
//                 each thread takes consecutive ones);
//   O^T = V^T P^T the values' codes of two tokens are interleaved by two logic
//                 operations a word before the conversion, which gives the
//                 pairs along tokens that the A fragment wants; the weights,
//                 packed to FP16, are transposed in the warp (movmatrix).
// Measured: 64 single tokens over 4 to 16 k tokens (64 query heads on 8, 741 MB)
// 140 us, 5.3 TB/s of a copy's 6.7; 3 over 100 to 128 k tokens, FP16, 405 MB,
// 89 us, 4.5 TB/s; one over 2 k tokens 10.6 us, which is the latency of two
// dependent launches, of the first loads and of the merge.  With long caches the
// issue of the conversions and their multiplications bounds it.
#include "kv4_join.cuh"

namespace dspark {
namespace kv4 {
namespace {

constexpr int kTeams = 6;            // pairs of warps take blocks in turn
constexpr int kWarps = 2 * kTeams;   // consumers
constexpr int kConsumers = 32 * kWarps;
constexpr int kProducers = 3;        // warps that issue copies, in turn: one takes 0.3 us a block, the memory 0.2
constexpr int kThreadsRows = kConsumers + 128;  // and the producers' warpgroup
// Registers a thread: the block is launched with 128; 3 x 128 x 152 + 128 x 56 = 512 x 128.
constexpr int kProducerRegs = 56;
constexpr int kConsumerRegs = 152;
static_assert(kConsumers * kConsumerRegs + 128 * kProducerRegs <= kThreadsRows * kLaunchRegs, "registers of a CTA");

// kTiles8 tiles of 8 rows.
template <int kDim, int kTiles8>
struct Shape {
  static constexpr int kRows = 8 * kTiles8;
  // A multiple of the teams and of the producers: each stage then has one team
  // and one producer, which see every phase of its barriers in turn (a waiter
  // that skipped a phase could take the phase before for the one it wants).
  static constexpr int kStages = (kDim == 128 ? 1 : 2) * (kTiles8 == 2 ? 12 : 18);
  static_assert(kStages % kTeams == 0 && kStages % kProducers == 0, "a stage has one team and one producer");
  static constexpr int kStageBytes = kBlock * (kDim + kDim / 8);
  static constexpr int kSteps = kDim / 16;     // k-steps of the first product, m-tiles of the second
  static constexpr int kLane = kDim / 8;       // consecutive dimensions of a thread (second product)
  // the merge buffer (half of the warps at a time): dimension d of a row at d + 2 (d / kLane), rows kRowStride
  // apart (4 modulo 16): stores of 8 bytes then meet no bank twice
  static constexpr int kRowStride = 8 * (kLane + 2) + 4;
  static constexpr int kMergeBytes = kWarps / 2 * kRows * kRowStride * 4;
  // ring, merge buffer, maxima and totals, barriers and page masks, prefix sums
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kStats = kRing + kMergeBytes;
  static constexpr int kBars = kStats + 4 * kWarps * kRows * 4;  // two of each, for turns
  static constexpr int kMasks = kBars + 2 * kStages * 8;
  static constexpr int kMisc = kMasks + kStages * 4;
  static constexpr int kPrefix = kMisc + (kThreadsRows / 32 + 3) * 4;
  static int smem(int32_t batch) { return kPrefix + (batch + 1) * 4; }
};

// Row n of an 8-token part of a score tile is token n ^ (n >> 2 & 1): with it
// the shared-memory reads of keys and of values are both free of avoidable
// bank conflicts at 64 and at 32 bytes a token.
__device__ __forceinline__ int token_of(int n) { return n ^ (n >> 2 & 1); }

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit values over the warp, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

// Reads of the ring: plain loads, which the compiler may move between the
// waits (their asm clobbers memory).
template <typename V>
__device__ __forceinline__ V ring_at(const uint8_t* p) {
  return *reinterpret_cast<const V*>(p);
}

// kSplit: weights enter the second product as two FP16 numbers.  Results in
// FP16 would show one's rounding (a relative error of 2.9e-4, with two 2.0e-4,
// the result's own); results in BF16 do not (1.7e-3 either way).
template <int kDim, int kTiles8, bool kSplit>
__global__ void __launch_bounds__(kThreadsRows, 1) rows_kernel(const __grid_constant__ Attn a) {
  using S = Shape<kDim, kTiles8>;
  constexpr int kRows = S::kRows;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBars);
  uint64_t* empty = full + S::kStages;
  uint32_t* masks = reinterpret_cast<uint32_t*>(smem + S::kMasks);
  int32_t* misc = reinterpret_cast<int32_t*>(smem + S::kMisc);
  int32_t* gave_up = misc + kThreadsRows / 32 + 1;
  int32_t* prefix = reinterpret_cast<int32_t*>(smem + S::kPrefix);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid < S::kStages) {
    ptx::mbar_init(&full[tid], 1);
    ptx::mbar_init(&empty[tid], 2);
    ptx::fence_mbar_init();
    *gave_up = 0;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  plan<kRows, kThreadsRows>(a, prefix, misc);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int32_t total = prefix[a.s.batch];
  const int32_t run = run_length<kRows>(total, gridDim.x);
  const int64_t begin64 = static_cast<int64_t>(run) * blockIdx.x;
  if (begin64 >= total || total == kTooMany) {
    leave_no_cut(a, total);
    return;
  }
  const int32_t begin = static_cast<int32_t>(begin64);
  const int32_t end = static_cast<int32_t>(begin64 + run < total ? begin64 + run : total);

  const int sub = make_stage(a.c).tokens, sub_shift = make_stage(a.c).shift;

  if (warp >= kWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    if (warp >= kWarps + kProducers) return;
    produce<kDim, kRows, S::kStages, kProducers>(a, prefix, begin, end, warp - kWarps, smem, full, empty, masks,
                                                 gave_up);
    return;
  }

  // ---- consumers -----------------------------------------------------------
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
  Walk<kRows> walk(a, prefix);
  int32_t skip = walk.seek(begin);
  const int g = lane >> 2, t = lane & 3;
  const int team = warp >> 1, part = (warp & 1) * 32;  // 32 tokens of a block, as two groups of 16
  using R = Record<kDim>;
  // Where this thread reads in a stage: its groups' key codes and scales; the
  // values' are a section further.
  const int tok_k = token_of(g), tok_a = token_of(2 * t), tok_b = token_of(2 * t + 1);
  const uint32_t v_step = sub * R::kCodeBytes, s_step = sub * R::kScaleBytes;
  uint32_t codes[2], scales[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int tok = part + 16 * u;
    const uint32_t rec = (tok >> sub_shift) * (sub * (kDim + kDim / 8));
    const int row0 = tok & (sub - 1);
    codes[u] = rec + row0 * R::kCodeBytes;
    scales[u] = rec + 2 * v_step + row0 * R::kScaleBytes;
  }
  const uint32_t all_valid = (1u << (kBlock >> sub_shift)) - 1;
  float* merge = reinterpret_cast<float*>(smem + S::kRing);
  bool failed = false;
  int turn = 0;
  int stage = team % S::kStages;  // of this team's next block
  uint32_t phase = (team / S::kStages) & 1;
  int32_t behind = team;  // blocks of the run before it, from the unit's first on

  for (int32_t at = begin + walk.lead; at < end;) {
    const int32_t blk0 = walk.x.lo + skip;
    const int32_t n = min(walk.x.hi - blk0, end - at);
    const int32_t rows = walk.r.rows * a.group;  // of the request's tile grid
    const int32_t first_row = walk.tile * kRows;
    const int32_t valid_rows = min(rows - first_row, kRows);
    const int32_t pos0 = walk.r.len - walk.r.rows;

    // Rows g of each tile of 8 as B fragments; factor and limit are those of
    // the rows of this thread's scores (2t and 2t + 1).
    uint32_t qb[kTiles8][S::kSteps][2];
    float factor[kTiles8][2];
    int32_t limit[kTiles8][2];
    const float gk = a.c.k_scale ? a.c.k_scale[walk.head] : 1.0f;
#pragma unroll
    for (int nt = 0; nt < kTiles8; ++nt) {
      const int32_t in_tile = 8 * nt + g, row = first_row + in_tile;
      const bool there = in_tile < valid_rows;
      const int32_t i = there ? row / a.group : 0;
      const int32_t h = walk.head * a.group + (there ? row - i * a.group : 0);
      uint32_t w[kDim / 8];  // kDim / 4 values
      load_raw<kDim / 4>(a, a.q + (walk.r.start + i) * a.q_row + h * a.q_head + t * (kDim / 4), there, w);
      float down = 1.0f;
      if (a.bf16) {  // the row is spread over the four threads of a quad
        uint32_t top = largest(w);
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const int e = query_shift(top);
        shift_queries(w, power_of_two(e));
        down = power_of_two(-e);
      }
#pragma unroll
      for (int j = 0; j < S::kSteps; ++j) qb[nt][j][0] = w[2 * j], qb[nt][j][1] = w[2 * j + 1];
      const float f = a.scale_log2 * gk * down;
      const int32_t lim = there ? pos0 + i : 0x7FFFFFFF;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        factor[nt][e] = __shfl_sync(0xFFFFFFFFu, f, 4 * (2 * t + e));
        limit[nt][e] = __shfl_sync(0xFFFFFFFFu, lim, 4 * (2 * t + e));
      }
    }

    float o[kTiles8][S::kSteps][4];
    float m[kTiles8][2], l[kTiles8][2];
#pragma unroll
    for (int nt = 0; nt < kTiles8; ++nt) {
#pragma unroll
      for (int j = 0; j < S::kSteps; ++j) o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.0f;
      m[nt][0] = m[nt][1] = kNone;
      l[nt][0] = l[nt][1] = 0.0f;
    }
    bool any = false;

    for (; behind < n; behind += kTeams) {
      const int32_t blk = blk0 + behind;
      any = true;
      if (!failed && !wait_for(Phase(&full[stage], phase), gave_up)) failed = true;
      const uint8_t* base = smem + stage * S::kStageBytes;
      uint64_t* const done = &empty[stage];
      const uint32_t valid = masks[stage] & ~kLastBlock;
      stage += kTeams;
      if (stage >= S::kStages) stage -= S::kStages, phase ^= 1;
      if (failed) continue;  // the producer stops by itself

      // scores of two groups of 16 tokens
      float x[2][kTiles8][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int nt = 0; nt < kTiles8; ++nt) x[u][nt][0] = x[u][nt][1] = x[u][nt][2] = x[u][nt][3] = 0.0f;
        uint32_t w[2][kDim / 32], s[2][2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint8_t* kc = base + codes[u] + (8 * half + tok_k) * R::kCodeBytes;
          const uint8_t* ks = base + scales[u] + (8 * half + tok_k) * R::kScaleBytes;
          if (kDim == 128) {
            const uint4 v = ring_at<uint4>(kc + 16 * t);
            w[half][0] = v.x, w[half][1] = v.y, w[half][kDim / 32 - 2] = v.z, w[half][kDim / 32 - 1] = v.w;
            const uint32_t s2 = scales_to_f16(ring_at<uint16_t>(ks + 2 * t));
            s[half][0] = __byte_perm(s2, s2, 0x1010), s[half][1] = __byte_perm(s2, s2, 0x3232);
          } else {
            const uint2 v = ring_at<uint2>(kc + 8 * t);
            w[half][0] = v.x, w[half][1] = v.y;
            s[half][0] = s[half][1] = scales_to_f16(ring_at<uint8_t>(ks + t) * 0x0101u);
          }
        }
#pragma unroll
        for (int j = 0; j < kDim / 32; ++j) {
          uint32_t b0[4], b1[4];
          e2m1x8_to_f16(w[0][j], b0);
          e2m1x8_to_f16(w[1][j], b1);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            b0[e] = mul_f16x2(b0[e], s[0][j / 2 & 1]);
            b1[e] = mul_f16x2(b1[e], s[1][j / 2 & 1]);
          }
#pragma unroll
          for (int nt = 0; nt < kTiles8; ++nt) {
            mma_16816(x[u][nt], b0[0], b1[0], b0[1], b1[1], qb[nt][2 * j][0], qb[nt][2 * j][1]);
            mma_16816(x[u][nt], b0[2], b1[2], b0[3], b1[3], qb[nt][2 * j + 1][0], qb[nt][2 * j + 1][1]);
          }
        }
      }

      // relative to the running maximum; what a row may not see is -inf
      const bool cut = blk * kBlock + kBlock - 1 > walk.x.p0 ||
                       (a.window > 0 && blk * kBlock <= walk.x.p1 - a.window) || valid != all_valid;
      float top[kTiles8][2];
#pragma unroll
      for (int nt = 0; nt < kTiles8; ++nt) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[u][nt][e] = __fmul_rn(x[u][nt][e], factor[nt][e & 1]);
      }
      if (cut) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const bool here = valid >> ((part + 16 * u) >> sub_shift) & 1;
#pragma unroll
          for (int nt = 0; nt < kTiles8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int32_t tok = blk * kBlock + part + 16 * u + 8 * (e >> 1) + tok_k;
              const int32_t p = limit[nt][e & 1];
              const bool seen = here && tok <= p && tok < walk.r.len && (a.window <= 0 || p - tok < a.window);
              if (!seen) x[u][nt][e] = -INFINITY;
            }
        }
      }
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < kTiles8; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[nt][e] = fmaxf(fmaxf(x[0][nt][e], x[0][nt][2 + e]), fmaxf(x[1][nt][e], x[1][nt][2 + e]));
          raise |= top[nt][e] > m[nt][e] + kSlack;
        }
      if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
        for (int nt = 0; nt < kTiles8; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = top[nt][e];
            v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
            v = fmaxf(v, m[nt][e]);
            const float down = ex2(m[nt][e] - v);
            m[nt][e] = v;
            l[nt][e] *= down;
#pragma unroll
            for (int j = 0; j < S::kSteps; ++j) o[nt][j][e] *= down, o[nt][j][2 + e] *= down;
          }
      }
      uint32_t pb[2][kTiles8][2];
      uint32_t pl[2][kTiles8][2];  // what FP16 lost of them
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int nt = 0; nt < kTiles8; ++nt) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = ex2(x[u][nt][e] - (m[nt][e & 1] - kShift));
            l[nt][e & 1] += p[e];
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t w = cvt_f16x2(p[2 * e], p[2 * e + 1]);
            pb[u][nt][e] = transpose8(w);
            if (kSplit) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
              pl[u][nt][e] = transpose8(cvt_f16x2(p[2 * e] - f.x, p[2 * e + 1] - f.y));
            }
          }
        }

      // values: tokens a, b (the pair of this thread's weights) and eight further
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint8_t* vs = base + scales[u] + s_step + (kDim == 128 ? g : g >> 1);
        const uint32_t s_ab =
            scales_to_f16(ring_at<uint8_t>(vs + tok_a * R::kScaleBytes) | ring_at<uint8_t>(vs + tok_b * R::kScaleBytes) << 8);
        const uint32_t s_cd =
            scales_to_f16(ring_at<uint8_t>(vs + (8 + tok_a) * R::kScaleBytes) | ring_at<uint8_t>(vs + (8 + tok_b) * R::kScaleBytes) << 8);
        uint32_t wa[kDim / 64], wb[kDim / 64], wc[kDim / 64], wd[kDim / 64];
        const uint8_t* vc = base + codes[u] + v_step + g * (kDim / 16);
        if (kDim == 128) {
          const uint2 v0 = ring_at<uint2>(vc + tok_a * R::kCodeBytes), v1 = ring_at<uint2>(vc + tok_b * R::kCodeBytes);
          const uint2 v2 = ring_at<uint2>(vc + (8 + tok_a) * R::kCodeBytes), v3 = ring_at<uint2>(vc + (8 + tok_b) * R::kCodeBytes);
          wa[0] = v0.x, wb[0] = v1.x, wc[0] = v2.x, wd[0] = v3.x;
          wa[kDim / 64 - 1] = v0.y, wb[kDim / 64 - 1] = v1.y, wc[kDim / 64 - 1] = v2.y, wd[kDim / 64 - 1] = v3.y;
        } else {
          wa[0] = ring_at<uint32_t>(vc + tok_a * R::kCodeBytes), wb[0] = ring_at<uint32_t>(vc + tok_b * R::kCodeBytes);
          wc[0] = ring_at<uint32_t>(vc + (8 + tok_a) * R::kCodeBytes), wd[0] = ring_at<uint32_t>(vc + (8 + tok_b) * R::kCodeBytes);
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
          for (int e = 0; e < 4; ++e) {
            const uint32_t a0 = mul_f16x2(even0[e], s_ab), a1 = mul_f16x2(odd0[e], s_ab);
            const uint32_t a2 = mul_f16x2(even1[e], s_cd), a3 = mul_f16x2(odd1[e], s_cd);
#pragma unroll
            for (int nt = 0; nt < kTiles8; ++nt)
              mma_16816(o[nt][4 * w + e], a0, a1, a2, a3, pb[u][nt][0], pb[u][nt][1]);
            if (kSplit) {
#pragma unroll
              for (int nt = 0; nt < kTiles8; ++nt)
                mma_16816(o[nt][4 * w + e], a0, a1, a2, a3, pl[u][nt][0], pl[u][nt][1]);
            }
          }
        }
      }
      // the stage may be filled again: these were generic reads, the copy is not
      __syncwarp();
      if (lane == 0) {
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(done);
      }
    }
    behind -= n;

    // ---- join the warps' parts ---------------------------------------------
    // The statistics are read until the rows are written; the next unit's go
    // to the other pair, and its sums only after its first barrier.
    float* st_max = reinterpret_cast<float*>(smem + S::kStats) + turn * 2 * kWarps * kRows;
    float* st_sum = st_max + kWarps * kRows;
    turn ^= 1;
#pragma unroll
    for (int nt = 0; nt < kTiles8; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l[nt][e];
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 16);
        if (failed) v = NAN;
        if (g == 0) {
          st_max[warp * kRows + 8 * nt + 2 * t + e] = any ? m[nt][e] : -INFINITY;
          st_sum[warp * kRows + 8 * nt + 2 * t + e] = v;
        }
      }
    ptx::named_bar_sync(1, kConsumers);
    // the second half of the warps leaves its sums, the first adds its own
#pragma unroll
    for (int round = 0; round < 2; ++round) {
      if (warp / (kWarps / 2) != round) {
#pragma unroll
        for (int nt = 0; nt < kTiles8; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = 8 * nt + 2 * t + e;
            float top = kNone;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, st_max[w * kRows + row]);
            const float down = ex2(m[nt][e] - top);
            float2* to = reinterpret_cast<float2*>(merge + (warp % (kWarps / 2) * kRows + row) * S::kRowStride +
                                                   g * (S::kLane + 2));
#pragma unroll
            for (int j = 0; j < S::kSteps; ++j) {
              float2 v = make_float2(o[nt][j][e] * down, o[nt][j][2 + e] * down);
              if (round == 1) v.x += to[j].x, v.y += to[j].y;
              to[j] = v;
            }
          }
      }
      ptx::named_bar_sync(1, kConsumers);
    }
    // unit whole in this run: its rows are done; else a slot of the workspace
    const bool whole_unit = skip == 0 && n == walk.x.hi - walk.x.lo;
    const float gv = a.c.v_scale ? a.c.v_scale[walk.head] : 1.0f;
    float* slot = a.partials + (2 * static_cast<int64_t>(blockIdx.x) + (skip > 0 ? 0 : 1)) * slot_floats<kRows, kDim>();
    for (int32_t it = tid; it < valid_rows * (kDim / 8); it += kConsumers) {
      const int32_t row = it / (kDim / 8), d0 = it % (kDim / 8) * 8;
      float top = kNone, sum = 0.0f, y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, st_max[w * kRows + row]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = st_max[w * kRows + row];
        if (mw == -INFINITY) continue;  // no blocks
        sum += st_sum[w * kRows + row] * ex2(mw - top);
      }
#pragma unroll
      for (int w = 0; w < kWarps / 2; ++w) {
        const float2* from =
            reinterpret_cast<const float2*>(merge + (w * kRows + row) * S::kRowStride + d0 + d0 / S::kLane * 2);
#pragma unroll
        for (int u = 0; u < 4; ++u) y[2 * u] += from[u].x, y[2 * u + 1] += from[u].y;
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
        if (d0 == 0) slot[kRows * kDim + row] = top, slot[kRows * (kDim + 1) + row] = sum;
      }
    }
    at += n + walk.kLead;
    skip = 0;
    if (at < end) walk.next();
  }
}

SmemAttr g_rows_attr[2][2][2];

template <int kDim, int kTiles8, bool kSplit>
cudaError_t launch_shape(const Attn& a, int grid, cudaStream_t stream) {
  using S = Shape<kDim, kTiles8>;
  if (!smem_attr_ready(g_rows_attr[kDim == 128][kTiles8 - 1][kSplit], rows_kernel<kDim, kTiles8, kSplit>,
                       S::smem(DSPARK_KV4_MAX_BATCH), kLaunchRegs))
    return cudaErrorInvalidValue;
  const cudaError_t e = launch_behind(rows_kernel<kDim, kTiles8, kSplit>, dim3(grid), kThreadsRows, S::smem(a.s.batch), stream, a);
  if (e != cudaSuccess) return e;
  return launch_join<kDim, S::kRows>(a, grid, stream);
}

}  // namespace

cudaError_t launch_rows(const Attn& a, int dim, int32_t tile, int grid, cudaStream_t stream) {
  using Launch = cudaError_t (*)(const Attn&, int, cudaStream_t);
  static const Launch launch[2][2][2] = {
      {{launch_shape<64, 1, true>, launch_shape<64, 1, false>}, {launch_shape<64, 2, true>, launch_shape<64, 2, false>}},
      {{launch_shape<128, 1, true>, launch_shape<128, 1, false>},
       {launch_shape<128, 2, true>, launch_shape<128, 2, false>}}};
  return launch[dim == 128][tile == 16][a.bf16 != 0](a, grid, stream);
}

}  // namespace kv4
}  // namespace dspark
