// kv4_tiles.cu -- attention of many rows over the paged 4-bit cache: tiles of
// 128 or 256 query rows on the tensor cores (tcgen05), for verifications of
// grouped heads and for chunks of prompts.
//
// Per block of 64 tokens and 128 rows: S = Q K^T into tensor memory, weights
// P = 2^(x - m) by one thread a row, O += P V in tensor memory.
//   - Q lies in tensor memory as the A operand of the first product (of two
//     tiles of 128 dimensions the second lies in shared memory: tensor memory
//     is full), P as the A operand of the second, so that shared memory serves
//     little more than the B operands.
//   - The packed block (9 KB at 128 dimensions) comes by bulk copies; four
//     warps turn it into FP16 rows of 128 swizzled bytes, keys and values
//     alike: 64 tokens x 64 dimensions an operand half, K-major for the keys
//     (N = tokens), MN-major for the values (N = dimensions).
//   - Two streams of scores keep the tensor cores busy while weights are
//     formed: with 256 rows a stream is half of the rows, with 128 rows the
//     even and the odd blocks of the same rows, whose sums are joined at the
//     unit's end (they share tensor-memory lanes).  A stream's next scores are
//     computed as soon as its last ones are in registers: weights have columns
//     of their own.
// Measured: 2048 rows over 16 k tokens (64 query heads on 8, 128 dimensions,
// 1.03 TFLOP) 758 us, 1.36 PFLOP/s of a dense product's 1.87 (794 on another GPU):
// the warps that form weights bound it, with FP16 results 954 us.  48 verifications of 6 rows over 1 to 8 k tokens, 265 MB,
// 127 us, 2.1 TB/s: 48 of a tile's 128 rows are used, and a block's way through
// conversion, product, weights and product bounds it.  Two or four lanes a row,
// each with a part of the columns, and twice the warps for conversions were
// measured for that and gave nothing (32 requests of 48 rows over 4 to 8 k
// tokens: 112 us, with them 113 to 125, before the runs were weighted).
#include "kv4_join.cuh"

namespace dspark {
namespace kv4 {
namespace {

constexpr int kThreadsTiles = 512;
constexpr int kDequantWarp = 8;   // warps 8 .. 11
constexpr int kFirstWarp = 12;    // issues the first products, and holds the tensor memory
constexpr int kProducerWarp = 13;  // two of them; warp 15 issues the second products
constexpr int kProducersTiles = 2;
// Registers a thread: launched with 128; 2 x 176 + 72 + 88 = 4 x 128 (the best of
// nine splits measured: 2048 rows over 16 k tokens 757 us, with 168 / 96 / 80 810).
constexpr int kSoftmaxRegs = 176;
constexpr int kDequantRegs = 72;
constexpr int kOtherRegs = 88;
static_assert(128 * (2 * kSoftmaxRegs + kDequantRegs + kOtherRegs) <= kThreadsTiles * kLaunchRegs, "registers of a CTA");
static_assert(kThreadsTiles * kLaunchRegs > 65536 / 2, "one CTA a SM, which may take all of its tensor memory");

template <int kDim, int kStreams, bool kSplit>
struct Tiles {
  static constexpr int kRows = 128 * kStreams;  // rows of a tile
  // Tiles of 128 query rows from this one on lie in shared memory (tensor memory is full).
  static constexpr int kQShared = kDim == 64 ? kStreams : kSplit ? 0 : 1;
  static constexpr bool kAnyShared = kQShared < kStreams;
  // Rings of four (eight and three: 2048 rows over 16 k tokens 761 us for 757).
  static constexpr int kPacked = 4;             // ring of packed blocks
  static constexpr int kPackedBytes = kBlock * (kDim + kDim / 8);
  static constexpr int kOps = kSplit && kDim == 128 && kStreams == 2 ? 3 : 4;  // ring of operand blocks
  static constexpr int kHalfBytes = kBlock * 128;           // 64 tokens x 64 dimensions
  static constexpr int kMatBytes = kDim / 64 * kHalfBytes;  // keys or values of a block
  static constexpr int kOpBytes = 2 * kMatBytes;
  static constexpr int kQHalf = 128 * 128;                  // 128 rows x 64 dimensions
  // tensor memory columns
  static constexpr int kO = 0;               // [stream][kDim]
  static constexpr int kS = 2 * kDim;        // [stream][64]
  static constexpr int kP = kS + 2 * kBlock;  // [stream][32]
  static constexpr int kLow = kP + kBlock;    // [stream][32] with kSplit
  static constexpr int kQ = kLow + (kSplit ? kBlock : 0);  // [tile][kDim / 2]
  static_assert(kQ + kQShared * kDim / 2 <= 512, "tensor memory");
  // shared memory: operands first (1024-byte atoms)
  static constexpr int kQAt = kOps * kOpBytes;
  static constexpr int kRing = kQAt + (kStreams - kQShared) * 2 * kQHalf;
  static constexpr int kStats = kRing + kPacked * kPackedBytes;  // [stream][128][2]
  static constexpr int kBars = kStats + 2 * 128 * 2 * 4;
  static constexpr int kNumBars = 2 * kPacked + 3 * kOps + 4 * 2 + 3;
  static constexpr int kMasks = kBars + kNumBars * 8;  // [kPacked], then [kOps]
  static constexpr int kMisc = kMasks + (kPacked + kOps) * 4;
  static constexpr int kPrefix = kMisc + (kThreadsTiles / 32 + 3) * 4;
  static int smem(int32_t batch) { return kPrefix + (batch + 1) * 4 + 1024; }
};

// Four warps' share of a block's keys or values (section `which`): 16 elements
// of a scale a thread and step.  Eight lanes that store together hold two
// tokens' four blocks of one half, which meet all banks once.
template <int kDim>
__device__ __forceinline__ void dequant(const uint8_t* packed, uint8_t* to, int which, const Stage& st, int warp, int lane) {
  using R = Record<kDim>;
  constexpr int kPer = kDim == 128 ? 4 : 8;  // tokens of a warp's step
  const int block = kDim == 128 ? (lane & 3) + 4 * (lane >> 3 & 1) : lane & 3;
  const int tok_in = kDim == 128 ? (lane >> 2 & 1) + 2 * (lane >> 4) : lane >> 2;
  const uint32_t code0 = R::codes(st.tokens, which), scale0 = R::scales(st.tokens, which);
  constexpr int kStepsOf = kBlock / (4 * kPer);
  uint2 code[kStepsOf];
  uint32_t scale[kStepsOf];
#pragma unroll
  for (int step = 0; step < kStepsOf; ++step) {
    const int tok = (step * 4 + warp) * kPer + tok_in, row = tok & (st.tokens - 1);
    const uint8_t* rec = packed + (tok >> st.shift) * (st.tokens * (kDim + kDim / 8));
    code[step] = *reinterpret_cast<const uint2*>(rec + code0 + row * R::kCodeBytes + block * 8);
    scale[step] = rec[scale0 + row * R::kScaleBytes + block];
  }
#pragma unroll
  for (int step = 0; step < kStepsOf; ++step) {
    const int tok = (step * 4 + warp) * kPer + tok_in;
    const uint32_t s2 = scales_to_f16(scale[step] * 0x0101u);
    uint32_t a[4], b[4];
    e2m1x8_to_f16(code[step].x, a);
    e2m1x8_to_f16(code[step].y, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = mul_f16x2(a[i], s2), b[i] = mul_f16x2(b[i], s2);
    uint8_t* at = to + (block >> 2) * (kBlock * 128) + tok * 128;
    const uint32_t chunk = 2 * (block & 3);
    *reinterpret_cast<uint4*>(at + ((chunk ^ (tok & 7)) << 4)) = make_uint4(a[0], a[1], a[2], a[3]);
    *reinterpret_cast<uint4*>(at + (((chunk + 1) ^ (tok & 7)) << 4)) = make_uint4(b[0], b[1], b[2], b[3]);
  }
}

// A word with its n lowest bits set (n of any size).
__device__ __forceinline__ uint32_t low_bits(int32_t n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; }

// The largest of three; pairs of FP32 in a 64-bit register.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  return static_cast<uint64_t>(__float_as_uint(hi)) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// kSplit: weights enter the second product as two FP16 numbers, FP16's 11 bits of
// them and what is left (FP16 results, as in kv4_rows.cu, so that their error
// does not depend on the kernel: 2.1e-4 against 64 bits, with one number 2.8e-4).
// That is half as many products again and four operations more a pair of
// weights: 2048 rows over 16 k tokens 748 -> 954 us, 48 verifications of 6 rows
// 119 -> 140 (64 dimensions 95 -> 109).  The low numbers have columns of their
// own, for which the queries leave tensor memory at 128 dimensions; lying where
// the scores did, they let no product run ahead (1540 and 191 us).
template <int kDim, int kStreams, bool kSplit>
__global__ void __launch_bounds__(kThreadsTiles, 1) tiles_kernel(const __grid_constant__ Attn a) {
  using T = Tiles<kDim, kStreams, kSplit>;
  constexpr int kRows = T::kRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (1024u - (ptx::smem_addr(smem_raw) & 1023u)) % 1024u;
  uint64_t* packed_full = reinterpret_cast<uint64_t*>(smem + T::kBars);
  uint64_t* packed_empty = packed_full + T::kPacked;
  uint64_t* k_full = packed_empty + T::kPacked;
  uint64_t* v_full = k_full + T::kOps;
  uint64_t* op_empty = v_full + T::kOps;
  uint64_t* s_full = op_empty + T::kOps;  // [stream]: scores are there
  uint64_t* s_read = s_full + 2;          // [stream]: they are in registers
  uint64_t* p_ready = s_read + 2;         // [stream]: weights are there
  uint64_t* pv_done = p_ready + 2;        // [stream]: the second product has ended
  uint64_t* q_ready = pv_done + 2;
  uint64_t* drained = q_ready + 1;  // [issuer]
  uint32_t* packed_masks = reinterpret_cast<uint32_t*>(smem + T::kMasks);
  uint32_t* op_masks = packed_masks + T::kPacked;
  int32_t* misc = reinterpret_cast<int32_t*>(smem + T::kMisc);
  int32_t* gave_up = misc + kThreadsTiles / 32 + 1;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(misc + kThreadsTiles / 32 + 2);
  int32_t* prefix = reinterpret_cast<int32_t*>(smem + T::kPrefix);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int i = 0; i < T::kPacked; ++i) {
      ptx::mbar_init(&packed_full[i], 1);
      ptx::mbar_init(&packed_empty[i], 4);
    }
    for (int i = 0; i < T::kOps; ++i) {
      ptx::mbar_init(&k_full[i], 4);
      ptx::mbar_init(&v_full[i], 4);
      ptx::mbar_init(&op_empty[i], kStreams);  // one second product of each stream that reads it
    }
    for (int x = 0; x < 2; ++x) {
      ptx::mbar_init(&s_full[x], 2);  // the product's end, and its issuer
      ptx::mbar_init(&s_read[x], 4);
      ptx::mbar_init(&p_ready[x], 4);
      ptx::mbar_init(&pv_done[x], 1);
    }
    ptx::mbar_init(q_ready, 8);
    ptx::mbar_init(&drained[0], 1);
    ptx::mbar_init(&drained[1], 1);
    ptx::fence_mbar_init();
    *gave_up = 0;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  plan<kRows, kThreadsTiles>(a, prefix, misc);
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

  if (warp == kFirstWarp) {
    ptx::tmem_alloc(tmem_at, 512);
    ptx::tmem_relinquish();
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_at;
  const Stage st = make_stage(a.c);
  const uint32_t ops = ptx::smem_addr(smem);

  if (warp >= kFirstWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp >= kProducerWarp && warp < kProducerWarp + kProducersTiles) {
      produce<kDim, kRows, T::kPacked, kProducersTiles>(a, prefix, begin, end, warp - kProducerWarp, smem + T::kRing,
                                                        packed_full, packed_empty, packed_masks, gave_up);
    } else {
      // ---- the tensor cores' issuers: a warp for each product, so that one's
      // waits pass while the other's work runs.  A warp runs uniformly
      // (descriptors stay in uniform registers), one lane issues.
      constexpr uint32_t kIdescS = ptx::idesc_f16_f32(128, kBlock);
      constexpr uint32_t kIdescO = ptx::idesc_f16_f32(128, kDim) | ptx::kIdescBMn;
      Walk<kRows> walk(a, prefix);
      int32_t skip = walk.seek(begin);
      uint32_t unit = 0, count = 0;     // units, blocks of the run so far
      uint32_t steps0 = 0, steps1 = 0;  // this warp's products of the streams so far
      bool ok = true;
      const auto first = [&](int x, uint32_t op) {  // S_x = Q_x K^T
        ptx::mbar_arrive(&s_full[x]);  // passes on what came with the keys: the block's mask
        const uint64_t b = ptx::sw128_desc(ops + op * T::kOpBytes, 1024);
        const uint32_t d = tmem + T::kS + x * kBlock;
#pragma unroll
        for (int j = 0; j < kDim / 16; ++j) {
          const uint32_t to = (j / 4 * T::kHalfBytes + j % 4 * 32) >> 4;  // in the descriptor's units
          const int tile = kStreams == 2 ? x : 0;
          if (tile >= T::kQShared) {
            const uint64_t q = ptx::sw128_desc(ops + T::kQAt + (tile - T::kQShared) * 2 * T::kQHalf, 1024) +
                               ((j / 4 * T::kQHalf + j % 4 * 32) >> 4);
            if (j == 0) ptx::mma_f16_c<false>(d, q, b, kIdescS);
            else ptx::mma_f16_c<true>(d, q, b + to, kIdescS);
          } else {
            const uint32_t q = tmem + T::kQ + tile * (kDim / 2) + j * 8;
            if (j == 0) ptx::mma_tmem_a_c<false>(d, q, b, kIdescS);
            else ptx::mma_tmem_a_c<true>(d, q, b + to, kIdescS);
          }
        }
        ptx::mma_commit(&s_full[x]);
      };
      const auto second = [&](int x, uint32_t op, bool accumulate) {  // O_x += P_x V
        const uint64_t b = ptx::sw128_desc_mn(ops + op * T::kOpBytes + T::kMatBytes, T::kHalfBytes, 1024);
        const uint32_t d = tmem + T::kO + x * kDim, p = tmem + T::kP + x * (kBlock / 2);
#pragma unroll
        for (int j = 0; j < kBlock / 16; ++j) {
          if (j == 0 && !accumulate) ptx::mma_tmem_a_c<false>(d, p, b, kIdescO);
          else ptx::mma_tmem_a_c<true>(d, p + j * 8, b + j * (2048 >> 4), kIdescO);
        }
        if (kSplit) {
#pragma unroll
          for (int j = 0; j < kBlock / 16; ++j)
            ptx::mma_tmem_a_c<true>(d, tmem + T::kLow + x * (kBlock / 2) + j * 8, b + j * (2048 >> 4), kIdescO);
        }
        ptx::mma_commit(&pv_done[x]);
        ptx::mma_commit(&op_empty[op]);  // its weights come from scores: the keys have been read too
      };
      for (int32_t at = begin + walk.lead; at < end && ok;) {
        const int32_t n = min(walk.x.hi - walk.x.lo - skip, end - at);
        for (int32_t b = 0; b < n && ok; ++b) {
          const uint32_t now = count + b, op = now % T::kOps;
#pragma unroll
          for (int y = 0; y < kStreams; ++y) {
            const int x = kStreams == 2 ? y : b & 1;
            const uint32_t steps = x ? steps1 : steps0;
            if (warp == kFirstWarp) {
              ok = wait_for(Phase(&k_full[op], now / T::kOps), Phase(&s_read[x], steps - 1, steps > 0),
                            Phase(q_ready, unit), gave_up);
              if (!ok) break;
              ptx::tc_fence_after();
              if (ptx::elect_one_lane()) first(x, op);
            } else {
              ok = wait_for(Phase(&p_ready[x], steps), Phase(&v_full[op], now / T::kOps), gave_up);
              if (!ok) break;
              ptx::tc_fence_after();
              if (ptx::elect_one_lane()) second(x, op, b >= (kStreams == 2 ? 1 : 2));
            }
            __syncwarp();
            if (x) ++steps1;
            else ++steps0;
          }
        }
        count += n;
        ++unit;
        at += n + walk.kLead;
        skip = 0;
        if (at < end) walk.next();
      }
      if (!ok) {  // what is in flight ends before tensor memory is freed
        uint64_t* bar = &drained[warp == kFirstWarp ? 0 : 1];
        if (ptx::elect_one_lane()) ptx::mma_commit(bar);
        __syncwarp();
        for (uint32_t t = 0; t < kPolls && !ptx::mbar_try_wait(bar, 0); ++t) {
        }
      }
    }
  } else if (warp >= kDequantWarp) {
    // ---- packed blocks to operands -----------------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kDequantRegs));
    const int w = warp - kDequantWarp;
    bool ok = true;
    bool last = false;
    for (int32_t i = 0; !last; ++i) {
      const int stage = i % T::kPacked, op = i % T::kOps;
      ok = wait_for(Phase(&packed_full[stage], i / T::kPacked), Phase(&op_empty[op], i / T::kOps - 1, i >= T::kOps),
                    gave_up);
      if (!ok) break;
      const uint8_t* packed = smem + T::kRing + stage * T::kPackedBytes;
      uint8_t* to = smem + op * T::kOpBytes;
      const uint32_t mask = packed_masks[stage];
      last = (mask & kLastBlock) != 0;
      if (w == 0 && lane == 0) op_masks[op] = mask & ~kLastBlock;
      dequant<kDim>(packed, to, 0, st, w, lane);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      ptx::mbar_arrive_if(&k_full[op], lane == 0);
      dequant<kDim>(packed, to + T::kMatBytes, 1, st, w, lane);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      ptx::mbar_arrive_if(&v_full[op], lane == 0);
      ptx::mbar_arrive_if(&packed_empty[stage], lane == 0);
    }
  } else {
    // ---- weights: one thread a row ------------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int x = warp >> 2;                 // stream
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's 32 lanes (lane << 16)
    const uint32_t s_at = tmem + lanes + T::kS + x * kBlock, p_at = tmem + lanes + T::kP + x * (kBlock / 2);
    const uint32_t o_at = tmem + lanes + T::kO + x * kDim;
    const int in_tile = (kStreams == 2 ? x * 128 : 0) + (warp & 3) * 32 + lane;  // row of the tile
    const uint32_t all_valid = (1u << (kBlock >> st.shift)) - 1;
    float* stats = reinterpret_cast<float*>(smem + T::kStats);  // [stream][row][2]
    Walk<kRows> walk(a, prefix);
    int32_t skip = walk.seek(begin);
    uint32_t steps = 0, count = 0;  // blocks of this stream, and of the run, so far
    bool failed = false;

    for (int32_t at = begin + walk.lead; at < end;) {
      const int32_t blk0 = walk.x.lo + skip;
      const int32_t n = min(walk.x.hi - blk0, end - at);
      const int32_t rows = walk.r.rows * a.group;
      const int32_t first_row = walk.tile * kRows;
      const int32_t valid_rows = min(rows - first_row, kRows);
      const int32_t pos0 = walk.r.len - walk.r.rows;
      const bool there = in_tile < valid_rows;
      const int32_t row = first_row + (there ? in_tile : 0), qi = row / a.group;
      const int32_t head = walk.head * a.group + (row - qi * a.group);
      const int32_t limit = max(pos0 + qi, -1);  // positions below 0 see nothing, and may be far below
      // the warp's rows: whether there are any, and their first and last position
      const int32_t warp_row = in_tile - lane;
      const bool active = warp_row < valid_rows;
      const int32_t p_first = pos0 + (first_row + warp_row) / a.group;
      const int32_t p_last = max(pos0 + (first_row + min(warp_row + 31, valid_rows - 1)) / a.group, -1);

      // the query row to tensor memory; with one tile for both streams, half of it each
      float factor = a.scale_log2 * (a.c.k_scale ? a.c.k_scale[walk.head] : 1.0f);
      const uint16_t* q = a.q + (walk.r.start + qi) * a.q_row + head * a.q_head;
      const bool flip = factor < 0.0f;
      if (flip) factor = -factor;
      {
        uint32_t w[kDim / 64][32];
#pragma unroll
        for (int c = 0; c < kDim / 64; ++c) load_raw<64>(a, q + 64 * c, there, w[c]);
        __syncwarp();  // rows that are not there took another way; what follows is for whole warps
        if (a.bf16) {
          uint32_t top = largest(w[0]);
          if (kDim == 128) top = max(top, largest(w[kDim / 64 - 1]));
          const int e = query_shift(top);
          factor *= power_of_two(-e);
#pragma unroll
          for (int c = 0; c < kDim / 64; ++c) shift_queries(w[c], power_of_two(e));
        }
#pragma unroll
        for (int c = 0; c < kDim / 64; ++c) {
          if (kStreams == 1 && c != (kDim == 128 ? x : 0)) continue;
          if (kStreams == 1 && kDim == 64 && x != 0) continue;
          if (flip) {
#pragma unroll
            for (int i = 0; i < 32; ++i) w[c][i] ^= 0x80008000u;
          }
          const int tile = kStreams == 2 ? x : 0;
          if (tile >= T::kQShared) {
            const int in_shared = T::kQShared == 1 ? 0 : tile;
            const int r = T::kQShared == 1 ? in_tile - 128 : in_tile & 127;
            uint8_t* to = smem + T::kQAt + (in_shared * 2 + c) * T::kQHalf + r * 128;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(to + ((i ^ (r & 7)) << 4)) =
                  make_uint4(w[c][4 * i], w[c][4 * i + 1], w[c][4 * i + 2], w[c][4 * i + 3]);
          } else {
            ptx::tmem_st32(tmem + lanes + T::kQ + tile * (kDim / 2) + c * 32, w[c]);
          }
        }
        ptx::tmem_st_wait();
        if (T::kAnyShared) ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        ptx::mbar_arrive_if(q_ready, lane == 0);
      }
      // A factor of 0 would make NaN of a score of -inf; any factor this small
      // gives the same weights.
      factor = fmaxf(factor, 1e-37f);

      float m = kNone, l = 0.0f;
      const int32_t mine = kStreams == 2 ? n : (n - x + 1) / 2;  // blocks of this stream
      // A poll of the next scores, made ahead of its use, where its answer costs
      // nothing (one that may not stay: the weights have to be handed over).
      bool early = false;
      for (int32_t i = 0; i < mine; ++i) {
        const int32_t b = kStreams == 2 ? i : 2 * i + x;
        const uint32_t number = count + b;
        if (!failed && !__all_sync(0xFFFFFFFFu, early)) failed = !wait_for(Phase(&s_full[x], steps), gave_up);
        early = false;
        ++steps;
        if (failed) continue;
        ptx::tc_fence_after();
        if (!active) {
          ptx::mbar_arrive_if(&s_read[x], lane == 0);
          // in step with the second products, a phase at a time
          if (i > 0) failed = !wait_for(Phase(&pv_done[x], steps), gave_up);
        } else {
          const int32_t blk = blk0 + b;
          const uint32_t valid = op_masks[number % T::kOps];
          uint32_t s[2][32];
          ptx::tmem_ld64_sync(s_at, s[0], s[1]);
          ptx::tc_fence_before();
          __syncwarp();
          ptx::mbar_arrive_if(&s_read[x], lane == 0);
          if (blk * kBlock + kBlock - 1 > p_first || (a.window > 0 && blk * kBlock <= p_last - a.window) ||
              valid != all_valid) {
            // the row's visible columns as two words of bits
            const int32_t end_col = min(limit + 1, walk.r.len) - blk * kBlock;
            const int32_t first_col = a.window > 0 ? limit - a.window + 1 - blk * kBlock : 0;
            uint32_t see[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              see[u] = low_bits(end_col - 32 * u) & ~low_bits(first_col - 32 * u);
              if (st.shift >= 6) see[u] &= valid & 1 ? ~0u : 0u;
              else if (st.shift == 5) see[u] &= valid >> u & 1 ? ~0u : 0u;
              else see[u] &= (valid >> (2 * u) & 1 ? 0xFFFFu : 0u) | (valid >> (2 * u + 1) & 1 ? 0xFFFF0000u : 0u);
            }
#pragma unroll
            for (int c = 0; c < kBlock; ++c)
              if (!(see[c / 32] >> (c % 32) & 1)) s[c / 32][c % 32] = 0xFF800000u;
          }
          float part[4] = {kNone, kNone, kNone, kNone};
#pragma unroll
          for (int c = 0; c < kBlock; c += 2)
            part[c / 2 & 3] =
                max3(part[c / 2 & 3], __uint_as_float(s[c / 32][c % 32]), __uint_as_float(s[c / 32][c % 32 + 1]));
          const float top = __fmul_rn(fmaxf(max3(part[0], part[1], part[2]), part[3]), factor);
          if (__any_sync(0xFFFFFFFFu, top > m + kSlack)) {
            const float now = fmaxf(top, m), down = ex2(m - now);
            m = now;
            l *= down;
            if (i > 0) {  // after the second product before
              failed = !wait_for(Phase(&pv_done[x], steps), gave_up);
              ptx::tc_fence_after();
#pragma unroll
              for (int c = 0; c < kDim; c += 32) {
                uint32_t o[32];
                ptx::tmem_ld32_sync(o_at + c, o);
#pragma unroll
                for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * down);
                ptx::tmem_st32(o_at + c, o);
              }
            }
          }
          const uint64_t factor2 = pack2(factor, factor), shift2 = pack2(kShift - m, kShift - m);
          uint32_t p[32], low[kSplit ? 32 : 1];
          uint64_t sum2[2] = {0, 0};
#pragma unroll
          for (int c = 0; c < kBlock; c += 2) {
            const uint64_t v =
                fma2(static_cast<uint64_t>(s[c / 32][c % 32 + 1]) << 32 | s[c / 32][c % 32], factor2, shift2);
            const float p0 = ex2(__uint_as_float(static_cast<uint32_t>(v)));
            const float p1 = ex2(__uint_as_float(static_cast<uint32_t>(v >> 32)));
            sum2[c / 2 & 1] = add2(sum2[c / 2 & 1], pack2(p0, p1));
            if constexpr (kSplit) {  // FP16's 11 bits, cut, and what is left
              constexpr uint32_t kHigh = 0xFFFFE000u;
              const uint32_t h0 = __float_as_uint(p0) & kHigh, h1 = __float_as_uint(p1) & kHigh;
              p[c / 2] = cvt_f16x2(__uint_as_float(h0), __uint_as_float(h1));
              const uint64_t left = fma2(static_cast<uint64_t>(h1) << 32 | h0, pack2(-1.0f, -1.0f), pack2(p0, p1));
              low[c / 2] = cvt_f16x2(__uint_as_float(static_cast<uint32_t>(left)),
                                     __uint_as_float(static_cast<uint32_t>(left >> 32)));
            } else {
              p[c / 2] = cvt_f16x2(p0, p1);
            }
          }
          const uint64_t both = add2(sum2[0], sum2[1]);
          l += __uint_as_float(static_cast<uint32_t>(both)) + __uint_as_float(static_cast<uint32_t>(both >> 32));
          const uint32_t pv_over = i > 0 ? ptx::mbar_try_wait(&pv_done[x], steps & 1) : 1u;
          // the second product before has read the weights that these replace
          if (!__all_sync(0xFFFFFFFFu, pv_over) && !failed) failed = !wait_for(Phase(&pv_done[x], steps), gave_up);
          ptx::tc_fence_after();
          ptx::tmem_st32(p_at, p);
          if constexpr (kSplit) ptx::tmem_st32(tmem + lanes + T::kLow + x * (kBlock / 2), low);
          if (i + 1 < mine) early = ptx::mbar_test_wait(&s_full[x], steps & 1);
          ptx::tmem_st_wait();
        }
        ptx::tc_fence_before();
        __syncwarp();
        ptx::mbar_arrive_if(&p_ready[x], lane == 0);
      }
      count += n;

      // ---- the unit's rows ----------------------------------------------------
      if (mine > 0 && !failed) failed = !wait_for(Phase(&pv_done[x], steps - 1), gave_up);
      ptx::tc_fence_after();
      if (failed) l = NAN;
      float w_own = 1.0f, w_other = 0.0f, sum = l, top = m;
      bool other = false;
      if (kStreams == 1) {  // both streams' parts of a row, half of its dimensions each
        stats[(x * 128 + in_tile) * 2] = m;
        stats[(x * 128 + in_tile) * 2 + 1] = l;
        ptx::tc_fence_before();
        __syncwarp();
        ptx::named_bar_sync(1, 256);
        ptx::tc_fence_after();
        const float m2 = stats[((1 - x) * 128 + in_tile) * 2], l2 = stats[((1 - x) * 128 + in_tile) * 2 + 1];
        other = x == 1 || n > 1;  // stream 1 has no block in a unit of one
        top = fmaxf(m, m2);
        w_own = ex2(m - top);
        w_other = ex2(m2 - top);
        sum = l * w_own + l2 * w_other;
      }
      const bool own = mine > 0;
      const bool whole_unit = skip == 0 && n == walk.x.hi - walk.x.lo;
      if (active) {
        const float gv = a.c.v_scale ? a.c.v_scale[walk.head] : 1.0f;
        const float by = whole_unit ? (sum == 0.0f ? 0.0f : gv / sum) : 1.0f;
        float* slot = a.partials + (2 * static_cast<int64_t>(blockIdx.x) + (skip > 0 ? 0 : 1)) *
                                       slot_floats<kRows, kDim>();
        uint16_t* out = a.out + (walk.r.start + qi) * a.out_row + head * a.out_head;
        constexpr int kSpan = kStreams == 2 ? kDim : kDim / 2;  // dimensions of this thread
        const int d_first = kStreams == 2 ? 0 : x * kSpan;
#pragma unroll
        for (int c = 0; c < kSpan; c += 32) {
          const int d0 = d_first + c;
          uint32_t o[32];
          float y[32];
#pragma unroll
          for (int u = 0; u < 32; ++u) y[u] = 0.0f;
          if (own) {
            ptx::tmem_ld32_sync(o_at + d0, o);
#pragma unroll
            for (int u = 0; u < 32; ++u) y[u] = __uint_as_float(o[u]) * w_own;
          }
          if (kStreams == 1 && other) {
            ptx::tmem_ld32_sync(tmem + lanes + T::kO + (1 - x) * kDim + d0, o);
#pragma unroll
            for (int u = 0; u < 32; ++u) y[u] += __uint_as_float(o[u]) * w_other;
          }
          if (there && whole_unit) {
#pragma unroll
            for (int u = 0; u < 32; u += 8) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) w[j] = pack_out(a.bf16, y[u + 2 * j] * by, y[u + 2 * j + 1] * by);
              if (a.out_vec) {
                *reinterpret_cast<uint4*>(out + d0 + u) = make_uint4(w[0], w[1], w[2], w[3]);
              } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  out[d0 + u + 2 * j] = w[j] & 0xFFFFu, out[d0 + u + 2 * j + 1] = w[j] >> 16;
              }
            }
          } else if (there) {
            float4* to = reinterpret_cast<float4*>(slot + in_tile * kDim + d0);
#pragma unroll
            for (int u = 0; u < 8; ++u) to[u] = make_float4(y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]);
          }
          __syncwarp();  // tensor memory is read by whole warps
        }
        if (there && (kStreams == 2 || x == 0)) {
          if (!whole_unit) {
            slot[kRows * kDim + in_tile] = top;
            slot[kRows * (kDim + 1) + in_tile] = sum;
          } else if (a.lse) {
            a.lse[static_cast<int64_t>(walk.r.start + qi) * (a.heads * a.group) + head] =
                sum == 0.0f ? -INFINITY : (top - kShift + log2f(sum)) * kLn2;
          }
        }
      }
      // tensor memory was read before the next unit's products may write it
      __syncwarp();
      ptx::tc_fence_before();
      if (kStreams == 1) ptx::named_bar_sync(1, 256);
      at += n + walk.kLead;
      skip = 0;
      if (at < end) walk.next();
    }
  }
  __syncwarp();
  __syncthreads();
  if (warp == kFirstWarp) ptx::tmem_dealloc(tmem, 512);
}

SmemAttr g_tiles_attr[2][2][2];

template <int kDim, int kStreams, bool kSplit>
cudaError_t launch_shape(const Attn& a, int grid, cudaStream_t stream) {
  using T = Tiles<kDim, kStreams, kSplit>;
  if (!smem_attr_ready(g_tiles_attr[kDim == 128][kStreams - 1][kSplit], tiles_kernel<kDim, kStreams, kSplit>,
                       T::smem(DSPARK_KV4_MAX_BATCH), kLaunchRegs))
    return cudaErrorInvalidValue;
  const cudaError_t e = launch_behind(tiles_kernel<kDim, kStreams, kSplit>, dim3(grid), kThreadsTiles,
                                      T::smem(a.s.batch), stream, a);
  if (e != cudaSuccess) return e;
  return launch_join<kDim, T::kRows>(a, grid, stream);
}

}  // namespace

cudaError_t launch_tiles(const Attn& a, int dim, int32_t tile, int grid, cudaStream_t stream) {
  using Launch = cudaError_t (*)(const Attn&, int, cudaStream_t);
  static const Launch launch[2][2][2] = {
      {{launch_shape<64, 1, true>, launch_shape<64, 1, false>}, {launch_shape<64, 2, true>, launch_shape<64, 2, false>}},
      {{launch_shape<128, 1, true>, launch_shape<128, 1, false>},
       {launch_shape<128, 2, true>, launch_shape<128, 2, false>}}};
  return launch[dim == 128][tile == 256][a.bf16 != 0](a, grid, stream);
}

}  // namespace kv4
}  // namespace dspark
