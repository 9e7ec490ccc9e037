// logits_adjust.cu -- the tokens that requests have said, and logits adjusted by
// them (include/dspark_logits.h).
//
// dspark_logits_adjust passes over [rows, vocab] once; with out apart from logits the
// memory's bytes bound it.  What makes a logit more than a copy (a token that the
// request holds, one of the drafts, one with a bias) concerns a few tokens of a
// hundred: a branch on it in every thread would be taken by every warp.  The work is
// a line of units, 512 tokens of a request and all of its rows; each warp has a run
// of them and works by itself, without a barrier.  For a unit it
//   1. lists the touched tokens, from the two bit planes (a bit a token each), the
//      drafts and the biases, and asks for their counts and logits;
//   2. copies the rows, 16 bytes a lane on the wider side, with the masks applied;
//   3. computes the listed tokens of all rows, a lane each, and stores them over
//      what it copied.
// Rows, bit planes and masks come into a ring by asynchronous copies, units ahead; a
// request's first drafts and biases stay in registers.  So nothing that a unit needs
// is waited for one after the other.  In place step 2 writes only what a mask rules
// out.
#include <cuda_bf16.h>
#include <math.h>

#include "dspark_logits.h"
#include "kv4.cuh"

namespace dspark {
namespace adjust {
namespace {

using kv4::aligned;

constexpr int32_t kMostVocab = 1 << 30;

// ---- the token table --------------------------------------------------------
// Bound by the bytes of the slots that are cleared.  A few tokens go straight to their
// slot, looked up first, since an atomic operation costs more than a load.  A long
// list's tokens are marked in a bit plane in shared memory, 8192 a CTA, whose words
// then go to the slot's one beside the other: random single words cost the L2 a
// sector each.
constexpr int kCountThreads = 256;
constexpr int kCountDepth = 4;  // tokens of a thread in flight

// Lists are numbered without a sign: the number behind a CTA's last may be 2^31 or more.
__global__ void __launch_bounds__(kCountThreads)
    clear_kernel(dspark_token_table t, int32_t n, const int32_t* slots, int32_t words) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // what is launched behind waits before it writes
  for (uint32_t i = blockIdx.y; i < static_cast<uint32_t>(n); i += gridDim.y) {
    const int32_t slot = slots ? slots[i] : static_cast<int32_t>(i);
    if (slot < 0 || slot >= t.max_slots) continue;
    int32_t* counts = t.counts + slot * t.counts_stride;
    int32_t* marks = t.marks + slot * t.marks_stride;
    const int32_t step = gridDim.x * kCountThreads, at = blockIdx.x * kCountThreads + threadIdx.x;
    int32_t done = 0;
    if ((reinterpret_cast<uintptr_t>(counts) & 15) == 0) {
      done = t.vocab / 4 * 4;
      for (int32_t v = at; v < t.vocab / 4; v += step) reinterpret_cast<int4*>(counts)[v] = make_int4(0, 0, 0, 0);
    }
    for (int64_t v = done + static_cast<int64_t>(at); v < t.vocab; v += step) counts[v] = 0;
    for (int64_t v = at; v < 2 * static_cast<int64_t>(words); v += step) marks[v] = 0;
  }
}

// What it reads before it waits was written before the kernel that clears the slots
// began.
template <typename Id>
__global__ void __launch_bounds__(kCountThreads)
    count_kernel(dspark_token_table t, int32_t n, const int32_t* slots, const Id* tokens, int64_t stride, int32_t width,
                 const int32_t* lens, int32_t prompt, int32_t words) {
  bool waited = false;
  for (uint32_t i = blockIdx.y; i < static_cast<uint32_t>(n); i += gridDim.y) {
    const int32_t slot = slots ? slots[i] : static_cast<int32_t>(i);
    if (slot < 0 || slot >= t.max_slots) continue;
    const int32_t len = min(max(lens[i], 0), width);
    int32_t* counts = t.counts + slot * t.counts_stride;
    int32_t* marks = t.marks + slot * t.marks_stride + (prompt ? 0 : words);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kCountThreads;
    for (int64_t at = blockIdx.x * kCountThreads + threadIdx.x; at < len; at += kCountDepth * step) {
      int64_t id[kCountDepth];
      int32_t held[kCountDepth];
#pragma unroll
      for (int u = 0; u < kCountDepth; ++u) {
        id[u] = at + u * step < len ? static_cast<int64_t>(tokens[i * stride + at + u * step]) : -1;
        if (id[u] >= t.vocab) id[u] = -1;
      }
      if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
      waited = true;
#pragma unroll
      for (int u = 0; u < kCountDepth; ++u) held[u] = id[u] >= 0 ? __ldcg(marks + (id[u] >> 5)) : 0;
#pragma unroll
      for (int u = 0; u < kCountDepth; ++u) {
        if (id[u] < 0) continue;
        const int32_t bit = static_cast<int32_t>(1u << (id[u] & 31));
        if (!(held[u] & bit)) atomicOr(marks + (id[u] >> 5), bit);
        if (!prompt) atomicAdd(counts + id[u], 1);
      }
    }
  }
  // Every thread waits, so that this kernel ends after the one before it.
  if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
}

constexpr int kLongThreads = 512;
constexpr int kLongTokens = 8192;    // of a CTA
// Taken from 2^19 tokens in lists of 4096 or more on (what the lists could hold: their
// lengths are on the device).  Measured without / with it, prompts into cleared
// slots of 129280 tokens: 1 x 16000 tokens 4.1 / 5.7 us, 64 x 4000 9.9 / 10.5, 64 x
// 32000 28.8 / 13.0; 8 x 131072 into 163840 29.7 / 9.6.
constexpr int kLongWidth = 4096;
constexpr int64_t kLongTotal = 1 << 19;
constexpr int kLongWords = 12288;    // of a plane that shared memory holds without asking for more

template <typename Id>
__global__ void __launch_bounds__(kLongThreads)
    count_long_kernel(dspark_token_table t, int32_t n, const int32_t* slots, const Id* tokens, int64_t stride,
                      int32_t width, const int32_t* lens, int32_t prompt, int32_t words) {
  extern __shared__ uint32_t plane[];
  const int tid = threadIdx.x;
  bool waited = false;
  for (uint32_t i = blockIdx.y; i < static_cast<uint32_t>(n); i += gridDim.y) {
    const int32_t slot = slots ? slots[i] : static_cast<int32_t>(i);
    if (slot < 0 || slot >= t.max_slots) continue;
    const int32_t len = min(max(lens[i], 0), width);
    int32_t* counts = t.counts + slot * t.counts_stride;
    int32_t* marks = t.marks + slot * t.marks_stride + (prompt ? 0 : words);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kLongTokens;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * kLongTokens; first < len; first += step) {
      const int32_t here = static_cast<int32_t>(len - first < kLongTokens ? len - first : kLongTokens);
      const Id* from = tokens + i * stride + first;
      for (int32_t w = tid; w < words; w += kLongThreads) plane[w] = 0;
      __syncthreads();
      if (!prompt && !waited) {  // counts are written below
        asm volatile("griddepcontrol.wait;" ::: "memory");
        waited = true;
      }
      for (int32_t at = tid; at < here; at += kCountDepth * kLongThreads) {
        int64_t id[kCountDepth];
#pragma unroll
        for (int u = 0; u < kCountDepth; ++u)
          id[u] = at + u * kLongThreads < here ? static_cast<int64_t>(from[at + u * kLongThreads]) : -1;
#pragma unroll
        for (int u = 0; u < kCountDepth; ++u) {
          if (id[u] < 0 || id[u] >= t.vocab) continue;
          const uint32_t bit = 1u << (id[u] & 31);
          if (!(*const_cast<volatile uint32_t*>(&plane[id[u] >> 5]) & bit)) atomicOr(&plane[id[u] >> 5], bit);
          if (!prompt) atomicAdd(counts + id[u], 1);
        }
      }
      __syncthreads();
      if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
      waited = true;
      for (int32_t w = tid; w < words; w += kLongThreads)
        if (plane[w] != 0) atomicOr(marks + w, static_cast<int32_t>(plane[w]));
      __syncthreads();
    }
  }
  if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // as above
}

// ---- logits -----------------------------------------------------------------
constexpr int kWarps = 4;         // of a CTA
constexpr int kThreads = 32 * kWarps;
template <bool kVec>
constexpr int kCtas = kVec ? 5 : 4;  // of an SM: loads of single tokens take more registers
constexpr int kTile = 512;        // tokens of a unit
constexpr int kPer = kTile / 32;  // of a lane

struct Adjust {
  dspark_adjust_args a;
  dspark_token_table t;
  int32_t words;  // of a mask's row, and of a plane of marks
  int32_t tiles;
  int32_t penalties;  // any of the three
  uint32_t row_magic;  // 2^32 / rows rounded up: the quotient of a number below 2^20 is a product's high word
};

template <typename T>
__device__ __forceinline__ float to_float(T x) {
  return static_cast<float>(x);
}
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <typename T>
__device__ __forceinline__ T from_float(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float x) {
  return __float2bfloat16_rn(x);
}

// kN values that are read and written together.
template <typename T, int kN>
struct alignas(sizeof(T) * kN) Pack {
  T x[kN];
};

// The bits from token v on, of those in its word.
__device__ __forceinline__ uint32_t bits_at(const int32_t* words, int32_t v) {
  return static_cast<uint32_t>(words[v >> 5]) >> (v & 31);
}

// Where a listed token is in its unit, and what is to be known of it.
constexpr uint32_t kInPrompt = 1u << 9, kWithBias = 1u << 10, kInDraft = 1u << 11;
static_assert(kTile <= 1 << 9, "a place and three bits");

constexpr int kWords = kTile / 32;   // of a unit in a bit plane or a mask
constexpr int kMaskRows = 8;         // rows whose masks come with the unit; others are loaded
constexpr int kBiases = 2;           // groups of 32 of a request's biases that stay in registers

// A stage of a warp's ring is a unit's part of a row.  Measured, 64 requests of 6
// rows, 163840 tokens, BF16 to FP32, 384 MB: 2 / 3 / 4 stages 81 / 73 / 80 us (5.3
// TB/s; a copy of 250 MB runs at 6.1), with 4 or 6 CTAs of an SM 78 or 79; units of
// 256 tokens and stages of two rows 76 us, bound by the issue of instructions.
template <typename In>
constexpr int kStagesOf = sizeof(In) == 2 ? 3 : 2;

// What a warp holds in shared memory beside its ring.
template <int kStages>
struct alignas(16) Held {
  uint32_t marks[kStages][2 * kWords];           // of a unit: prompt, outputs
  uint32_t masks[kStages][kMaskRows * kWords];
  float biases[kTile];  // of the tokens that have one
  uint16_t list[kTile];
  uint32_t drafted[kWords], biased[kWords];
};

// kVec: 16 bytes at a time on the wider side, a lane has kN consecutive tokens of
// each of kParts parts of the unit; else one of each of 8 parts.
template <typename In, typename Out, bool kVec, bool kInPlace>
__global__ void __launch_bounds__(kThreads, kCtas<kVec>) adjust_kernel(const __grid_constant__ Adjust p) {
  constexpr int kN = kVec ? 16 / (sizeof(In) > sizeof(Out) ? sizeof(In) : sizeof(Out)) : 1;
  constexpr int kParts = kPer / kN;
  constexpr bool kRing = !kInPlace && kVec;
  constexpr int kRowBytes = kTile * static_cast<int>(sizeof(In));
  constexpr int kStages = kStagesOf<In>;
  constexpr uint32_t kAll = (1u << kN) - 1;
  using Piece = Pack<In, kN>;
  extern __shared__ __align__(16) uint8_t ring_bytes[];
  __shared__ Held<kStages> held_of[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Held<kStages>& mem = held_of[warp];
  uint8_t* const ring = ring_bytes + warp * (kStages * kRowBytes);
  const int32_t rows = p.a.drafts + 1, vocab = p.a.vocab;
  const int64_t units = static_cast<int64_t>(p.a.batch) * p.tiles, all = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t self = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t begin = units * self / all, end = units * (self + 1) / all;
  if (begin >= end) return;
  const auto token = [&](int k) { return (k * 32 + lane) * kN; };  // in the unit
  const auto slot_of = [&](int32_t i) {
    const int32_t slot = p.a.slots ? p.a.slots[i] : i;
    return slot >= 0 && slot < p.a.max_slots ? slot : -1;
  };
  // The mask's row for the logits' row r of request i, -1 for none.
  const auto mask_row = [&](int32_t i, int32_t r) {
    const int64_t row = static_cast<int64_t>(i) * rows + r;
    if (!p.a.mask || r >= rows) return -1;
    const int64_t m = p.a.mask_row ? p.a.mask_row[row] : row;
    return m >= 0 && m < p.a.mask_rows ? static_cast<int32_t>(m) : -1;
  };
  const bool planes = p.penalties && p.t.marks;

  // Stages are asked for ahead of their use.
  constexpr int kSize = static_cast<int>(sizeof(In));
  constexpr int kOf = 16 / kSize, kCopies = kRowBytes / 512;  // elements of a copy, copies of a row
  int32_t ask_i = static_cast<int32_t>(begin / p.tiles);
  int32_t ask_tile = static_cast<int32_t>(begin - static_cast<int64_t>(ask_i) * p.tiles);
  int32_t ask_row = 0, ask_stage = 0, ask_unit = 0, ask_slot = slot_of(ask_i), ask_mask = mask_row(ask_i, lane);
  int64_t ask_left = end - begin;
  const In* ask_from = static_cast<const In*>(p.a.logits) + static_cast<int64_t>(ask_i) * rows * p.a.logits_stride +
                       ask_tile * kTile + lane * kOf;  // of the next row
  const auto ask = [&]() {
    if (ask_left > 0) {
      if (ask_row == 0) {
        if (planes && ask_slot >= 0) {
          const int32_t w = ask_tile * kWords + lane % kWords;
          ptx::cp_async<4>(&mem.marks[ask_unit][lane],
                        p.t.marks + ask_slot * p.t.marks_stride + (lane < kWords ? 0 : p.words) + min(w, p.words - 1),
                        w < p.words ? 4 : 0);
        }
        if (p.a.mask) {
          const int32_t w = ask_tile * kWords + lane % kWords;
#pragma unroll
          for (int u = 0; u < kMaskRows; u += 32 / kWords) {
            if (u >= rows) break;
            const int32_t m = __shfl_sync(0xFFFFFFFFu, ask_mask, u + lane / kWords);
            if (m >= 0)
              ptx::cp_async<4>(&mem.masks[ask_unit][u * kWords + lane],
                            p.a.mask + m * p.a.mask_stride + min(w, p.words - 1), w < p.words ? 4 : 0);
          }
        }
      }
      if (kRing) {
        const int32_t left = vocab - ask_tile * kTile - lane * kOf;  // of the lane's first copy on
        uint8_t* to = ring + ask_stage * kRowBytes + lane * 16;
#pragma unroll
        for (int k = 0; k < kCopies; ++k) {
          const int32_t n = min(max(left - k * 32 * kOf, 0), kOf);
          ptx::cp_async<16>(to + k * 512, n > 0 ? ask_from + k * 32 * kOf : p.a.logits, n * kSize);
        }
        ask_from += p.a.logits_stride;
      }
      if (++ask_row == rows) {
        ask_row = 0, --ask_left;
        ask_unit = ask_unit + 1 == kStages ? 0 : ask_unit + 1;
        ask_from += kTile - rows * p.a.logits_stride;
        if (++ask_tile == p.tiles && ask_left > 0) {
          ask_from += rows * p.a.logits_stride - static_cast<int64_t>(p.tiles) * kTile;
          ask_tile = 0, ++ask_i;
          ask_slot = slot_of(ask_i), ask_mask = mask_row(ask_i, lane);
        }
      }
      ask_stage = ask_stage + 1 == kStages ? 0 : ask_stage + 1;
    }
    ptx::cp_async_commit();
  };
  int stage = 0, at_unit = 0;
  int32_t i = ask_i, tile = ask_tile - 1;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) ask();

  // of the request
  int32_t slot = -1, masks = -1;  // masks: of the rows, a lane each
  int32_t entry = 0, bias_id[kBiases];
  uint32_t entries = 0;  // biases from `entry` on
  float bias[kBiases], repetition = 1.0f, frequency = 0.0f, presence = 0.0f;
  int64_t draft = -1;
  bool drafting = false;
  for (int64_t unit = begin; unit < end; ++unit) {
    if (++tile == p.tiles || unit == begin) {  // another request
      if (unit != begin) tile = 0, ++i;
      slot = slot_of(i);
      masks = mask_row(i, lane);
      drafting = slot >= 0 && p.penalties && p.a.drafts > 0;
      draft = drafting && lane < p.a.drafts ? p.a.draft[i * p.a.draft_stride + lane] : -1;
      entry = 0, entries = 0;
      if (slot >= 0) {
        if (p.a.bias_start) {
          entry = min(max(p.a.bias_start[slot], 0), static_cast<int32_t>(p.a.bias_entries));
          const int32_t behind = min(max(p.a.bias_start[slot + 1], 0), static_cast<int32_t>(p.a.bias_entries));
          entries = max(behind - entry, 0);
        }
        if (p.a.repetition) repetition = p.a.repetition[slot];
        if (p.a.frequency) frequency = p.a.frequency[slot];
        if (p.a.presence) presence = p.a.presence[slot];
      }
#pragma unroll
      for (int g = 0; g < kBiases; ++g) {
        const uint32_t e = 32 * g + lane;
        bias_id[g] = e < entries ? p.a.bias_id[entry + e] : -1;
        bias[g] = e < entries ? p.a.bias[entry + e] : 0.0f;
      }
    }
    const int64_t row0 = static_cast<int64_t>(i) * rows;
    const int32_t v0 = tile * kTile;
    const In* logits = static_cast<const In*>(p.a.logits) + row0 * p.a.logits_stride;
    Out* out = static_cast<Out*>(p.a.out) + row0 * p.a.out_stride;
    const bool held = planes && slot >= 0;
    const auto allowed = [&](int32_t r, int32_t m, int32_t u) {  // bits from the unit's token u on
      if (m < 0) return ~0u;
      if (r < kMaskRows) return mem.masks[at_unit][r * kWords + (u >> 5)] >> (u & 31);
      return bits_at(p.a.mask + m * p.a.mask_stride, min(v0 + u, vocab - 1) & ~(kN - 1));
    };

    // without a ring a row's logits are asked for before the one before it is written
    Piece next[kRing || kInPlace ? 1 : kParts];
    const auto fetch = [&](int32_t r) {
#pragma unroll
      for (int k = 0; k < kParts; ++k)
        if (r < rows && v0 + token(k) < vocab) next[k].x[0] = logits[r * p.a.logits_stride + v0 + token(k)];
    };
    if (!kRing && !kInPlace) fetch(0);

    // 1. the touched tokens
    if (lane < kWords) mem.drafted[lane] = mem.biased[lane] = 0;
    ptx::cp_async_wait<kStages - 2>();
    __syncwarp();
    if (drafting) {
      for (int32_t d = lane; d < p.a.drafts; d += 32) {
        const int64_t u = (d < 32 ? draft : p.a.draft[i * p.a.draft_stride + d]) - v0;
        if (u >= 0 && u < kTile && u < vocab - v0) atomicOr(&mem.drafted[u >> 5], 1u << (u & 31));
      }
    }
    // biases in their order: 32 entries at a time, those of a token one after another
    const auto add_biases = [&](int32_t id, float b) {
      const int32_t u = id - v0;
      const bool here = id >= 0 && u >= 0 && u < kTile && u < vocab - v0;
      if (!__any_sync(0xFFFFFFFFu, here)) return;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, here ? u : -1 - lane);
      const int nth = __popc(same & ((1u << lane) - 1));
      for (int k = 0; __any_sync(0xFFFFFFFFu, here && nth >= k); ++k) {
        if (here && nth == k) mem.biases[u] = __fadd_rn(mem.biased[u >> 5] >> (u & 31) & 1 ? mem.biases[u] : 0.0f, b);
        __syncwarp();
        if (here && nth == k && k == 0) atomicOr(&mem.biased[u >> 5], 1u << (u & 31));
        __syncwarp();
      }
    };
    if (entries > 0) {
#pragma unroll
      for (int g = 0; g < kBiases; ++g)
        if (32 * g < entries) add_biases(bias_id[g], bias[g]);
      for (uint32_t e = 32 * kBiases + lane; e - lane < entries; e += 32)
        add_biases(e < entries ? p.a.bias_id[entry + e] : -1, e < entries ? p.a.bias[entry + e] : 0.0f);
    }
    __syncwarp();
    // a lane's tokens in the list: 16 in a row, whatever the rows' parts are
    int32_t listed;
    {
      constexpr int kLanes = 32 / kPer;  // of a word
      constexpr uint32_t kMine = (1u << kPer) - 1;
      const int w = lane / kLanes, first = lane % kLanes * kPer;
      const uint32_t prompt = held ? mem.marks[at_unit][w] >> first & kMine : 0u;
      const uint32_t said = held ? mem.marks[at_unit][kWords + w] >> first & kMine : 0u;
      const uint32_t drafted = mem.drafted[w] >> first & kMine, biased = mem.biased[w] >> first & kMine;
      uint32_t any = prompt | said | drafted | biased;
      const int32_t behind = vocab - v0 - kPer * lane;  // bits behind the last token are not
      if (behind < kPer) any &= (1u << max(behind, 0)) - 1;
      const int32_t mine = __popc(any);
      const int32_t upto = kv4::scan_warp(mine, [](int32_t a, int32_t b) { return a + b; });
      listed = __shfl_sync(0xFFFFFFFFu, upto, 31);
      for (int32_t at = upto - mine; any != 0; any &= any - 1) {
        const int e = __ffs(any) - 1;
        mem.list[at++] = static_cast<uint16_t>(kPer * lane + e | (prompt >> e & 1 ? kInPrompt : 0u) |
                                               (biased >> e & 1 ? kWithBias : 0u) | (drafted >> e & 1 ? kInDraft : 0u));
      }
    }
    __syncwarp();
    // the items of step 3: listed tokens by rows
    const int32_t items = listed * rows;
    struct Item {
      int32_t r, v, n;  // row, token, how often it was said
      uint32_t what;
      float l;
    };
    const auto item_of = [&](int32_t t) {
      Item x;
      const int32_t nth = rows == 1 ? t : static_cast<int32_t>(__umulhi(static_cast<uint32_t>(t), p.row_magic));
      x.r = t - nth * rows;
      x.what = mem.list[nth];
      x.v = v0 + static_cast<int32_t>(x.what & (kTile - 1));
      x.l = to_float(logits[x.r * p.a.logits_stride + x.v]);
      x.n = held ? p.t.counts[slot * p.t.counts_stride + x.v] : 0;
      return x;
    };
    Item ahead{};
    if (lane < items) ahead = item_of(lane);

    // 2. the rows
    for (int32_t r = 0; r < rows; ++r) {
      if (r > 0) {
        if (r % 32 == 0) masks = mask_row(i, r + lane);
        ptx::cp_async_wait<kStages - 2>();
        __syncwarp();
      }
      Piece x[kParts];
#pragma unroll
      for (int k = 0; k < kParts; ++k) {
        if (kRing) x[k] = *reinterpret_cast<const Piece*>(ring + stage * kRowBytes + token(k) * kSize);
        else if (!kInPlace) x[k] = next[k];
      }
      if (!kRing && !kInPlace) fetch(r + 1);
      stage = stage + 1 == kStages ? 0 : stage + 1;
      const int32_t m = p.a.mask ? __shfl_sync(0xFFFFFFFFu, masks, r & 31) : -1;  // the same for the whole warp
      uint32_t allow[kParts];
      if (m >= 0) {
#pragma unroll
        for (int k = 0; k < kParts; ++k) allow[k] = allowed(r, m, token(k)) & kAll;
      }
      ask();  // into the stage before, which every lane has read
      if (kInPlace && m < 0) continue;
      Out* const row = out + r * p.a.out_stride + v0;
      if (m < 0 && v0 + kTile <= vocab) {  // all of it as it is
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
          Pack<Out, kN> y;
#pragma unroll
          for (int e = 0; e < kN; ++e) y.x[e] = from_float<Out>(to_float(x[k].x[e]));
          *reinterpret_cast<Pack<Out, kN>*>(row + token(k)) = y;
        }
        continue;
      }
      if (!kInPlace && v0 + kTile <= vocab) {  // all of it, with a mask
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
          Pack<Out, kN> y;
#pragma unroll
          for (int e = 0; e < kN; ++e) y.x[e] = from_float<Out>(allow[k] & 1u << e ? to_float(x[k].x[e]) : -INFINITY);
          *reinterpret_cast<Pack<Out, kN>*>(row + token(k)) = y;
        }
        continue;
      }
#pragma unroll
      for (int k = 0; k < kParts; ++k) {
        const int32_t v = v0 + token(k);
        const uint32_t may = m < 0 ? kAll : allow[k];
        if (v >= vocab || (kInPlace && may == kAll)) continue;
        Pack<Out, kN> y;
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          y.x[e] = from_float<Out>(-INFINITY);
          if (!kInPlace && (may >> e & 1)) y.x[e] = from_float<Out>(to_float(x[k].x[e]));
        }
        if (v + kN <= vocab && !(kInPlace && may != 0)) {
          *reinterpret_cast<Pack<Out, kN>*>(row + token(k)) = y;
        } else {
#pragma unroll
          for (int e = 0; e < kN; ++e)
            if (v + e < vocab && !(kInPlace && may >> e & 1)) row[token(k) + e] = y.x[e];
        }
      }
    }
    __syncwarp();  // the copies are before what comes over them

    // 3. the touched tokens of all rows
    for (int32_t t0 = 0; t0 < items; t0 += 32) {
      if (t0 > 0 && t0 + lane < items) ahead = item_of(t0 + lane);
      const Item x = ahead;
      const int32_t m = !p.a.mask ? -1 : rows <= 32 ? __shfl_sync(0xFFFFFFFFu, masks, x.r) : mask_row(i, x.r);
      if (t0 + lane >= items) continue;
      const int32_t u = x.v - v0;
      if (m >= 0 && !((x.r < kMaskRows ? mem.masks[at_unit][x.r * kWords + (u >> 5)] >> (u & 31)
                                       : bits_at(p.a.mask + m * p.a.mask_stride, x.v)) & 1))
        continue;  // is -inf
      float l = x.l;
      int32_t n = x.n;
      if (x.what & kInDraft)
        for (int32_t d = 0; d < x.r; ++d) n += p.a.draft[i * p.a.draft_stride + d] == x.v;
      if (p.a.repetition && (n > 0 || (x.what & kInPrompt)))
        l = l > 0.0f ? __fdiv_rn(l, repetition) : __fmul_rn(l, repetition);
      if (n > 0) l = __fsub_rn(__fsub_rn(l, __fmul_rn(frequency, static_cast<float>(n))), presence);
      if (x.what & kWithBias) l = __fadd_rn(l, mem.biases[u]);
      out[x.r * p.a.out_stride + x.v] = from_float<Out>(l);
    }
    if (rows > 32) masks = mask_row(i, lane);
    at_unit = at_unit + 1 == kStages ? 0 : at_unit + 1;
    __syncwarp();  // before the list is written again
  }
}

int check_table(const dspark_token_table* t) {
  if (!t || t->vocab < 1 || t->vocab > kMostVocab || t->max_slots < 0) return DSPARK_ERR_INVALID_ARG;
  const int64_t words = (static_cast<int64_t>(t->vocab) + 31) / 32;
  if (t->counts_stride < t->vocab || t->marks_stride < 2 * words || (t->max_slots > 0 && (!t->counts || !t->marks)))
    return DSPARK_ERR_INVALID_ARG;
  return aligned(t->counts, 4) && aligned(t->marks, 4) ? DSPARK_OK : DSPARK_ERR_MISALIGNED;
}

template <typename In, typename Out, bool kMayBeInPlace>
cudaError_t launch(const Adjust& p, bool vec, bool in_place, cudaStream_t stream) {
  // as many warps as there are units, or what fills the SMs
  const int64_t ctas = (static_cast<int64_t>(p.a.batch) * p.tiles + kWarps - 1) / kWarps;
  const int most = 152 * (vec ? kCtas<true> : kCtas<false>);
  const unsigned grid = static_cast<unsigned>(ctas < most ? ctas : most);
  const int smem = vec && !in_place ? kWarps * kStagesOf<In> * kTile * static_cast<int>(sizeof(In)) : 0;
  if (in_place) {
    if (vec) adjust_kernel<In, Out, true, kMayBeInPlace><<<grid, kThreads, smem, stream>>>(p);
    else adjust_kernel<In, Out, false, kMayBeInPlace><<<grid, kThreads, smem, stream>>>(p);
  } else {
    if (vec) adjust_kernel<In, Out, true, false><<<grid, kThreads, smem, stream>>>(p);
    else adjust_kernel<In, Out, false, false><<<grid, kThreads, smem, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace adjust
}  // namespace dspark

extern "C" {

int dspark_tokens_count(const dspark_token_table* table, int32_t n, const int32_t* slots, const void* tokens,
                        int32_t wide, int64_t stride, int32_t width, const int32_t* lens, int32_t prompt,
                        int32_t reset, cudaStream_t stream) {
  using namespace dspark::adjust;
  const int rc = check_table(table);
  if (rc != DSPARK_OK) return rc;
  if (n < 0 || width < 0 || stride < width) return DSPARK_ERR_INVALID_ARG;
  if (!aligned(slots, 4) || !aligned(lens, 4) || !aligned(tokens, wide ? 8 : 4)) return DSPARK_ERR_MISALIGNED;
  if (n == 0 || table->max_slots == 0) return DSPARK_OK;
  if (!lens || (!tokens && width > 0)) return DSPARK_ERR_INVALID_ARG;
  const int32_t words = static_cast<int32_t>((static_cast<int64_t>(table->vocab) + 31) / 32);
  const unsigned lists = n < 65535 ? n : 65535;
  if (reset) {
    const unsigned parts = (table->vocab + 16 * kCountThreads - 1) / (16 * kCountThreads);
    clear_kernel<<<dim3(parts, lists), kCountThreads, 0, stream>>>(*table, n, slots, words);
    if (cudaGetLastError() != cudaSuccess) return DSPARK_ERR_CUDA;
  }
  if (width == 0) return DSPARK_OK;
  const bool is_long =
      width >= kLongWidth && static_cast<int64_t>(n) * width >= kLongTotal && words <= kLongWords;
  const int64_t of_cta = is_long ? kLongTokens : kCountDepth * kCountThreads;
  unsigned parts = static_cast<unsigned>((static_cast<int64_t>(width) + of_cta - 1) / of_cta);
  if (parts > 256) parts = 256;
  const dim3 grid(parts, lists);
  const int threads = is_long ? kLongThreads : kCountThreads, smem = is_long ? words * 4 : 0;
  const auto count = [&](auto id) {
    using Id = decltype(id);
    const Id* from = static_cast<const Id*>(tokens);
    const auto kernel = is_long ? count_long_kernel<Id> : count_kernel<Id>;
    if (reset)
      return dspark::kv4::launch_behind(kernel, grid, threads, smem, stream, *table, n, slots, from, stride, width,
                                        lens, prompt, words);
    kernel<<<grid, threads, smem, stream>>>(*table, n, slots, from, stride, width, lens, prompt, words);
    return cudaGetLastError();
  };
  return (wide ? count(int64_t{}) : count(int32_t{})) == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

int dspark_logits_adjust(const dspark_token_table* table, const dspark_adjust_args* args, cudaStream_t stream) {
  using namespace dspark::adjust;
  Adjust p{};
  if (!args) return DSPARK_ERR_INVALID_ARG;
  p.a = *args;
  const dspark_adjust_args& a = p.a;
  if (a.batch < 0 || a.drafts < 0 || a.vocab < 1 || a.vocab > kMostVocab || a.max_slots < 0)
    return DSPARK_ERR_INVALID_ARG;
  if (a.drafts > DSPARK_ADJUST_MAX_DRAFTS) return DSPARK_ERR_TOO_MANY_ROWS;
  if (table) {
    const int rc = check_table(table);
    if (rc != DSPARK_OK) return rc;
    if (table->vocab != a.vocab || table->max_slots != a.max_slots) return DSPARK_ERR_INVALID_ARG;
    p.t = *table;
  }
  const bool in32 = a.dtype == DSPARK_DTYPE_F32, out32 = a.out_dtype == DSPARK_DTYPE_F32;
  if ((!in32 && a.dtype != DSPARK_DTYPE_BF16) || (!out32 && a.out_dtype != DSPARK_DTYPE_BF16) || (in32 && !out32))
    return DSPARK_ERR_INVALID_ARG;
  if (a.logits_stride < a.vocab || a.out_stride < a.vocab) return DSPARK_ERR_INVALID_ARG;
  const bool in_place = a.logits == a.out;
  if (in_place && a.logits && (in32 != out32 || a.logits_stride != a.out_stride)) return DSPARK_ERR_INVALID_ARG;
  if (a.draft && a.draft_stride < a.drafts) return DSPARK_ERR_INVALID_ARG;
  const bool any_bias = a.bias_start || a.bias_id || a.bias;
  if (any_bias && (!a.bias_start || a.bias_entries < 0 || a.bias_entries > 0x7FFFFFFF ||
                   (a.bias_entries > 0 && (!a.bias_id || !a.bias))))
    return DSPARK_ERR_INVALID_ARG;
  p.words = static_cast<int32_t>((static_cast<int64_t>(a.vocab) + 31) / 32);
  if (a.mask && (a.mask_stride < p.words || a.mask_rows < 0 || a.mask_rows > 0x7FFFFFFF)) return DSPARK_ERR_INVALID_ARG;
  if (!aligned(a.logits, in32 ? 4 : 2) || !aligned(a.out, out32 ? 4 : 2) || !aligned(a.slots, 4) ||
      !aligned(a.draft, 8) || !aligned(a.repetition, 4) || !aligned(a.frequency, 4) || !aligned(a.presence, 4) ||
      !aligned(a.bias_start, 4) || !aligned(a.bias_id, 4) || !aligned(a.bias, 4) || !aligned(a.mask, 4) ||
      !aligned(a.mask_row, 4))
    return DSPARK_ERR_MISALIGNED;
  p.tiles = static_cast<int32_t>((static_cast<int64_t>(a.vocab) + kTile - 1) / kTile);
  if (a.batch == 0) return DSPARK_OK;
  p.row_magic = static_cast<uint32_t>(((int64_t{1} << 32) + a.drafts) / (a.drafts + 1));
  p.penalties = a.repetition || a.frequency || a.presence;
  if (!a.logits || !a.out || (a.drafts > 0 && p.penalties && !a.draft)) return DSPARK_ERR_INVALID_ARG;
  const auto wide = [](const void* ptr, int64_t stride, int bytes) {
    return aligned(ptr, 16) && stride * bytes % 16 == 0;
  };
  const bool vec = wide(a.logits, a.logits_stride, in32 ? 4 : 2) && wide(a.out, a.out_stride, out32 ? 4 : 2);
  const cudaError_t e = in32    ? launch<float, float, true>(p, vec, in_place, stream)
                        : out32 ? launch<__nv_bfloat16, float, false>(p, vec, false, stream)
                                : launch<__nv_bfloat16, __nv_bfloat16, true>(p, vec, in_place, stream);
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

}  // extern "C"
