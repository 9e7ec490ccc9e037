// logits_adjust.cu -- the tokens that requests have said, and logits adjusted by
// them (include/dspark_logits.h).
//
// dspark_logits_adjust passes over [rows, vocab] once: with out apart from logits
// that is what bounds it.  What makes a logit more than a copy (a token that the
// request holds, one of the drafts, one with a bias) concerns a few tokens of a
// hundred, so that a pass that decided token by token would spend its time on
// divergent branches.  A CTA takes 2048 tokens of a request and all of its rows:
//   1. it lists the tokens of its part that are touched at all, from the two bit
//      planes (a bit a token each), the drafts and the biases, and fetches their
//      counts;
//   2. it copies the rows, 16 bytes a thread at a time, with the masks applied;
//   3. it computes the touched tokens of all rows, a thread each, and stores them
//      over what step 2 left.
// In place step 2 writes only what a mask rules out.
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
constexpr int kCountThreads = 256;

__global__ void __launch_bounds__(kCountThreads)
    clear_kernel(dspark_token_table t, int32_t n, const int32_t* slots, int32_t words) {
  for (int32_t i = blockIdx.y; i < n; i += gridDim.y) {
    const int32_t slot = slots ? slots[i] : i;
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

template <typename Id>
__global__ void __launch_bounds__(kCountThreads)
    count_kernel(dspark_token_table t, int32_t n, const int32_t* slots, const Id* tokens, int64_t stride, int32_t width,
                 const int32_t* lens, int32_t prompt, int32_t words) {
  for (int32_t i = blockIdx.y; i < n; i += gridDim.y) {
    const int32_t slot = slots ? slots[i] : i;
    if (slot < 0 || slot >= t.max_slots) continue;
    const int32_t len = min(max(lens[i], 0), width);
    int32_t* counts = t.counts + slot * t.counts_stride;
    int32_t* marks = t.marks + slot * t.marks_stride + (prompt ? 0 : words);
    for (int64_t at = blockIdx.x * kCountThreads + threadIdx.x; at < len; at += gridDim.x * kCountThreads) {
      const int64_t id = tokens[i * stride + at];
      if (id < 0 || id >= t.vocab) continue;
      const int32_t bit = static_cast<int32_t>(1u << (id & 31));
      if (!(__ldcg(marks + (id >> 5)) & bit)) atomicOr(marks + (id >> 5), bit);  // most tokens come again
      if (!prompt) atomicAdd(counts + id, 1);
    }
  }
}

// ---- logits -----------------------------------------------------------------
constexpr int kThreads = 256;
constexpr int kTile = 2048;             // tokens of a CTA
constexpr int kPer = kTile / kThreads;  // tokens of a thread

struct Adjust {
  dspark_adjust_args a;
  dspark_token_table t;
  int32_t words;  // of a mask's row, and of a plane of marks
  int32_t tiles;
  int32_t penalties;  // any of the three
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

// The mask of a row of logits, or null.
__device__ __forceinline__ const int32_t* mask_of(const Adjust& p, int64_t row) {
  if (!p.a.mask) return nullptr;
  const int64_t at = p.a.mask_row ? p.a.mask_row[row] : row;
  return at >= 0 && at < p.a.mask_rows ? p.a.mask + at * p.a.mask_stride : nullptr;
}

template <typename In, typename Out, bool kVec, bool kInPlace>
__global__ void __launch_bounds__(kThreads) adjust_kernel(const __grid_constant__ Adjust p) {
  __shared__ uint32_t prompt[kTile / 32], touched[kTile / 32];
  __shared__ uint16_t list[kTile];   // touched tokens
  __shared__ int32_t said[kTile];    // how often, of each listed one
  __shared__ float biases[kTile];    // of each token
  __shared__ int32_t drafts[DSPARK_ADJUST_MAX_DRAFTS + 1];
  __shared__ int32_t warp_sum[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t i = blockIdx.x / p.tiles, tile = blockIdx.x % p.tiles, v0 = tile * kTile;
  const int32_t rows = p.a.drafts + 1, vocab = p.a.vocab;
  const int32_t slot = p.a.slots ? p.a.slots[i] : i;
  const bool known = slot >= 0 && slot < p.a.max_slots;
  const int64_t row0 = static_cast<int64_t>(i) * rows;
  const In* logits = static_cast<const In*>(p.a.logits) + row0 * p.a.logits_stride;
  Out* out = static_cast<Out*>(p.a.out) + row0 * p.a.out_stride;

  // 1. what is touched
  const int32_t* counts = nullptr;
  if (tid < kTile / 32) {
    uint32_t held = 0, any = 0;
    const int32_t w = v0 / 32 + tid;
    if (known && p.penalties && p.t.marks && w < p.words) {
      const int32_t* marks = p.t.marks + slot * p.t.marks_stride + w;
      held = marks[0];
      any = held | marks[p.words];
    }
    prompt[tid] = held;
    touched[tid] = any;
  }
  if (known && p.penalties && p.t.marks) counts = p.t.counts + slot * p.t.counts_stride + v0;
  int32_t entry = 0, entries = 0;
  if (known && p.a.bias_start) {
    const int64_t most = p.a.bias_entries;
    const int64_t lo = p.a.bias_start[slot], hi = p.a.bias_start[slot + 1];
    entry = static_cast<int32_t>(min(max(lo, int64_t{0}), most));
    entries = static_cast<int32_t>(min(max(hi, int64_t{0}), most));
  }
  if (entry < entries)
    for (int u = tid; u < kTile; u += kThreads) biases[u] = 0.0f;
  __syncthreads();
  const bool drafted = known && p.penalties && p.a.drafts > 0;
  if (drafted) {
    for (int32_t d = tid; d < p.a.drafts; d += kThreads) {
      const int64_t id = p.a.draft[i * p.a.draft_stride + d];
      const bool here = id >= v0 && id - v0 < kTile && id < vocab;
      drafts[d] = here ? static_cast<int32_t>(id - v0) : -1;
      if (here) atomicOr(&touched[(id - v0) >> 5], 1u << (id & 31));
    }
  }
  if (entry < entries && warp == 0) {  // in order: 32 entries at a time, equal ids one after another
    for (int32_t e = entry; e < entries; e += 32) {
      const int32_t id = e + lane < entries ? p.a.bias_id[e + lane] : -1;
      const bool here = id >= v0 && id - v0 < kTile && id < vocab;
      const float b = here ? p.a.bias[e + lane] : 0.0f;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, here ? id : -1 - lane);
      const int nth = __popc(same & ((1u << lane) - 1));
      for (int k = 0; __any_sync(0xFFFFFFFFu, here && nth >= k); ++k) {
        if (here && nth == k) {
          biases[id - v0] += b;
          if (k == 0) atomicOr(&touched[(id - v0) >> 5], 1u << (id & 31));
        }
        __syncwarp();
      }
    }
  }
  __syncthreads();
  int32_t items = 0;
  {
    const uint32_t mine = touched[tid * kPer / 32] >> (tid * kPer % 32) & ((1u << kPer) - 1);
    const int32_t n = __popc(mine);
    const int32_t upto = kv4::scan_warp(n, [](int32_t a, int32_t b) { return a + b; });
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    int32_t at = upto - n;
    for (int w = 0; w < kThreads / 32; ++w) {
      at += w < warp ? warp_sum[w] : 0;
      items += warp_sum[w];
    }
    for (uint32_t m = mine; m != 0; m &= m - 1) {
      const int u = tid * kPer + __ffs(m) - 1;
      list[at] = static_cast<uint16_t>(u);
      said[at++] = counts ? counts[u] : 0;
    }
  }

  // 2. the rows, 16 bytes at a time on the wider side
  if (kVec) {
    constexpr int kN = 16 / (sizeof(In) > sizeof(Out) ? sizeof(In) : sizeof(Out));
    constexpr int kParts = kPer / kN;  // of a row
    constexpr int kRows = 4;           // in flight
    for (int32_t r0 = 0; r0 < rows; r0 += kRows) {
      Pack<In, kN> x[kRows][kParts];
      uint32_t allow[kRows][kParts];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        if (r0 + u >= rows) continue;
        const int32_t* mask = mask_of(p, row0 + r0 + u);
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
          const int32_t v = v0 + (k * kThreads + tid) * kN;
          allow[u][k] = ~0u;
          if (v >= vocab) continue;
          if (mask) allow[u][k] = static_cast<uint32_t>(mask[v / 32]) >> (v % 32);
          if (kInPlace) continue;
          const In* from = logits + (r0 + u) * p.a.logits_stride + v;
          if (v + kN <= vocab) {
            x[u][k] = *reinterpret_cast<const Pack<In, kN>*>(from);
          } else {
#pragma unroll
            for (int e = 0; e < kN; ++e) x[u][k].x[e] = v + e < vocab ? from[e] : In{};
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        if (r0 + u >= rows) continue;
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
          const int32_t v = v0 + (k * kThreads + tid) * kN;
          if (v >= vocab) continue;
          Out* to = out + (r0 + u) * p.a.out_stride + v;
          Pack<Out, kN> y;
          const uint32_t all = (1u << kN) - 1, may = allow[u][k] & all;
          if (kInPlace && may == all) continue;
#pragma unroll
          for (int e = 0; e < kN; ++e)
            y.x[e] = may >> e & 1 ? (kInPlace ? Out{} : from_float<Out>(to_float(x[u][k].x[e]))) : from_float<Out>(-INFINITY);
          if (v + kN <= vocab && (!kInPlace || may == 0)) {
            *reinterpret_cast<Pack<Out, kN>*>(to) = y;
          } else {
#pragma unroll
            for (int e = 0; e < kN; ++e)
              if (v + e < vocab && !(kInPlace && may >> e & 1)) to[e] = y.x[e];
          }
        }
      }
    }
  } else {
    for (int32_t r = 0; r < rows; ++r) {
      const int32_t* mask = mask_of(p, row0 + r);
      if (kInPlace && !mask) continue;
      const In* from = logits + r * p.a.logits_stride;
      Out* to = out + r * p.a.out_stride;
      In x[kPer];
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int32_t v = v0 + u * kThreads + tid;
        if (!kInPlace && v < vocab) x[u] = from[v];
      }
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int32_t v = v0 + u * kThreads + tid;
        if (v >= vocab) continue;
        const bool may = !mask || (static_cast<uint32_t>(mask[v / 32]) >> (v % 32) & 1);
        if (!may) to[v] = from_float<Out>(-INFINITY);
        else if (!kInPlace) to[v] = from_float<Out>(to_float(x[u]));
      }
    }
  }
  __syncthreads();

  // 3. the touched tokens of all rows
  if (items == 0) return;
  const float rep = p.a.repetition ? p.a.repetition[slot] : 1.0f;
  const float freq = p.a.frequency ? p.a.frequency[slot] : 0.0f;
  const float pres = p.a.presence ? p.a.presence[slot] : 0.0f;
  for (int64_t at = tid; at < static_cast<int64_t>(items) * rows; at += kThreads) {
    const int32_t r = static_cast<int32_t>(at / items), k = static_cast<int32_t>(at - static_cast<int64_t>(r) * items);
    const int32_t u = list[k], v = v0 + u;
    if (v >= vocab) continue;  // a bit behind the last token
    Out* to = out + r * p.a.out_stride + v;
    const int32_t* mask = mask_of(p, row0 + r);
    if (mask && !(static_cast<uint32_t>(mask[v / 32]) >> (v % 32) & 1)) continue;  // is -inf
    float l = to_float(logits[r * p.a.logits_stride + v]);
    int32_t n = said[k];
    if (drafted)
      for (int32_t d = 0; d < r; ++d) n += drafts[d] == u;
    if (p.a.repetition && (n > 0 || (prompt[u / 32] >> (u % 32) & 1))) l = l > 0.0f ? __fdiv_rn(l, rep) : __fmul_rn(l, rep);
    if (n > 0) l = __fsub_rn(__fsub_rn(l, __fmul_rn(freq, static_cast<float>(n))), pres);
    if (entry < entries) l = __fadd_rn(l, biases[u]);
    *to = from_float<Out>(l);
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
  const unsigned grid = static_cast<unsigned>(p.a.batch) * static_cast<unsigned>(p.tiles);
  if (in_place) {
    if (vec) adjust_kernel<In, Out, true, kMayBeInPlace><<<grid, kThreads, 0, stream>>>(p);
    else adjust_kernel<In, Out, false, kMayBeInPlace><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (vec) adjust_kernel<In, Out, true, false><<<grid, kThreads, 0, stream>>>(p);
    else adjust_kernel<In, Out, false, false><<<grid, kThreads, 0, stream>>>(p);
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
  unsigned parts = static_cast<unsigned>((static_cast<int64_t>(width) + 4 * kCountThreads - 1) / (4 * kCountThreads));
  if (parts > 256) parts = 256;
  if (wide)
    count_kernel<<<dim3(parts, lists), kCountThreads, 0, stream>>>(*table, n, slots, static_cast<const int64_t*>(tokens),
                                                                   stride, width, lens, prompt, words);
  else
    count_kernel<<<dim3(parts, lists), kCountThreads, 0, stream>>>(*table, n, slots, static_cast<const int32_t*>(tokens),
                                                                   stride, width, lens, prompt, words);
  return cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
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
  if (a.drafts > 0 && a.draft_stride < a.drafts) return DSPARK_ERR_INVALID_ARG;
  const bool any_bias = a.bias_start || a.bias_id || a.bias;
  if (any_bias && (!a.bias_start || a.bias_entries < 0 || (a.bias_entries > 0 && (!a.bias_id || !a.bias))))
    return DSPARK_ERR_INVALID_ARG;
  p.words = static_cast<int32_t>((static_cast<int64_t>(a.vocab) + 31) / 32);
  if (a.mask && (a.mask_stride < p.words || a.mask_rows < 0)) return DSPARK_ERR_INVALID_ARG;
  if (!aligned(a.logits, in32 ? 4 : 2) || !aligned(a.out, out32 ? 4 : 2) || !aligned(a.slots, 4) ||
      !aligned(a.draft, 8) || !aligned(a.repetition, 4) || !aligned(a.frequency, 4) || !aligned(a.presence, 4) ||
      !aligned(a.bias_start, 4) || !aligned(a.bias_id, 4) || !aligned(a.bias, 4) || !aligned(a.mask, 4) ||
      !aligned(a.mask_row, 4))
    return DSPARK_ERR_MISALIGNED;
  p.tiles = static_cast<int32_t>((static_cast<int64_t>(a.vocab) + kTile - 1) / kTile);
  if (static_cast<int64_t>(p.tiles) * a.batch > 0x7FFFFFFF) return DSPARK_ERR_INVALID_ARG;
  if (a.batch == 0) return DSPARK_OK;
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
