// kv4.cuh -- the paged 4-bit cache's format on the device (include/dspark_kv4.h):
// where a token's codes and scales are, E2M1 and E4M3 conversion, and the
// lookup of a step's rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "dspark_kv4.h"
#include "kernels.h"
#include "ptx.cuh"

namespace dspark {
namespace kv4 {

// A cache as the kernels see it (validated on the host).
struct Cache {
  uint8_t* data;
  int64_t page_stride;
  int32_t num_pages;
  int32_t page_size;
  int32_t page_shift;  // log2(page_size)
  int32_t kv_heads;
  const float* k_scale;
  const float* v_scale;
};

// Tokens of a request: positions, less a window and a tile's rows or a block
// more, stay within 32 bits.
constexpr int32_t kMostTokens = 0x7FFFFFFF - 4096;

struct Batch {
  int32_t batch;
  int32_t total_rows;
  int32_t max_pages;
  int32_t max_slots;
  int32_t max_tokens;  // max_pages * page_size, at most kMostTokens
  const int32_t* row_start;  // null: row i is request i's, if its length is not negative (a selection's rows)
  const int32_t* slots;
  const int32_t* lens;
  const int32_t* table;
  int64_t table_stride;
};

// A request's rows: first row, number of rows, cached tokens, page table row.
struct Request {
  int32_t start;
  int32_t rows;
  int32_t len;
  const int32_t* pages;
};

__device__ __forceinline__ Request load_request(const Batch& s, int32_t i) {
  Request r;
  if (!s.row_start) {
    const int32_t len = s.lens[i];
    r.start = i;
    r.rows = len >= 0;
    r.len = min(max(len, 0), s.max_tokens);
    r.pages = s.table + static_cast<int64_t>(i) * s.table_stride;
    return r;
  }
  int32_t a = s.row_start[i], b = s.row_start[i + 1];
  const int32_t slot = s.slots ? s.slots[i] : i;
  a = min(max(a, 0), s.total_rows);
  b = min(max(b, a), s.total_rows);
  r.start = a;
  r.rows = b - a;
  r.len = 0;
  r.pages = s.table;
  if (slot < 0 || slot >= s.max_slots) return r;  // no tokens
  r.len = min(max(s.lens[slot], 0), s.max_tokens);
  r.pages = s.table + static_cast<int64_t>(slot) * s.table_stride;
  return r;
}

// The request that has row `row`, or -1: the last i with row_start[i] <= row.
__device__ __forceinline__ int32_t find_request(const Batch& s, int32_t row) {
  int32_t lo = 0, hi = s.batch;  // row_start[lo] <= row < row_start[hi], if at all
  if (s.row_start[0] > row || s.row_start[s.batch] <= row) return -1;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (s.row_start[mid] <= row) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The same by a whole warp, for one row: each round looks at 32 places at once.
__device__ __forceinline__ int32_t find_request_warp(const Batch& s, int32_t row) {
  const int lane = threadIdx.x & 31;
  int32_t lo = 0, hi = s.batch;  // row_start[lo] <= row < row_start[hi], if at all
  const int32_t end = s.row_start[s.batch];
  while (hi > lo) {
    const int32_t step = (hi - lo + 31) / 32, at = lo + lane * step;
    const uint32_t here = __ballot_sync(0xFFFFFFFFu, at < hi && s.row_start[at] <= row);
    if (here == 0) return -1;  // before the first request's rows
    const int32_t last = lo + (31 - __clz(here)) * step;
    if (step == 1) return end > row ? last : -1;
    lo = last, hi = min(last + step, hi);
  }
  return -1;
}

// Byte offsets inside a head's record.
template <int kDim>
struct Record {
  static constexpr int kCodeBytes = kDim / 2;    // of a token, keys or values
  static constexpr int kScaleBytes = kDim / 16;  // the same
  static __host__ __device__ __forceinline__ int bytes(int page) { return page * (kDim + kDim / 8); }
  static __device__ __forceinline__ int codes(int page, int which) { return which * page * kCodeBytes; }
  static __device__ __forceinline__ int scales(int page, int which) {
    return 2 * page * kCodeBytes + which * page * kScaleBytes;
  }
};

// Two E2M1 codes (a byte) to FP16x2, the low four bits to the low half; all
// four bytes of a word at once.  Exact.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&out)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
      : "r"(w));
}

// Two E4M3 scales to FP16x2, exact; a NaN reads as 448 (min drops a NaN).
__device__ __forceinline__ uint32_t scales_to_f16(uint32_t two) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(two)));
  asm("min.f16x2 %0, %0, %1;" : "+r"(d) : "r"(0x5F005F00u));  // 448 = 0x5F00
  return d;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// An inclusive scan over the warp with the sum add(before, behind).
template <typename Add>
__device__ __forceinline__ int32_t scan_warp(int32_t v, Add add) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t u = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v = add(v, u);
  }
  return v;
}

// ---- host side -------------------------------------------------------------
inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The arguments as the kernels take them, or a DSPARK_ERR_* code.
int make_cache(const dspark_kv4_cache* c, Cache* out);
int make_batch(const dspark_kv4_batch* b, const Cache& c, Batch* out);

// A kernel's shared-memory limit, set once per device context.  `registers`: what
// it has to be compiled to, a thread (0: anything); a kernel that gives its
// warps other shares waits for ever for registers that it was not launched with.
constexpr int kMaxDevices = 64;
struct SmemAttr {
  std::atomic<unsigned long long> ctx[kMaxDevices];
};
template <typename Kernel>
bool smem_attr_ready(SmemAttr& attr, Kernel kernel, int bytes, int registers = 0) {
  int device = -1;
  if (cudaGetDevice(&device) != cudaSuccess || device < 0 || device >= kMaxDevices) {
    (void)cudaGetLastError();
    return false;
  }
  const unsigned long long ctx = current_context_id();
  if (ctx != 0 && attr.ctx[device].load(std::memory_order_acquire) == ctx) return true;
  cudaFuncAttributes made{};
  if ((registers > 0 && (cudaFuncGetAttributes(&made, kernel) != cudaSuccess || made.numRegs != registers)) ||
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
    (void)cudaGetLastError();
    return false;
  }
  attr.ctx[device].store(ctx, std::memory_order_release);
  return true;
}

// A kernel that may be launched while the one before it runs: it waits for that
// one (griddepcontrol.wait) before it touches memory that it may write.
template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t stream,
                          Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace kv4
}  // namespace dspark
