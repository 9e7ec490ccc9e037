// kv4_join.cuh -- the kernel that joins the partial sums of units that the
// CTAs' runs of blocks have cut.
#pragma once

#include "kv4_attn.cuh"

namespace dspark {
namespace kv4 {
namespace {

// CTA (c, y) joins the parts of the unit that run c starts and its end cuts, rows
// 64 y to 64 y + 63, a warp a row at a time.  The CTAs also share the requests
// with more rows than tokens: rows at negative positions, which no block may
// reach, become 0.
constexpr int kJoinWarps = 16;
constexpr int kJoinRows = 64;
constexpr int kJoinDepth = 4;  // parts whose loads are in flight together

template <int kDim, int kRows>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ Attn a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t q_heads = a.heads * a.group;
  constexpr int kPer = kDim / 32;  // dimensions of a lane
  struct alignas(4 * kPer) Lane {
    float x[kPer];
  };

  for (int32_t i = blockIdx.x + gridDim.x * blockIdx.y; i < a.s.batch; i += gridDim.x * gridDim.y) {
    const Request r = load_request(a.s, i);
    const int64_t none = static_cast<int64_t>(max(r.rows - r.len, 0)) * q_heads;
    for (int64_t j = warp; j < none; j += kJoinWarps) {
      const int64_t row = r.start + j / q_heads, h = j % q_heads;
      uint16_t* out = a.out + row * a.out_row + h * a.out_head + lane * kPer;
#pragma unroll
      for (int u = 0; u < kPer; ++u) out[u] = 0;
      if (a.lse && lane == 0) a.lse[row * q_heads + h] = -INFINITY;
    }
  }
  // Every CTA waits, so that this kernel ends after the one before it.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Cut cut = a.cuts[blockIdx.x];
  if (cut.parts < 0) {  // nothing was computed
    __syncthreads();
    for (int32_t i = blockIdx.x + gridDim.x * blockIdx.y; i < a.s.batch; i += gridDim.x * gridDim.y) {
      const Request r = load_request(a.s, i);
      for (int64_t j = warp; j < static_cast<int64_t>(r.rows) * q_heads; j += kJoinWarps) {
        const int64_t row = r.start + j / q_heads, h = j % q_heads;
        uint16_t* out = a.out + row * a.out_row + h * a.out_head + lane * kPer;
#pragma unroll
        for (int u = 0; u < kPer; ++u) out[u] = 0x7FFF;  // NaN in either type
        if (a.lse && lane == 0) a.lse[row * q_heads + h] = NAN;
      }
    }
    return;
  }
  if (cut.parts == 0) return;
  const int32_t rows = cut.rows, first = cut.first;
  const int32_t c0 = blockIdx.x, c1 = c0 + cut.parts - 1;
  const auto slot_of = [&](int32_t c) {
    return a.partials + (2 * static_cast<int64_t>(c) + (c == c0 ? 1 : 0)) * slot_floats<kRows, kDim>();
  };
  const float gv = a.c.v_scale ? a.c.v_scale[cut.head] : 1.0f;

  for (int32_t in_tile = kJoinRows * blockIdx.y + warp; in_tile < min(rows, kJoinRows * (static_cast<int>(blockIdx.y) + 1));
       in_tile += kJoinWarps) {
    // The first parts' sums are asked for before anything waits for maxima.
    Lane v[kJoinDepth];
    const auto load = [&](int32_t c) {
#pragma unroll
      for (int j = 0; j < kJoinDepth; ++j) {
        v[j] = Lane{};
        if (c + j <= c1) v[j] = *reinterpret_cast<const Lane*>(slot_of(c + j) + in_tile * kDim + lane * kPer);
      }
    };
    load(c0);
    float top = kNone;
    for (int32_t c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, slot_of(c)[kRows * kDim + in_tile]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    float y[kPer], sum = 0.0f;
#pragma unroll
    for (int u = 0; u < kPer; ++u) y[u] = 0.0f;
    for (int32_t base = c0; base <= c1; base += 32) {  // 32 parts: a lane each for their weights
      float w = 0.0f, l = 0.0f;
      if (base + lane <= c1) {
        const float* p = slot_of(base + lane);
        w = ex2(p[kRows * kDim + in_tile] - top);
        l = p[kRows * (kDim + 1) + in_tile] * w;
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
      sum += l;
      const int32_t n = min(c1 - base + 1, 32);
      for (int32_t j0 = 0; j0 < n; j0 += kJoinDepth) {
        if (base + j0 > c0) load(base + j0);
#pragma unroll
        for (int j = 0; j < kJoinDepth; ++j) {
          const float wj = __shfl_sync(0xFFFFFFFFu, w, j0 + j);
#pragma unroll
          for (int u = 0; u < kPer; ++u) y[u] += v[j].x[u] * wj;
        }
      }
    }
    const int32_t i = (first + in_tile) / a.group;
    const int32_t h = cut.head * a.group + (first + in_tile - i * a.group);
    const int64_t row = cut.start + i;
    const float by = sum == 0.0f ? 0.0f : gv / sum;
    uint16_t* out = a.out + row * a.out_row + h * a.out_head + lane * kPer;
#pragma unroll
    for (int u = 0; u < kPer; u += 2) {
      const uint32_t w = pack_out(a.bf16, y[u] * by, y[u + 1] * by);
      out[u] = w & 0xFFFFu, out[u + 1] = w >> 16;
    }
    if (a.lse && lane == 0) a.lse[row * q_heads + h] = sum == 0.0f ? -INFINITY : (top - kShift + log2f(sum)) * kLn2;
  }
}

template <int kDim, int kRows>
cudaError_t launch_join(const Attn& a, int grid, cudaStream_t stream) {
  return launch_behind(join_kernel<kDim, kRows>, dim3(grid, (kRows + kJoinRows - 1) / kJoinRows), 32 * kJoinWarps,
                       0, stream, a);
}

}  // namespace
}  // namespace kv4
}  // namespace dspark
