// kv4_join.cuh -- the kernel that joins the partial sums of units that the
// CTAs' runs of blocks have cut.
#pragma once

#include "kv4_attn.cuh"

namespace dspark {
namespace kv4 {
namespace {

constexpr int32_t kLeast = 1;  // blocks of a run

// Joins a unit's parts: one warp for each row and head.  Rows whose unit has
// no blocks are written here too.
constexpr int kJoinWarps = 8;

template <int kDim, int kRows>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ Attn a, int grid) {
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
  const int32_t tile = in_grid / kRows, in_tile = in_grid % kRows;
  Tile x{0, 0, 0, 0};
  int32_t before = 0;
  if (r.len > 0) {
    for (int32_t t = 0; t < tile; ++t) {
      x = make_tile<kRows>(a, r, t);
      before += (x.hi - x.lo) * a.heads;
    }
    x = make_tile<kRows>(a, r, tile);
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
                              slot_floats<kRows, kDim>();
    };
    for (int32_t c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, slot_of(c)[kRows * kDim + in_tile]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    for (int32_t c = c0; c <= c1; ++c) {
      const float* p = slot_of(c);
      const float w = ex2(p[kRows * kDim + in_tile] - top);
      sum += p[kRows * (kDim + 1) + in_tile] * w;
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

template <int kDim, int kRows>
cudaError_t launch_join(const Attn& a, int grid, cudaStream_t stream) {
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
  return cudaLaunchKernelEx(&cfg, join_kernel<kDim, kRows>, a, grid);
}

}  // namespace
}  // namespace kv4
}  // namespace dspark
