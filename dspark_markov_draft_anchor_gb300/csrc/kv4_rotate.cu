// kv4_rotate.cu -- storing rows whose keys are rotated on the way, and rotating
// their queries (dspark_kv4_append_rotated of include/dspark_kv4.h).
//
//   a' = RN(RN(a c) - RN(b s)),  b' = RN(RN(b c) + RN(a s))
// for the pairs (a, b) of a head's first `dims` elements; keys go from these FP32
// values to codes as in kv4_cache.cu, queries are rounded once.  Bound by the
// memory: a row of 64 query heads on 8 of 128 dimensions is 32 KB of queries read
// and written, 4 KB of keys and values and 1.2 KB of codes and scales.
//
// A row's heads stand in a line, keys, values, queries; a thread takes the same 16
// elements of every 16th (128 dimensions) or 32nd head, so that it loads its 8
// cosines and sines once a row.  Its 16 elements are two groups of 8, far apart so
// that both loads and stores of neighbouring threads touch: with pairs of halves a
// group and the one that it is turned with, else groups half a head apart.  The
// scale of 16 elements then needs the maxima of two threads beside one another (one
// shuffle), each of which writes 4 bytes of codes.
#include "kv4_quant.cuh"

namespace dspark {
namespace kv4 {
namespace {

constexpr int kThreads = 128;
constexpr int kDepth = 5;     // heads a thread has in a stage
// Measured, 22 k rows of 64 and 8 heads of 128 dimensions, 840 MB: 3 stages and 3
// CTAs of an SM 152 us, 2 and 4 138 us (6.1 TB/s), 2 and 5 187 us (96 registers,
// which spill), 4 and 2 180 us.
constexpr int kStages = 2;
constexpr int kCtas = 4;      // of an SM
// Heads of a line, so that 31 bits count a stage's places (kDepth times 32 at most)
// behind the last one, too.
constexpr int32_t kMostHeads = 0x7FFFFFFF - 1024;

struct Rotate {
  Cache c;
  Batch s;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* q;
  uint16_t* out;
  int64_t k_row, k_head, v_row, v_head, q_row, q_head, out_row, out_head;
  const float* cos;
  const float* sin;
  int64_t stride;
  const int32_t* at;
  int32_t positions;
  int32_t dims;
  int32_t interleaved;
  int32_t table_vec;  // 16-byte loads of cos and sin
  int32_t heads;      // of the line: 2 kv_heads + q_heads
  int32_t part;       // heads of a CTA
};

struct Place {
  uint8_t* page;     // null: the row has no place
  int32_t in_page;
  int32_t turn;      // row of the table, or one of the following
};
constexpr int32_t kNoRow = -1;    // no request has the row
constexpr int32_t kNoPlace = -2;  // at a negative position: queries become 0
constexpr int32_t kNoTurn = -3;   // outside the table: queries become NaN

__device__ __forceinline__ Place find_place(const Rotate& p, int32_t row) {
  Place x{nullptr, 0, kNoRow};
  const int32_t i = find_request(p.s, row);
  if (i < 0) return x;
  const Request r = load_request(p.s, i);
  const int32_t j = row - r.start;
  if (j < 0 || j >= r.rows) return x;
  const int32_t pos = r.len - r.rows + j;
  x.turn = kNoPlace;
  if (pos < 0) return x;
  const int32_t turn = p.at ? p.at[row] : pos;
  x.turn = kNoTurn;
  if (turn < 0 || turn >= p.positions) return x;
  x.turn = turn;
  const int32_t id = r.pages[pos >> p.c.page_shift];
  if (id >= 0 && id < p.c.num_pages) x.page = p.c.data + static_cast<int64_t>(id) * p.c.page_stride;
  x.in_page = pos & (p.c.page_size - 1);
  return x;
}

// RN(x / d), for x of 24 bits: quotient() of kv4_quant.cuh wants a first quotient
// within one unit of its last place, which the product with RN(1 / d) alone does not
// give; one more step makes it so.  The same range.
__device__ __forceinline__ float quotient24(float x, float d, float inverse) {
  const float q = quotient(x, d, inverse);
  return __fmaf_rn(__fmaf_rn(-q, d, x), inverse, q);
}

// x / g (NaN as 0, what saturates every code held to 2^40).  By value: an array
// that a call may write would live in memory for the whole kernel.
struct Eight {
  float v[8];
};
__device__ __noinline__ Eight scale8_any(Eight x, float g) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = __fdiv_rn(x.v[i], g);
    x.v[i] = isnan(v) ? 0.0f : fminf(fmaxf(v, -0x1p40f), 0x1p40f);
  }
  return x;
}
// x / g in place; the largest.
__device__ __forceinline__ float scale8(float (&x)[8], const float* scale_of_head) {
  const float g = scale_of_head ? *scale_of_head : 1.0f, size = fabsf(g);
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(x[i]));
  if (!(top < 0x1p40f && size >= 0x1p-20f && size < 0x1p40f)) {
    Eight y{{x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]}};
    y = scale8_any(y, g);
    top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y.v[i], top = fmaxf(top, fabsf(x[i]));
    return top;
  }
  if (!scale_of_head) return top;
  const float inverse = __frcp_rn(g);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = quotient24(x[i], g, inverse);
  return fabsf(quotient24(top, g, inverse));  // rounding keeps the order: the largest stays the largest
}

// The codes of 8 quotients, of the scale `byte`.  A scale's significand is an odd
// number m below 16 (or the quotient exact), so that a quotient is at least 1 / (2 m)
// units from where rounding changes: one step of quotient() is enough.
__device__ __forceinline__ uint32_t encode8(const float (&y)[8], uint32_t byte) {
  const float scale = __half2float(__ushort_as_half(static_cast<uint16_t>(scales_to_f16(byte))));
  if (scale == 0.0f) return 0u;
  const float inverse = __frcp_rn(scale);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    w |= e2m1x2(quotient(y[i], scale, inverse), quotient(y[i + 1], scale, inverse)) << (4 * i);
  return w;
}

// A pair turned; each operation rounded.  (With packed pairs of FP32 products and sums
// some results were those of fused ones, although each asks for its own rounding.)
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

// The angles of a thread's 8 pairs in a row.
struct Angles {
  float c[8], s[8];
};

template <int kDim, bool kBf16, bool kVec>
__global__ void __launch_bounds__(kThreads, kCtas) rotate_kernel(const __grid_constant__ Rotate p) {
  using R = Record<kDim>;
  constexpr int kPer = kDim / 16;           // threads of a head
  constexpr int kStep = kThreads / kPer;    // heads of a CTA at a time
  extern __shared__ __align__(16) uint4 ring[];  // [stage][group][thread]
  __shared__ Place places[kThreads];
  const int tid = threadIdx.x, j = tid % kPer;
  const int32_t begin = static_cast<int32_t>(static_cast<int64_t>(p.s.total_rows) * blockIdx.x / gridDim.x);
  const int32_t end = static_cast<int32_t>(static_cast<int64_t>(p.s.total_rows) * (blockIdx.x + 1) / gridDim.x);
  const int32_t part0 = blockIdx.y * p.part, head_end = min(p.heads, part0 + p.part), head0 = part0 + tid / kPer;
  const int32_t parts = (head_end - part0 + kDepth * kStep - 1) / (kDepth * kStep);  // stages of a row
  const int32_t kv = p.c.kv_heads;
  // the thread's groups, and whether they are turned (pairs of halves: both or none)
  const int pairs = p.interleaved ? 0 : p.dims / 16;  // threads with a pair of groups
  const int e0 = j < pairs ? 8 * j : p.interleaved ? 8 * j : p.dims + 8 * (j - pairs);
  const int e1 = j < pairs           ? p.dims / 2 + 8 * j
                 : p.interleaved     ? kDim / 2 + 8 * j
                                     : p.dims + (kDim - p.dims) / 2 + 8 * (j - pairs);
  const bool turned0 = e0 < p.dims, turned1 = e1 < p.dims;

  const auto source = [&](int32_t row, int32_t h) {
    return (h < kv       ? p.k + row * p.k_row + h * p.k_head
            : h < 2 * kv ? p.v + row * p.v_row + (h - kv) * p.v_head
                         : p.q + row * p.q_row + (h - 2 * kv) * p.q_head) + e0;
  };
  // Stages are asked for ahead of their use; each thread reads only what it asked for.
  int32_t ask_row = begin, ask_part = 0, ask_stage = 0;
  const auto ask = [&]() {
    if (kVec && ask_row < end) {
      uint4* to = ring + ask_stage * (2 * kDepth * kThreads) + tid;
#pragma unroll
      for (int u = 0; u < kDepth; ++u) {
        const int32_t h = head0 + (ask_part * kDepth + u) * kStep;
        if (h >= head_end) continue;
        const uint16_t* from = source(ask_row, h);
        ptx::cp_async16(to + 2 * u * kThreads, from);
        ptx::cp_async16(to + (2 * u + 1) * kThreads, from + (e1 - e0));
      }
      if (++ask_part == parts) ask_part = 0, ++ask_row;
      ask_stage = ask_stage + 1 == kStages ? 0 : ask_stage + 1;
    }
    ptx::cp_async_commit();
  };
  const auto angles = [&](const Place& at) {
    Angles x{};
    if (at.turn < 0) return x;
#pragma unroll
    for (int g = 0; g < 2; ++g) {  // of group 0 and group 1, or of the first and the last 4 of 8 pairs
      const int from = p.interleaved ? (g ? e1 : e0) / 2 : e0 + 4 * g;
      if (!(g && p.interleaved ? turned1 : turned0)) continue;
      const float* c = p.cos + at.turn * p.stride + from;
      const float* s = p.sin + at.turn * p.stride + from;
      if (p.table_vec) {
        const float4 a = *reinterpret_cast<const float4*>(c), b = *reinterpret_cast<const float4*>(s);
        x.c[4 * g] = a.x, x.c[4 * g + 1] = a.y, x.c[4 * g + 2] = a.z, x.c[4 * g + 3] = a.w;
        x.s[4 * g] = b.x, x.s[4 * g + 1] = b.y, x.s[4 * g + 2] = b.z, x.s[4 * g + 3] = b.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x.c[4 * g + i] = c[i], x.s[4 * g + i] = s[i];
      }
    }
    return x;
  };

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // what is launched behind waits before it reads
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) ask();
  int stage = 0;
  for (int32_t first = begin, rows; first < end; first += rows) {
    rows = min(end - first, kThreads);
    __syncthreads();
    if (tid < rows) places[tid] = find_place(p, first + tid);
    __syncthreads();
    Angles next = angles(places[0]);
    for (int32_t r = 0; r < rows; ++r) {
      const Place at = places[r];
      const int32_t row = first + r;
      const Angles now = next;
      if (r + 1 < rows) next = angles(places[r + 1]);
      for (int32_t part = 0; part < parts; ++part) {
        uint4 w[kDepth][2];
        if (kVec) {
          ptx::cp_async_wait<kStages - 2>();
#pragma unroll
          for (int u = 0; u < kDepth; ++u)
#pragma unroll
            for (int g = 0; g < 2; ++g) w[u][g] = ring[(stage * kDepth * 2 + 2 * u + g) * kThreads + tid];
          stage = stage + 1 == kStages ? 0 : stage + 1;
          ask();  // into the stage before, whose values have been used
        }
#pragma unroll
        for (int u = 0; u < kDepth; ++u) {
          const int32_t base = part0 + (part * kDepth + u) * kStep;  // of the CTA's heads
          if (base >= head_end) break;
          const int32_t h = base + tid / kPer;
          const bool there = h < head_end, value = h >= kv && h < 2 * kv;
          float x[2][8];
          if (kVec) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const uint32_t word[4] = {w[u][g].x, w[u][g].y, w[u][g].z, w[u][g].w};
#pragma unroll
              for (int i = 0; i < 8; ++i) x[g][i] = widen<kBf16>(i & 1 ? word[i / 2] >> 16 : word[i / 2] & 0xFFFFu);
            }
          } else {
            const uint16_t* from = source(row, there ? h : part0);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[0][i] = widen<kBf16>(from[i]), x[1][i] = widen<kBf16>(from[e1 - e0 + i]);
          }
          if (!value && at.turn >= 0) {
            if (p.interleaved) {
#pragma unroll
              for (int g = 0; g < 2; ++g)
                if (g ? turned1 : turned0) {
#pragma unroll
                  for (int i = 0; i < 4; ++i) turn(x[g][2 * i], x[g][2 * i + 1], now.c[4 * g + i], now.s[4 * g + i]);
                }
            } else if (turned0) {
#pragma unroll
              for (int i = 0; i < 8; ++i) turn(x[0][i], x[1][i], now.c[i], now.s[i]);
            }
          }
          if (h >= 2 * kv && there && at.turn != kNoRow) {
            uint16_t* out = p.out + row * p.out_row + (h - 2 * kv) * p.out_head + e0;
            uint32_t y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float a = x[i / 4][2 * i % 8], b = x[i / 4][2 * i % 8 + 1];
              y[i] = kBf16 ? ptx::cvt_bf16x2(a, b) : cvt_f16x2(a, b);
            }
            if (at.turn < 0) {
#pragma unroll
              for (int i = 0; i < 8; ++i) y[i] = at.turn == kNoPlace ? 0u : 0x7FFF7FFFu;  // NaN in either type
            }
            if (kVec) {
              *reinterpret_cast<uint4*>(out) = make_uint4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<uint4*>(out + (e1 - e0)) = make_uint4(y[4], y[5], y[6], y[7]);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                uint16_t* to = out + (i < 4 ? 2 * i : e1 - e0 + 2 * i - 8);
                to[0] = static_cast<uint16_t>(y[i]);
                to[1] = static_cast<uint16_t>(y[i] >> 16);
              }
            }
          }
          if (base < 2 * kv) {  // keys and values among the CTA's heads: the same for all threads
            const bool mine = h < 2 * kv && there && at.page;
            const float* gs = value ? p.c.v_scale : p.c.k_scale;
            const int32_t hk = value ? h - kv : h;
            float top0 = 0.0f, top1 = 0.0f;
            if (mine) {
              top0 = scale8(x[0], gs ? gs + hk : nullptr);
              top1 = scale8(x[1], gs ? gs + hk : nullptr);
            }
            // each group is half of a scale's elements, the next thread's the other
            top0 = fmaxf(top0, __shfl_xor_sync(0xFFFFFFFFu, top0, 1));
            top1 = fmaxf(top1, __shfl_xor_sync(0xFFFFFFFFu, top1, 1));
            if (mine) {
              const uint32_t b0 = e4m3(fminf(__fdiv_rn(top0, 6.0f), 448.0f));
              const uint32_t b1 = e4m3(fminf(__fdiv_rn(top1, 6.0f), 448.0f));
              uint8_t* rec = at.page + static_cast<int64_t>(hk) * R::bytes(p.c.page_size);
              uint8_t* codes = rec + R::codes(p.c.page_size, value) + at.in_page * R::kCodeBytes;
              uint8_t* scales = rec + R::scales(p.c.page_size, value) + at.in_page * R::kScaleBytes;
              *reinterpret_cast<uint32_t*>(codes + e0 / 2) = encode8(x[0], b0);
              *reinterpret_cast<uint32_t*>(codes + e1 / 2) = encode8(x[1], b1);
              if (j % 2 == 0) {
                scales[e0 / 16] = static_cast<uint8_t>(b0);
                scales[e1 / 16] = static_cast<uint8_t>(b1);
              }
            }
          }
        }
      }
    }
  }
}

SmemAttr g_rotate_attr[2][2][2];

}  // namespace
}  // namespace kv4
}  // namespace dspark

extern "C" {

int dspark_kv4_append_rotated(const dspark_kv4_cache* cache, const dspark_kv4_batch* batch,
                              const dspark_kv4_rotation* rotation, const dspark_kv4_rotated_args* args,
                              cudaStream_t stream) {
  using namespace dspark::kv4;
  Rotate p{};
  int rc = make_cache(cache, &p.c);
  if (rc != DSPARK_OK) return rc;
  rc = make_batch(batch, p.c, &p.s);
  if (rc != DSPARK_OK) return rc;
  if (!rotation || !args) return DSPARK_ERR_INVALID_ARG;
  if (args->dtype != DSPARK_DTYPE_BF16 && args->dtype != DSPARK_DTYPE_F16) return DSPARK_ERR_INVALID_ARG;
  if (rotation->dims < 32 || rotation->dims % 32 != 0 || rotation->dims > cache->head_dim || rotation->positions < 0 ||
      rotation->stride < rotation->dims / 2)
    return DSPARK_ERR_INVALID_ARG;
  if (args->k_row < 0 || args->k_head < 0 || args->v_row < 0 || args->v_head < 0) return DSPARK_ERR_INVALID_ARG;
  if (!args->q != !args->q_out) return DSPARK_ERR_INVALID_ARG;
  if (args->q && (args->q_heads < 1 || args->q_heads > kMostHeads - 2 * p.c.kv_heads || args->q_row < 0 ||
                  args->q_head < 0 || args->out_row < 0 || args->out_head < 0))
    return DSPARK_ERR_INVALID_ARG;
  if (args->q == args->q_out && args->q && (args->q_row != args->out_row || args->q_head != args->out_head))
    return DSPARK_ERR_INVALID_ARG;
  if (!aligned(args->k, 2) || !aligned(args->v, 2) || !aligned(args->q, 2) || !aligned(args->q_out, 2) ||
      !aligned(rotation->cos, 4) || !aligned(rotation->sin, 4) || !aligned(rotation->at, 4))
    return DSPARK_ERR_MISALIGNED;
  if (p.s.batch == 0 || p.s.total_rows == 0) return DSPARK_OK;
  if (!args->k || !args->v || (rotation->positions > 0 && (!rotation->cos || !rotation->sin)))
    return DSPARK_ERR_INVALID_ARG;
  p.k = static_cast<const uint16_t*>(args->k), p.k_row = args->k_row, p.k_head = args->k_head;
  p.v = static_cast<const uint16_t*>(args->v), p.v_row = args->v_row, p.v_head = args->v_head;
  p.q = static_cast<const uint16_t*>(args->q), p.q_row = args->q_row, p.q_head = args->q_head;
  p.out = static_cast<uint16_t*>(args->q_out), p.out_row = args->out_row, p.out_head = args->out_head;
  p.cos = rotation->cos, p.sin = rotation->sin, p.stride = rotation->stride, p.at = rotation->at;
  p.positions = rotation->positions, p.dims = rotation->dims, p.interleaved = rotation->interleaved;
  p.table_vec = aligned(p.cos, 16) && aligned(p.sin, 16) && p.stride % 4 == 0;
  p.heads = 2 * p.c.kv_heads + (p.q ? args->q_heads : 0);
  const auto wide = [](const void* t, int64_t row, int64_t head) {
    return aligned(t, 16) && row % 8 == 0 && head % 8 == 0;
  };
  const bool vec = wide(p.k, p.k_row, p.k_head) && wide(p.v, p.v_row, p.v_head) && wide(p.q, p.q_row, p.q_head) &&
                   wide(p.out, p.out_row, p.out_head);
  // Few rows: a CTA each, or several with some of its heads; many: CTAs that stay,
  // with a run of rows each.
  const int step = kThreads / (cache->head_dim / 16);
  const int32_t groups = (p.heads + step - 1) / step, most_ctas = 152 * kCtas;
  int32_t parts = p.s.total_rows < most_ctas ? most_ctas / p.s.total_rows : 1;
  if (parts > groups) parts = groups;
  const int32_t most = (groups + 65534) / 65535;  // heads' groups of a CTA, so that the grid holds them
  int32_t per = (groups + parts - 1) / parts;
  if (per < most) per = most;
  p.part = per * step;
  parts = (groups + per - 1) / per;
  const dim3 grid(p.s.total_rows < most_ctas ? p.s.total_rows : most_ctas, parts);
  const bool bf16 = args->dtype == DSPARK_DTYPE_BF16;
  using Kernel = void (*)(Rotate);
  static const Kernel kernels[2][2][2] = {
      {{rotate_kernel<64, false, false>, rotate_kernel<64, false, true>},
       {rotate_kernel<64, true, false>, rotate_kernel<64, true, true>}},
      {{rotate_kernel<128, false, false>, rotate_kernel<128, false, true>},
       {rotate_kernel<128, true, false>, rotate_kernel<128, true, true>}}};
  const Kernel kernel = kernels[cache->head_dim == 128][bf16][vec];
  const int smem = vec ? kStages * kDepth * 2 * kThreads * 16 : 0;
  if (!smem_attr_ready(g_rotate_attr[cache->head_dim == 128][bf16][vec], kernel, smem)) return DSPARK_ERR_CUDA;
  kernel<<<grid, kThreads, smem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

}  // extern "C"
