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
// cosines and sines once a row.  Its 16 elements are two groups of 8: neighbouring
// ones where the pairs are neighbours or nothing is turned, else 8 and the 8 that
// are half of the turned dimensions behind them, so that both of a pair are in one
// thread.  The scale of 16 elements then needs the maxima of two threads beside
// one another (one shuffle), each of which writes 4 bytes of codes.
#include "kv4_quant.cuh"

namespace dspark {
namespace kv4 {
namespace {

constexpr int kThreads = 128;
constexpr int kMostRows = 4;  // rows of a CTA
constexpr int kDepth = 5;     // heads a thread has in flight

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
  int32_t rows;       // of a CTA
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
// within one unit of its last place, which the product with RN(1 / d) alone gives
// for short x only; one more step makes it so.  The same range.
__device__ __forceinline__ float quotient24(float x, float d, float inverse) {
  const float q = quotient(x, d, inverse);
  return __fmaf_rn(__fmaf_rn(-q, d, x), inverse, q);
}

// x / g in place (NaN as 0, what saturates every code held to 2^40); the largest.
__device__ __noinline__ float scale8_any(float (&x)[8], float g) {
  float top = 0.0f;
  for (int i = 0; i < 8; ++i) {
    const float v = __fdiv_rn(x[i], g);
    x[i] = isnan(v) ? 0.0f : fminf(fmaxf(v, -0x1p40f), 0x1p40f);
    top = fmaxf(top, fabsf(x[i]));
  }
  return top;
}
__device__ __forceinline__ float scale8(float (&x)[8], const float* scale_of_head) {
  const float g = scale_of_head ? *scale_of_head : 1.0f, size = fabsf(g);
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(x[i]));
  if (!(top < 0x1p40f && size >= 0x1p-20f && size < 0x1p40f)) return scale8_any(x, g);
  if (!scale_of_head) return top;
  const float inverse = __frcp_rn(g);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = quotient24(x[i], g, inverse);
  return fabsf(quotient24(top, g, inverse));  // rounding keeps the order: the largest stays the largest
}

// The codes of 8 quotients, of the scale `byte`.
__device__ __forceinline__ uint32_t encode8(const float (&y)[8], uint32_t byte) {
  const float scale = __half2float(__ushort_as_half(static_cast<uint16_t>(scales_to_f16(byte))));
  if (scale == 0.0f) return 0u;
  const float inverse = __frcp_rn(scale);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    w |= e2m1x2(quotient24(y[i], scale, inverse), quotient24(y[i + 1], scale, inverse)) << (4 * i);
  return w;
}

template <int kDim, bool kBf16, bool kVec>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const __grid_constant__ Rotate p) {
  using R = Record<kDim>;
  constexpr int kPer = kDim / 16;           // threads of a head
  constexpr int kStep = kThreads / kPer;    // heads of a CTA at a time
  __shared__ Place places[kMostRows];
  const int32_t first = blockIdx.x * p.rows;
  const int32_t rows = min(p.rows, p.s.total_rows - first);
  const int tid = threadIdx.x, j = tid % kPer;
  const int32_t head0 = blockIdx.y * p.part + tid / kPer, head_end = min(p.heads, (static_cast<int32_t>(blockIdx.y) + 1) * p.part);
  const int32_t kv = p.c.kv_heads;
  const bool turned = 16 * j < p.dims;
  const bool apart = turned && !p.interleaved;  // the groups are half of the turned dimensions apart
  const int e0 = apart ? 8 * j : 16 * j, e1 = apart ? p.dims / 2 + 8 * j : 16 * j + 8;

  uint32_t w[kDepth][8];
  const auto load = [&](int32_t row, int32_t base) {
#pragma unroll
    for (int u = 0; u < kDepth; ++u) {
      const int32_t h = base + u * kStep;
      if (h >= head_end) continue;
      const uint16_t* src = h < kv       ? p.k + row * p.k_row + h * p.k_head
                            : h < 2 * kv ? p.v + row * p.v_row + (h - kv) * p.v_head
                                         : p.q + row * p.q_row + (h - 2 * kv) * p.q_head;
      if (h >= kv && h < 2 * kv) src += 16 * j;
      const int d1 = h >= kv && h < 2 * kv ? 8 : e1 - e0;
      if (h < kv || h >= 2 * kv) src += e0;
      if (kVec) {
        const uint4 a = __ldcs(reinterpret_cast<const uint4*>(src));
        const uint4 b = __ldcs(reinterpret_cast<const uint4*>(src + d1));
        w[u][0] = a.x, w[u][1] = a.y, w[u][2] = a.z, w[u][3] = a.w;
        w[u][4] = b.x, w[u][5] = b.y, w[u][6] = b.z, w[u][7] = b.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[u][i] = src[2 * i] | (static_cast<uint32_t>(src[2 * i + 1]) << 16);
          w[u][4 + i] = src[d1 + 2 * i] | (static_cast<uint32_t>(src[d1 + 2 * i + 1]) << 16);
        }
      }
    }
  };

  load(first, head0);
  if (tid < rows) places[tid] = find_place(p, first + tid);
  __syncthreads();
  for (int32_t r = 0; r < rows; ++r) {
    const Place at = places[r];
    const int32_t row = first + r;
    float cs[8], sn[8];
    if (turned && at.turn >= 0) {
      const float* c = p.cos + at.turn * p.stride + 8 * j;
      const float* s = p.sin + at.turn * p.stride + 8 * j;
      if (p.table_vec) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 a = reinterpret_cast<const float4*>(c)[i], b = reinterpret_cast<const float4*>(s)[i];
          cs[4 * i] = a.x, cs[4 * i + 1] = a.y, cs[4 * i + 2] = a.z, cs[4 * i + 3] = a.w;
          sn[4 * i] = b.x, sn[4 * i + 1] = b.y, sn[4 * i + 2] = b.z, sn[4 * i + 3] = b.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = c[i], sn[i] = s[i];
      }
    }
    // whole warps stay together for the shuffle
    for (int32_t base = head0, lead = head0 - tid / kPer; lead < head_end; base += kDepth * kStep, lead += kDepth * kStep) {
      if (r > 0 || base != head0) load(row, base);
#pragma unroll
      for (int u = 0; u < kDepth; ++u) {
        const int32_t h = base + u * kStep;
        const bool value = h >= kv && h < 2 * kv;
        float x[2][8];
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            x[g][i] = widen<kBf16>(i & 1 ? w[u][4 * g + i / 2] >> 16 : w[u][4 * g + i / 2] & 0xFFFFu);
        if (turned && !value && at.turn >= 0) {
          if (p.interleaved) {
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float a = x[g][2 * i], b = x[g][2 * i + 1], c = cs[4 * g + i], s = sn[4 * g + i];
                x[g][2 * i] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
                x[g][2 * i + 1] = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
              }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float a = x[0][i], b = x[1][i];
              x[0][i] = __fsub_rn(__fmul_rn(a, cs[i]), __fmul_rn(b, sn[i]));
              x[1][i] = __fadd_rn(__fmul_rn(b, cs[i]), __fmul_rn(a, sn[i]));
            }
          }
        }
        if (h >= 2 * kv && h < head_end && at.turn != kNoRow) {
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
        // keys and values: the same for the whole warp whether any lane has one
        if (__any_sync(0xFFFFFFFFu, h < 2 * kv && h < head_end)) {
          const bool mine = h < 2 * kv && h < head_end && at.page;
          const bool split = apart && !value;  // the groups belong to two scales, each shared with the next thread
          const float* gs = value ? p.c.v_scale : p.c.k_scale;
          const int32_t hk = value ? h - kv : h;
          float top[2] = {0.0f, 0.0f};
          if (mine) {
            top[0] = scale8(x[0], gs ? gs + hk : nullptr);
            top[1] = scale8(x[1], gs ? gs + hk : nullptr);
          }
          const float next0 = __shfl_xor_sync(0xFFFFFFFFu, top[0], 1), next1 = __shfl_xor_sync(0xFFFFFFFFu, top[1], 1);
          if (mine) {
            const float t0 = fmaxf(top[0], split ? next0 : top[1]), t1 = split ? fmaxf(top[1], next1) : t0;
            const uint32_t b0 = e4m3(fminf(__fdiv_rn(t0, 6.0f), 448.0f));
            const uint32_t b1 = split ? e4m3(fminf(__fdiv_rn(t1, 6.0f), 448.0f)) : b0;
            const uint32_t w0 = encode8(x[0], b0), w1 = encode8(x[1], b1);
            uint8_t* rec = at.page + static_cast<int64_t>(hk) * R::bytes(p.c.page_size);
            uint8_t* codes = rec + R::codes(p.c.page_size, value) + at.in_page * R::kCodeBytes;
            uint8_t* scales = rec + R::scales(p.c.page_size, value) + at.in_page * R::kScaleBytes;
            const int c0 = value ? 16 * j : e0, c1 = value ? 16 * j + 8 : e1;
            if (split) {
              *reinterpret_cast<uint32_t*>(codes + c0 / 2) = w0;
              *reinterpret_cast<uint32_t*>(codes + c1 / 2) = w1;
              if (j % 2 == 0) {
                scales[c0 / 16] = static_cast<uint8_t>(b0);
                scales[c1 / 16] = static_cast<uint8_t>(b1);
              }
            } else {
              *reinterpret_cast<uint2*>(codes + c0 / 2) = make_uint2(w0, w1);
              scales[c0 / 16] = static_cast<uint8_t>(b0);
            }
          }
        }
      }
    }
  }
}

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
  if (args->q && (args->q_heads < 1 || args->q_heads > 0x7FFFFFFF - 2 * p.c.kv_heads || args->q_row < 0 ||
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
  // Few rows: a CTA each, or several with some of its heads; many: 4 rows a CTA,
  // which look their pages up together.
  const int step = kThreads / (cache->head_dim / 16);
  const int32_t groups = (p.heads + step - 1) / step;
  int32_t rows = p.s.total_rows / (152 * 8);
  p.rows = rows < 1 ? 1 : rows > kMostRows ? kMostRows : rows;
  int32_t parts = p.s.total_rows < 152 * 2 ? (152 * 2 + p.s.total_rows - 1) / p.s.total_rows : 1;
  if (parts > groups) parts = groups;
  const int32_t most = (groups + 65534) / 65535;  // heads' groups of a CTA, so that the grid holds them
  int32_t per = (groups + parts - 1) / parts;
  if (per < most) per = most;
  p.part = per * step;
  parts = (groups + per - 1) / per;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(p.s.total_rows) + p.rows - 1) / p.rows), parts);
  const bool bf16 = args->dtype == DSPARK_DTYPE_BF16;
  using Kernel = void (*)(Rotate);
  static const Kernel kernels[2][2][2] = {
      {{rotate_kernel<64, false, false>, rotate_kernel<64, false, true>},
       {rotate_kernel<64, true, false>, rotate_kernel<64, true, true>}},
      {{rotate_kernel<128, false, false>, rotate_kernel<128, false, true>},
       {rotate_kernel<128, true, false>, rotate_kernel<128, true, true>}}};
  kernels[cache->head_dim == 128][bf16][vec]<<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

}  // extern "C"
