// kv4_cache.cu -- storing rows in the paged 4-bit cache and reading them back
// (dspark_kv4_append, dspark_kv4_read of include/dspark_kv4.h).
//
// A value x is held as code * scale * g: for each 16 elements of a head
//   y = RN(x / g),  scale = E4M3(min(RN(max|y| / 6), 448)),  code = E2M1(RN(y / scale)).
// Both quotients are correctly rounded, so that ties (frequent: x has 8 bits,
// a scale 4) go the way the formula says.  One thread takes the 16 elements
// of a scale: two 16-byte loads, one 8-byte store of codes and one byte.
#include "kv4.cuh"
#include "markov_math.cuh"

namespace dspark {
namespace kv4 {

int make_cache(const dspark_kv4_cache* c, Cache* out) {
  if (!c) return DSPARK_ERR_INVALID_ARG;
  int shift = 0;
  while (shift < 9 && (1 << shift) != c->page_size) ++shift;
  if (shift < 4 || shift > 8) return DSPARK_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return DSPARK_ERR_INVALID_ARG;
  if (c->kv_heads < 1 || c->kv_heads > 65535 || c->num_pages < 0) return DSPARK_ERR_INVALID_ARG;
  const int64_t record = static_cast<int64_t>(c->page_size) * (c->head_dim + c->head_dim / 8);
  if (c->page_stride < record * c->kv_heads) return DSPARK_ERR_INVALID_ARG;
  if (c->num_pages > 0 && !c->data) return DSPARK_ERR_INVALID_ARG;
  if (!aligned(c->data, 16) || c->page_stride % 16 != 0) return DSPARK_ERR_MISALIGNED;
  if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)) return DSPARK_ERR_MISALIGNED;
  *out = Cache{static_cast<uint8_t*>(c->data), c->page_stride, c->num_pages, c->page_size, shift, c->kv_heads,
               c->k_scale, c->v_scale};
  return DSPARK_OK;
}

int make_batch(const dspark_kv4_batch* b, const Cache& c, Batch* out) {
  if (!b || b->batch < 0 || b->total_rows < 0 || b->max_rows < 0 || b->max_pages < 0 || b->max_slots < 0)
    return DSPARK_ERR_INVALID_ARG;
  if (b->batch > DSPARK_KV4_MAX_BATCH) return DSPARK_ERR_TOO_MANY_ROWS;
  if (b->table_stride < b->max_pages) return DSPARK_ERR_INVALID_ARG;
  if (b->batch > 0 && (!b->row_start || !b->lens || (!b->table && b->max_pages > 0))) return DSPARK_ERR_INVALID_ARG;
  if (!aligned(b->row_start, 4) || !aligned(b->slots, 4) || !aligned(b->lens, 4) || !aligned(b->table, 4))
    return DSPARK_ERR_MISALIGNED;
  *out = Batch{b->batch, b->total_rows, b->max_pages, b->max_slots,
               static_cast<int64_t>(b->max_pages) << c.page_shift, b->row_start, b->slots, b->lens, b->table,
               b->table_stride};
  return DSPARK_OK;
}

namespace {

constexpr int kThreads = 256;

struct RowTensor {
  uint8_t* p;
  int64_t row, head;  // strides in elements
};

// Where a row's codes and scales of head h go, or null: the row's position is
// negative or its page is not there.
template <int kDim>
__device__ __forceinline__ uint8_t* row_record(const Cache& c, const Batch& s, int32_t row, int32_t* in_page) {
  const int32_t i = find_request(s, row);
  if (i < 0) return nullptr;
  const Request r = load_request(s, i);
  const int32_t j = row - r.start;
  if (j < 0 || j >= r.rows) return nullptr;
  const int32_t pos = r.len - r.rows + j;
  if (pos < 0) return nullptr;
  const int32_t page = r.pages[pos >> c.page_shift];
  if (page < 0 || page >= c.num_pages) return nullptr;
  *in_page = pos & (c.page_size - 1);
  return c.data + static_cast<int64_t>(page) * c.page_stride;
}

// The E2M1 code of a quotient: nearest, ties to the even code, saturating.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t d;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
      "mov.b32 %0, {b, 0, 0, 0};\n\t}"
      : "=r"(d)
      : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ uint32_t e4m3(float x) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.0f), "f"(x));
  return d & 0xFFu;
}

template <bool kBf16>
__device__ __forceinline__ float widen(uint32_t bits) {
  return kBf16 ? __uint_as_float(bits << 16) : __half2float(__ushort_as_half(static_cast<uint16_t>(bits)));
}

template <int kDim, bool kBf16, bool kVec>
__global__ void __launch_bounds__(kThreads)
    append_kernel(Cache c, Batch s, RowTensor k, RowTensor v) {
  const int which = blockIdx.y;
  const RowTensor t = which ? v : k;
  constexpr int kBlocks = kDim / 16;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int32_t block = static_cast<int32_t>(item % kBlocks);
  const int64_t rh = item / kBlocks;
  const int32_t head = static_cast<int32_t>(rh % c.kv_heads);
  const int64_t row = rh / c.kv_heads;
  if (row >= s.total_rows) return;
  const uint16_t* src = reinterpret_cast<const uint16_t*>(t.p) + row * t.row + head * t.head + block * 16;
  uint32_t x[8];  // 16 values
  if (kVec) {
    const uint4 a = reinterpret_cast<const uint4*>(src)[0], b = reinterpret_cast<const uint4*>(src)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = src[2 * i] | (static_cast<uint32_t>(src[2 * i + 1]) << 16);
  }
  int32_t in_page = 0;
  uint8_t* page = row_record<kDim>(c, s, static_cast<int32_t>(row), &in_page);
  if (!page) return;
  const float* gs = which ? c.v_scale : c.k_scale;
  const Divider by_g = make_divider(gs ? gs[head] : 1.0f);
  float y[16];
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float w = widen<kBf16>(i & 1 ? x[i / 2] >> 16 : x[i / 2] & 0xFFFFu);
    if (gs) w = div_rn(w, by_g);
    if (isnan(w)) w = 0.0f;
    y[i] = w;
    top = fmaxf(top, fabsf(w));
  }
  const uint32_t sbyte = e4m3(fminf(__fdiv_rn(top, 6.0f), 448.0f));
  const float scale = __half2float(__ushort_as_half(static_cast<uint16_t>(scales_to_f16(sbyte))));
  uint32_t w[2] = {0u, 0u};
  if (scale != 0.0f) {
    const Divider by_s = make_divider(scale);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      w[i / 8] |= e2m1x2(div_rn(y[i], by_s), div_rn(y[i + 1], by_s)) << (4 * (i % 8));
    }
  }
  using R = Record<kDim>;
  uint8_t* rec = page + static_cast<int64_t>(head) * R::bytes(c.page_size);
  *reinterpret_cast<uint2*>(rec + R::codes(c.page_size, which) + in_page * R::kCodeBytes + block * 8) =
      make_uint2(w[0], w[1]);
  rec[R::scales(c.page_size, which) + in_page * R::kScaleBytes + block] = static_cast<uint8_t>(sbyte);
}

// One thread reads the 16 elements of a scale.
template <int kDim, int kDtype, bool kVec>
__global__ void __launch_bounds__(kThreads)
    read_kernel(Cache c, Batch s, RowTensor k, RowTensor v) {
  const int which = blockIdx.y;
  const RowTensor t = which ? v : k;
  if (!t.p) return;
  constexpr int kBlocks = kDim / 16;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int32_t block = static_cast<int32_t>(item % kBlocks);
  const int64_t rh = item / kBlocks;
  const int32_t head = static_cast<int32_t>(rh % c.kv_heads);
  const int64_t row = rh / c.kv_heads;
  if (row >= s.total_rows) return;
  if (row < s.row_start[0] || row >= s.row_start[s.batch]) return;  // no request's row
  int32_t in_page = 0;
  const uint8_t* page = row_record<kDim>(c, s, static_cast<int32_t>(row), &in_page);
  using R = Record<kDim>;
  uint2 code = make_uint2(0u, 0u);
  uint32_t sbyte = 0;
  if (page) {
    const uint8_t* rec = page + static_cast<int64_t>(head) * R::bytes(c.page_size);
    code = *reinterpret_cast<const uint2*>(rec + R::codes(c.page_size, which) + in_page * R::kCodeBytes + block * 8);
    sbyte = rec[R::scales(c.page_size, which) + in_page * R::kScaleBytes + block];
  }
  const float* gs = which ? c.v_scale : c.k_scale;
  const float g = gs ? gs[head] : 1.0f;
  const uint32_t s2 = scales_to_f16(sbyte | (sbyte << 8));
  uint32_t h[8];
  {
    uint32_t a[4], b[4];
    e2m1x8_to_f16(code.x, a);
    e2m1x8_to_f16(code.y, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = mul_f16x2(a[i], s2), h[4 + i] = mul_f16x2(b[i], s2);
  }
  float y[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    y[2 * i] = __fmul_rn(f.x, g);
    y[2 * i + 1] = __fmul_rn(f.y, g);
  }
  const int64_t at = row * t.row + head * t.head + block * 16;
  if (kDtype == DSPARK_DTYPE_F32) {
    float* out = reinterpret_cast<float*>(t.p) + at;
    if (kVec) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4*>(out)[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) out[i] = y[i];
    }
  } else {
    uint16_t* out = reinterpret_cast<uint16_t*>(t.p) + at;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (kDtype == DSPARK_DTYPE_BF16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      } else {
        w[i] = cvt_f16x2(y[2 * i], y[2 * i + 1]);
      }
    }
    if (kVec) {
      reinterpret_cast<uint4*>(out)[0] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint4*>(out)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        out[2 * i] = static_cast<uint16_t>(w[i]);
        out[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
      }
    }
  }
}

// Arguments common to append and read, and their grid.
int check_rows(const dspark_kv4_cache* cache, const dspark_kv4_batch* batch, const void* k, int64_t k_row,
               int64_t k_head, const void* v, int64_t v_row, int64_t v_head, int elem, Cache* c, Batch* s,
               unsigned* blocks, bool* vec) {
  int rc = make_cache(cache, c);
  if (rc != DSPARK_OK) return rc;
  rc = make_batch(batch, *c, s);
  if (rc != DSPARK_OK) return rc;
  if (k_row < 0 || k_head < 0 || v_row < 0 || v_head < 0) return DSPARK_ERR_INVALID_ARG;
  if (!aligned(k, elem) || !aligned(v, elem)) return DSPARK_ERR_MISALIGNED;
  const int64_t items = static_cast<int64_t>(s->total_rows) * c->kv_heads * (cache->head_dim / 16);
  const int64_t n = (items + kThreads - 1) / kThreads;
  if (n > 0x7FFFFFFF) return DSPARK_ERR_INVALID_ARG;
  *blocks = static_cast<unsigned>(n);
  const int64_t per16 = 16 / elem;
  *vec = aligned(k, 16) && aligned(v, 16) && k_row % per16 == 0 && k_head % per16 == 0 && v_row % per16 == 0 &&
         v_head % per16 == 0;
  return DSPARK_OK;
}

}  // namespace
}  // namespace kv4
}  // namespace dspark

extern "C" {

int dspark_kv4_append(const dspark_kv4_cache* cache, const dspark_kv4_batch* batch, const void* k, int64_t k_row,
                      int64_t k_head, const void* v, int64_t v_row, int64_t v_head, int32_t dtype,
                      cudaStream_t stream) {
  using namespace dspark::kv4;
  if (dtype != DSPARK_DTYPE_BF16 && dtype != DSPARK_DTYPE_F16) return DSPARK_ERR_INVALID_ARG;
  Cache c;
  Batch s;
  unsigned blocks = 0;
  bool vec = false;
  const int rc = check_rows(cache, batch, k, k_row, k_head, v, v_row, v_head, 2, &c, &s, &blocks, &vec);
  if (rc != DSPARK_OK) return rc;
  if (s.batch == 0 || blocks == 0 || c.num_pages == 0) return DSPARK_OK;
  if (!k || !v) return DSPARK_ERR_INVALID_ARG;
  const RowTensor kt{static_cast<uint8_t*>(const_cast<void*>(k)), k_row, k_head};
  const RowTensor vt{static_cast<uint8_t*>(const_cast<void*>(v)), v_row, v_head};
  const dim3 grid(blocks, 2);
  const bool bf16 = dtype == DSPARK_DTYPE_BF16;
  const auto kernel = cache->head_dim == 128
                          ? (bf16 ? (vec ? append_kernel<128, true, true> : append_kernel<128, true, false>)
                                  : (vec ? append_kernel<128, false, true> : append_kernel<128, false, false>))
                          : (bf16 ? (vec ? append_kernel<64, true, true> : append_kernel<64, true, false>)
                                  : (vec ? append_kernel<64, false, true> : append_kernel<64, false, false>));
  kernel<<<grid, kThreads, 0, stream>>>(c, s, kt, vt);
  return cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

int dspark_kv4_read(const dspark_kv4_cache* cache, const dspark_kv4_batch* batch, void* k, int64_t k_row,
                    int64_t k_head, void* v, int64_t v_row, int64_t v_head, int32_t dtype, cudaStream_t stream) {
  using namespace dspark::kv4;
  if (dtype < DSPARK_DTYPE_BF16 || dtype > DSPARK_DTYPE_F32) return DSPARK_ERR_INVALID_ARG;
  Cache c;
  Batch s;
  unsigned blocks = 0;
  bool vec = false;
  const int rc = check_rows(cache, batch, k, k_row, k_head, v, v_row, v_head, dtype == DSPARK_DTYPE_F32 ? 4 : 2, &c,
                            &s, &blocks, &vec);
  if (rc != DSPARK_OK) return rc;
  if (s.batch == 0 || blocks == 0 || (!k && !v)) return DSPARK_OK;
  const RowTensor kt{static_cast<uint8_t*>(k), k_row, k_head};
  const RowTensor vt{static_cast<uint8_t*>(v), v_row, v_head};
  const dim3 grid(blocks, 2);
  using Kernel = void (*)(Cache, Batch, RowTensor, RowTensor);
  static const Kernel kernels[2][3][2] = {
      {{read_kernel<64, 0, false>, read_kernel<64, 0, true>},
       {read_kernel<64, 1, false>, read_kernel<64, 1, true>},
       {read_kernel<64, 2, false>, read_kernel<64, 2, true>}},
      {{read_kernel<128, 0, false>, read_kernel<128, 0, true>},
       {read_kernel<128, 1, false>, read_kernel<128, 1, true>},
       {read_kernel<128, 2, false>, read_kernel<128, 2, true>}}};
  kernels[cache->head_dim == 128][dtype][vec]<<<grid, kThreads, 0, stream>>>(c, s, kt, vt);
  return cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

}  // extern "C"
