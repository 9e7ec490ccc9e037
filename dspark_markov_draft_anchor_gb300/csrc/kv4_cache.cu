// kv4_cache.cu -- storing rows in the paged 4-bit cache and reading them back
// (dspark_kv4_append, dspark_kv4_read of include/dspark_kv4.h).
//
// A value x is held as code * scale * g: for each 16 elements of a head
//   y = RN(x / g),  scale = E4M3(min(RN(max|y| / 6), 448)),  code = E2M1(RN(y / scale)).
// Both quotients are correctly rounded, so that ties (frequent: x has 8 bits,
// a scale 4) go the way the formula says.  Bound by the memory's 2.56 bytes an
// element, if the arithmetic stays below about a dozen operations.  A CTA takes
// up to four rows: one of its warps finds their requests and pages, a row a lane,
// while the first loads of all are on their way; a thread takes the 16 elements
// of a scale (two 16-byte loads, one 8-byte store of codes and one byte), two of
// them at a time; and a quotient costs one product and two fused multiply-adds.
// Measured: 18 k rows of 8 heads of 128 dimensions stored and read back, 37 M
// elements, 189 MB, 53 us, 3.6 TB/s (append 31.6, read 23.3 in a profile, for 14.2
// each at a copy's rate); 16 verifications of 6 rows 12 us, the latency of two
// launches.  Neither issue (70 % active in append, 59 % in read) nor the memory is
// spent: each CTA's chain of dependent loads (request, slot, length, page) and
// the barrier behind it overlap with nothing of the rows before.
#include "kv4.cuh"

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
  const int64_t tokens = static_cast<int64_t>(b->max_pages) << c.page_shift;
  *out = Batch{b->batch, b->total_rows, b->max_pages, b->max_slots,
               tokens < kMostTokens ? static_cast<int32_t>(tokens) : kMostTokens, b->row_start, b->slots, b->lens,
               b->table, b->table_stride};
  return DSPARK_OK;
}

namespace {

constexpr int kThreads = 128;
constexpr int kMostRows = 4;    // rows of a CTA
constexpr int kDepth = 2;      // scales a thread has in flight

struct RowTensor {
  uint8_t* p;
  int64_t row, head;  // strides in elements
};

// How a call's work is cut: rows of a CTA, and 2^32 / (scales of a row) rounded
// up (the quotient of a number below 2^16 is then the product's high word).
struct Split {
  int32_t rows;
  uint32_t magic;
};

// A CTA's rows: where each one's page is (null: the row has no place), the row
// in it, and whether a request has the row.
struct Places {
  uint8_t* page[kMostRows];
  int32_t in_page[kMostRows];
  bool some[kMostRows];
};

// By one warp, a row a lane.
__device__ __forceinline__ void find_places(const Cache& c, const Batch& s, int64_t first, int32_t rows, Places& out) {
  const int lane = threadIdx.x & 31;
  if (lane >= rows) return;
  const int32_t row = static_cast<int32_t>(first) + lane;
  uint8_t* page = nullptr;
  int32_t in_page = 0;
  const int32_t i = find_request(s, row);
  if (i >= 0) {
    const Request r = load_request(s, i);
    const int32_t j = row - r.start;
    const int32_t pos = r.len - r.rows + j;
    if (j >= 0 && j < r.rows && pos >= 0) {
      const int32_t id = r.pages[pos >> c.page_shift];
      if (id >= 0 && id < c.num_pages) page = c.data + static_cast<int64_t>(id) * c.page_stride;
      in_page = pos & (c.page_size - 1);
    }
  }
  out.page[lane] = page;
  out.in_page[lane] = in_page;
  out.some[lane] = i >= 0;
}

// Item `n` of a CTA: its row, and which 16 elements of it.
template <int kDim>
struct Item {
  int32_t row, which, head, block;
  __device__ __forceinline__ Item(int32_t n, int32_t per_row, const Split& split) {
    row = split.rows == 1 ? 0 : static_cast<int32_t>(__umulhi(static_cast<uint32_t>(n), split.magic));
    const int32_t in_row = n - row * per_row;
    which = in_row >= per_row / 2;
    const int32_t at = which ? in_row - per_row / 2 : in_row;
    head = at / (kDim / 16);
    block = at % (kDim / 16);
  }
};

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

// The larger, or NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

template <bool kBf16>
__device__ __forceinline__ float widen(uint32_t bits) {
  return kBf16 ? __uint_as_float(bits << 16) : __half2float(__ushort_as_half(static_cast<uint16_t>(bits)));
}

// RN(x / d) by a product with RN(1 / d) and its exact remainder (P. Markstein, IBM
// J. Res. Dev. 34(1), 1990), for d between 2^-20 and 2^40 and |x| below 2^60.
// Quotients below 2^-60 may be off; they are nothing to a code or a scale.
__device__ __forceinline__ float quotient(float x, float d, float inverse) {
  const float q = __fmul_rn(x, inverse);
  return __fmaf_rn(__fmaf_rn(-q, d, x), inverse, q);
}

struct Coded {
  uint32_t w[2];  // the codes of 16 elements
  uint32_t byte;  // their scale
};

// Of 16 quotients by their scale's byte.
__device__ __forceinline__ Coded encode16(const float (&y)[16], uint32_t byte) {
  Coded c{{0u, 0u}, byte};
  const float scale = __half2float(__ushort_as_half(static_cast<uint16_t>(scales_to_f16(byte))));
  if (scale == 0.0f) return c;
  const float inverse = __frcp_rn(scale);
#pragma unroll
  for (int i = 0; i < 16; i += 2)
    c.w[i / 8] |= e2m1x2(quotient(y[i], scale, inverse), quotient(y[i + 1], scale, inverse)) << (4 * (i % 8));
  return c;
}

// Infinities, NaN and the largest values, or a head scale outside of
// quotient()'s range: NaN is 0, and what saturates every code is held to 2^40.
template <bool kBf16>
__device__ __noinline__ Coded quantise16_any(uint4 a, uint4 b, float g) {
  const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float y[16], top = 0.0f;
  for (int i = 0; i < 16; ++i) {
    const float v = __fdiv_rn(widen<kBf16>(i & 1 ? x[i / 2] >> 16 : x[i / 2] & 0xFFFFu), g);
    y[i] = isnan(v) ? 0.0f : fminf(fmaxf(v, -0x1p40f), 0x1p40f);
    top = fmaxf(top, fabsf(y[i]));
  }
  return encode16(y, e4m3(fminf(__fdiv_rn(top, 6.0f), 448.0f)));
}

template <bool kBf16>
__device__ __forceinline__ Coded quantise16(const uint32_t (&x)[8], const float* scale_of_head) {
  const float g = scale_of_head ? *scale_of_head : 1.0f;
  float y[16], top = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    y[i] = widen<kBf16>(i & 1 ? x[i / 2] >> 16 : x[i / 2] & 0xFFFFu);
    top = max_nan(top, fabsf(y[i]));
  }
  const float size = fabsf(g);
  if (!(top < 0x1p40f && size >= 0x1p-20f && size < 0x1p40f))
    return quantise16_any<kBf16>(make_uint4(x[0], x[1], x[2], x[3]), make_uint4(x[4], x[5], x[6], x[7]), g);
  if (scale_of_head) {
    const float inverse = __frcp_rn(g);
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = quotient(y[i], g, inverse);
    top = fabsf(quotient(top, g, inverse));  // rounding keeps the order: the largest stays the largest
  }
  return encode16(y, e4m3(fminf(__fdiv_rn(top, 6.0f), 448.0f)));
}

template <int kDim, bool kBf16, bool kVec>
__global__ void __launch_bounds__(kThreads)
    append_kernel(Cache c, Batch s, RowTensor k, RowTensor v, Split split) {
  using R = Record<kDim>;
  __shared__ Places places;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * split.rows;
  const int32_t rows = static_cast<int32_t>(first + split.rows < s.total_rows ? split.rows : s.total_rows - first);
  const int32_t per_row = 2 * c.kv_heads * (kDim / 16), items = rows * per_row;
  uint32_t x[kDepth][8];
  const auto load = [&](int32_t base) {
#pragma unroll
    for (int u = 0; u < kDepth; ++u) {
      const int32_t n = base + u * kThreads;
      if (n >= items) continue;
      const Item<kDim> it(n, per_row, split);
      const RowTensor& t = it.which ? v : k;
      const uint16_t* src =
          reinterpret_cast<const uint16_t*>(t.p) + (first + it.row) * t.row + it.head * t.head + it.block * 16;
      if (kVec) {
        const uint4 a = __ldcs(reinterpret_cast<const uint4*>(src));
        const uint4 b = __ldcs(reinterpret_cast<const uint4*>(src) + 1);
        x[u][0] = a.x, x[u][1] = a.y, x[u][2] = a.z, x[u][3] = a.w;
        x[u][4] = b.x, x[u][5] = b.y, x[u][6] = b.z, x[u][7] = b.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[u][i] = src[2 * i] | (static_cast<uint32_t>(src[2 * i + 1]) << 16);
      }
    }
  };
  load(threadIdx.x);
  if (threadIdx.x < 32) find_places(c, s, first, rows, places);
  __syncthreads();
  for (int32_t base = threadIdx.x; base < items; base += kDepth * kThreads) {
    if (base >= kThreads) load(base);
#pragma unroll
    for (int u = 0; u < kDepth; ++u) {
      const int32_t n = base + u * kThreads;
      if (n >= items) continue;
      const Item<kDim> it(n, per_row, split);
      uint8_t* page = places.page[it.row];
      if (!page) continue;
      const float* gs = it.which ? c.v_scale : c.k_scale;
      const Coded coded = quantise16<kBf16>(x[u], gs ? gs + it.head : nullptr);
      uint8_t* rec = page + static_cast<int64_t>(it.head) * R::bytes(c.page_size);
      const int32_t in_page = places.in_page[it.row];
      *reinterpret_cast<uint2*>(rec + R::codes(c.page_size, it.which) + in_page * R::kCodeBytes + it.block * 8) =
          make_uint2(coded.w[0], coded.w[1]);
      rec[R::scales(c.page_size, it.which) + in_page * R::kScaleBytes + it.block] = static_cast<uint8_t>(coded.byte);
    }
  }
}

template <int kDim, int kDtype, bool kVec>
__global__ void __launch_bounds__(kThreads)
    read_kernel(Cache c, Batch s, RowTensor k, RowTensor v, Split split) {
  using R = Record<kDim>;
  __shared__ Places places;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * split.rows;
  const int32_t rows = static_cast<int32_t>(first + split.rows < s.total_rows ? split.rows : s.total_rows - first);
  const int32_t per_row = 2 * c.kv_heads * (kDim / 16), items = rows * per_row;
  if (threadIdx.x < 32) find_places(c, s, first, rows, places);
  __syncthreads();
  for (int32_t base = threadIdx.x; base < items; base += kDepth * kThreads) {
    uint2 code[kDepth];
    uint32_t byte[kDepth];
#pragma unroll
    for (int u = 0; u < kDepth; ++u) {
      const int32_t n = base + u * kThreads;
      code[u] = make_uint2(0u, 0u);
      byte[u] = 0;
      if (n >= items) continue;
      const Item<kDim> it(n, per_row, split);
      const uint8_t* page = places.page[it.row];
      if (!page || !(it.which ? v.p : k.p)) continue;
      const uint8_t* rec = page + static_cast<int64_t>(it.head) * R::bytes(c.page_size);
      const int32_t in_page = places.in_page[it.row];
      code[u] = *reinterpret_cast<const uint2*>(rec + R::codes(c.page_size, it.which) + in_page * R::kCodeBytes +
                                                it.block * 8);
      byte[u] = rec[R::scales(c.page_size, it.which) + in_page * R::kScaleBytes + it.block];
    }
#pragma unroll
    for (int u = 0; u < kDepth; ++u) {
      const int32_t n = base + u * kThreads;
      if (n >= items) continue;
      const Item<kDim> it(n, per_row, split);
      const RowTensor& t = it.which ? v : k;
      if (!t.p || !places.some[it.row]) continue;
      const float* gs = it.which ? c.v_scale : c.k_scale;
      const float g = gs ? gs[it.head] : 1.0f;
      const uint32_t s2 = scales_to_f16(byte[u] * 0x0101u);
      uint32_t a[4], b[4];
      e2m1x8_to_f16(code[u].x, a);
      e2m1x8_to_f16(code[u].y, b);
      float y[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t h = mul_f16x2(i < 4 ? a[i & 3] : b[i & 3], s2);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        y[2 * i] = __fmul_rn(f.x, g);
        y[2 * i + 1] = __fmul_rn(f.y, g);
      }
      const int64_t at = (first + it.row) * t.row + it.head * t.head + it.block * 16;
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
        for (int i = 0; i < 8; ++i)
          w[i] = kDtype == DSPARK_DTYPE_BF16 ? ptx::cvt_bf16x2(y[2 * i], y[2 * i + 1])
                                             : cvt_f16x2(y[2 * i], y[2 * i + 1]);
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
  }
}

// Arguments common to append and read, and their grid.
int check_rows(const dspark_kv4_cache* cache, const dspark_kv4_batch* batch, const void* k, int64_t k_row,
               int64_t k_head, const void* v, int64_t v_row, int64_t v_head, int elem, Cache* c, Batch* s,
               unsigned* blocks, Split* split, bool* vec) {
  int rc = make_cache(cache, c);
  if (rc != DSPARK_OK) return rc;
  rc = make_batch(batch, *c, s);
  if (rc != DSPARK_OK) return rc;
  if (k_row < 0 || k_head < 0 || v_row < 0 || v_head < 0) return DSPARK_ERR_INVALID_ARG;
  if (!aligned(k, elem) || !aligned(v, elem)) return DSPARK_ERR_MISALIGNED;
  // Few rows: a CTA each, so that all SMs work; many: 4 rows a CTA, which share
  // the search for their pages (18 k rows of 8 heads, append: 1 row a CTA 48 us,
  // 4 rows 44, 8 rows 46, 16 rows 50, 32 rows 62, before the quotients were cut).
  const int64_t per_row = static_cast<int64_t>(c->kv_heads) * (cache->head_dim / 8);
  int64_t rows = s->total_rows / (152 * 4);
  if (rows > kMostRows) rows = kMostRows;
  if (rows * per_row > 65535) rows = 65535 / per_row;
  if (rows < 1) rows = 1;
  split->rows = static_cast<int32_t>(rows);
  split->magic = static_cast<uint32_t>((int64_t{1} << 32) / per_row + 1);
  *blocks = static_cast<unsigned>((s->total_rows + rows - 1) / rows);
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
  Split split{};
  bool vec = false;
  const int rc = check_rows(cache, batch, k, k_row, k_head, v, v_row, v_head, 2, &c, &s, &blocks, &split, &vec);
  if (rc != DSPARK_OK) return rc;
  if (s.batch == 0 || blocks == 0 || c.num_pages == 0) return DSPARK_OK;
  if (!k || !v) return DSPARK_ERR_INVALID_ARG;
  const RowTensor kt{static_cast<uint8_t*>(const_cast<void*>(k)), k_row, k_head};
  const RowTensor vt{static_cast<uint8_t*>(const_cast<void*>(v)), v_row, v_head};
  const dim3 grid(blocks);
  const bool bf16 = dtype == DSPARK_DTYPE_BF16;
  const auto kernel = cache->head_dim == 128
                          ? (bf16 ? (vec ? append_kernel<128, true, true> : append_kernel<128, true, false>)
                                  : (vec ? append_kernel<128, false, true> : append_kernel<128, false, false>))
                          : (bf16 ? (vec ? append_kernel<64, true, true> : append_kernel<64, true, false>)
                                  : (vec ? append_kernel<64, false, true> : append_kernel<64, false, false>));
  kernel<<<grid, kThreads, 0, stream>>>(c, s, kt, vt, split);
  return cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

int dspark_kv4_read(const dspark_kv4_cache* cache, const dspark_kv4_batch* batch, void* k, int64_t k_row,
                    int64_t k_head, void* v, int64_t v_row, int64_t v_head, int32_t dtype, cudaStream_t stream) {
  using namespace dspark::kv4;
  if (dtype < DSPARK_DTYPE_BF16 || dtype > DSPARK_DTYPE_F32) return DSPARK_ERR_INVALID_ARG;
  Cache c;
  Batch s;
  unsigned blocks = 0;
  Split split{};
  bool vec = false;
  const int rc = check_rows(cache, batch, k, k_row, k_head, v, v_row, v_head, dtype == DSPARK_DTYPE_F32 ? 4 : 2, &c,
                            &s, &blocks, &split, &vec);
  if (rc != DSPARK_OK) return rc;
  if (s.batch == 0 || blocks == 0 || (!k && !v)) return DSPARK_OK;
  const RowTensor kt{static_cast<uint8_t*>(k), k_row, k_head};
  const RowTensor vt{static_cast<uint8_t*>(v), v_row, v_head};
  const dim3 grid(blocks);
  using Kernel = void (*)(Cache, Batch, RowTensor, RowTensor, Split);
  static const Kernel kernels[2][3][2] = {
      {{read_kernel<64, 0, false>, read_kernel<64, 0, true>},
       {read_kernel<64, 1, false>, read_kernel<64, 1, true>},
       {read_kernel<64, 2, false>, read_kernel<64, 2, true>}},
      {{read_kernel<128, 0, false>, read_kernel<128, 0, true>},
       {read_kernel<128, 1, false>, read_kernel<128, 1, true>},
       {read_kernel<128, 2, false>, read_kernel<128, 2, true>}}};
  kernels[cache->head_dim == 128][dtype][vec]<<<grid, kThreads, 0, stream>>>(c, s, kt, vt, split);
  return cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

}  // extern "C"
