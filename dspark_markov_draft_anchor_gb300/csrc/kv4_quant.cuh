// kv4_quant.cuh -- how values become codes and scales of the paged 4-bit cache
// (kv4_cache.cu, kv4_rotate.cu).
#pragma once

#include "kv4.cuh"

namespace dspark {
namespace kv4 {
namespace {

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

}  // namespace
}  // namespace kv4
}  // namespace dspark
