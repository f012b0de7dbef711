// kv_rows.cuh -- where a row of the paged cache lies, and how rows are rounded to
// the cache's 8 and 4 bits: what the kernels that write and read rows share.
#pragma once

#include <cuda_fp8.h>

#include "attn.cuh"

namespace qre {

constexpr int kBlock4 = 16;   // elements that share a scale in a QRE_E2M1 cache

// Bytes of one head of one page.
__host__ __device__ __forceinline__ size_t kv_head_bytes(const qre_kv_cache& c) {
  const size_t n = (size_t)c.page_size * c.head_dim;
  return c.dtype == QRE_E4M3 ? n : c.dtype == QRE_E2M1 ? n / 16 * 9 : 2 * n;
}

// Byte at which head 0 of the page of position pos of sequence s begins in layer `layer` of k and of v;
// -1: no page there.
__device__ __forceinline__ long long kv_page_at(const qre_kv_cache& c, int layer, int s, int pos, int ps_shift) {
  if (s < 0 || s >= c.max_seqs || pos < 0 || (pos >> ps_shift) >= c.max_pages) return -1;
  const int p = c.page_table[(size_t)s * c.max_pages + (pos >> ps_shift)];
  if (p < 0 || p >= c.n_pages) return -1;
  return ((long long)layer * c.n_pages + p) * c.n_kv_heads * (long long)kv_head_bytes(c);
}

// 1 / scale of a head, correctly rounded; 1 without scales.
__device__ __forceinline__ float kv_inverse(const float* scales, size_t i) { return scales ? __frcp_rn(scales[i]) : 1.0f; }

// Four fp32 as E4M3 bytes (nearest even, clamped).
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
         (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3) << 16;
}

// Eight fp32 as E2M1 codes, the first in the lowest four bits (nearest even, clamped to 6).
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// Two E2M1 codes, byte B of w, as an fp16 pair (the low four bits first).  The conversion takes any byte of a register;
// a shift in front of it would be an instruction more.
template <int B>
__device__ __forceinline__ uint32_t e2m1x2_to_half2(uint32_t w) {
  uint32_t r;
  if constexpr (B == 0) asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
  if constexpr (B == 1) asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
  if constexpr (B == 2) asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
  if constexpr (B == 3) asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
// Eight codes as four pairs.
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, uint32_t (&y)[4]) {
  y[0] = e2m1x2_to_half2<0>(w);
  y[1] = e2m1x2_to_half2<1>(w);
  y[2] = e2m1x2_to_half2<2>(w);
  y[3] = e2m1x2_to_half2<3>(w);
}

// The scale of a block whose largest magnitude is `most` (NaN if it has one).  The quotient is correctly
// rounded, so that the E4M3 rounding behind it decides as it would on the exact one: most / 6 is next to a
// middle of two E4M3 values only if it is that middle.
struct Scale4 {
  uint32_t byte;
  float s, inverse;   // inverse 0: all codes are 0
  bool infinite;
  __device__ __forceinline__ explicit Scale4(float most) {
    infinite = most == INFINITY;
    byte = (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(most, 6.0f), __NV_SATFINITE, __NV_E4M3);
    s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
    inverse = s > 0.0f ? __frcp_rn(s) : 0.0f;
  }
};

// Codes of eight elements of a block.  x / s is x times the inverse, corrected by its residual once (one step of
// Newton's method): where x / s is a middle of two codes exactly, this is that middle, and the tie goes to the
// even code; elsewhere the error of 2^-23 is far below the distance to one.
__device__ __forceinline__ uint32_t quantize4(const float (&x)[8], const Scale4& q) {
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = x[i] * q.inverse;
    t[i] = fmaf(fmaf(-y, q.s, x[i]), q.inverse, y);
  }
  if (q.infinite)   // an infinity has no residual
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (fabsf(x[i]) == INFINITY) t[i] = x[i];
  return q.inverse > 0.0f ? to_e2m1x8(t) : 0u;
}

template <int DT>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bits_to_float<DT>(u[i] & 0xffffu);
    x[2 * i + 1] = bits_to_float<DT>(u[i] >> 16);
  }
}
template <int DT>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]), pack2<DT>(x[4], x[5]), pack2<DT>(x[6], x[7]));
}

// The larger of two numbers' magnitudes, NaN if one is NaN (magnitudes order as their bits do).
__device__ __forceinline__ float max_magnitude(float a, float b) {
  const uint32_t x = __float_as_uint(a) & 0x7fffffffu, y = __float_as_uint(b) & 0x7fffffffu;
  return __uint_as_float(x > y ? x : y);
}
__device__ __forceinline__ float max_magnitude8(const float (&x)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_magnitude(m, x[i]);
  return m;
}

}  // namespace qre
