// The 8-bit cache's number formats: e4m3 codes (four exponent bits, three of
// mantissa, no infinity, largest value 448) and the power-of-two scale of a page and
// KV head, held as the exponent byte b of 2^(b - 127).
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace metis {

// A byte, a piece of codes or of rows: ordinary loads (see pdl_wait)
__device__ __forceinline__ uint32_t ld_byte(const uint8_t* p) { return *p; }

template <typename T>
__device__ __forceinline__ T ld_codes(const T* p) {
  return *p;
}

// 2^(b - 127): b = 0 is the subnormal 2^-127, b = 255 (never written) is NaN
__device__ __forceinline__ float scale_of_byte(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7fc00000u : b << 23);
}

// Its exponent (finite for 255 too, which the caller has to treat apart)
__device__ __forceinline__ float exponent_of_byte(uint32_t b) { return (float)((int)b - 127); }

// The exponent byte of the smallest 2^k with amax <= 448 * 2^k, at least 1 (2^-126).
// amax is finite and >= 0: with amax = m * 2^e, 1 <= m < 2, and 448 = 1.75 * 2^8, that
// is k = e - 8, or e - 7 when m > 1.75.
__device__ __forceinline__ uint32_t byte_of_amax(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int b = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(b, 1);
}

// Two floats to e4m3, round to nearest even (`lo` in the low byte); NaN becomes 0x7f,
// values past 448 saturate (a page's scale leaves none).
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  return pack_e4m3x2(a, b) | (pack_e4m3x2(c, d) << 16);
}

// Four codes to fp16 (exact): bytes 0, 1 -> *lo, bytes 2, 3 -> *hi
__device__ __forceinline__ void unpack_e4m3x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// Four codes to fp32 (exact)
__device__ __forceinline__ void unpack_e4m3x4_f32(uint32_t w, float* v) {
  uint32_t lo, hi;
  unpack_e4m3x4(w, lo, hi);
  const float2 a = unpack_f16x2(lo), b = unpack_f16x2(hi);
  v[0] = a.x;
  v[1] = a.y;
  v[2] = b.x;
  v[3] = b.y;
}

__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}

// fp16 pair to e4m3, round to nearest even, past 448 saturated
__device__ __forceinline__ uint16_t e4m3x2_of_f16x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// max that returns NaN if either is NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// A pair of fp16 pairs as two e4m3 parts, x = hi + lo up to lo's rounding (|x| at most 448).
// Results: the codes of (a lo, a hi, b lo, b hi), low byte first.
__device__ __forceinline__ void split_e4m3x2x2(uint32_t a, uint32_t b, uint32_t& hi, uint32_t& lo) {
  const uint16_t ha = e4m3x2_of_f16x2(a), hb = e4m3x2_of_f16x2(b);
  const uint32_t ba = f16x2_of_e4m3x2(ha), bb = f16x2_of_e4m3x2(hb);
  // exact: x and its code lie within a factor of two or in the subnormals of one grid
  const __half2 ra = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&ba));
  const __half2 rb = __hsub2(*reinterpret_cast<const __half2*>(&b), *reinterpret_cast<const __half2*>(&bb));
  hi = ha | ((uint32_t)hb << 16);
  lo = e4m3x2_of_f16x2(*reinterpret_cast<const uint32_t*>(&ra)) |
       ((uint32_t)e4m3x2_of_f16x2(*reinterpret_cast<const uint32_t*>(&rb)) << 16);
}

// Two floats to fp16 (round to nearest even)
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Four bf16 values times `up` (a power of two) as two e4m3 parts
__device__ __forceinline__ void split_e4m3x4(const uint2& v, float up, uint32_t& hi, uint32_t& lo) {
  const uint64_t up2 = f2_pack(up, up);
  float x0, x1, x2, x3;
  f2_unpack(f2_mul(f2_pack(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u)), up2), x0, x1);
  f2_unpack(f2_mul(f2_pack(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u)), up2), x2, x3);
  split_e4m3x2x2(pack_f16x2(x0, x1), pack_f16x2(x2, x3), hi, lo);
}

// D(16x8, f32) += A(16x16, fp16, row) * B(16x8, fp16, col)
__device__ __forceinline__ void mma_f16_16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

}  // namespace metis
