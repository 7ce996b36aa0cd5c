// Microscaled 4-bit floating point on the device: E2M1 values (sign, two exponent bits, one
// mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), 32 of them sharing one E8M0
// scale 2^(code - 127), code 255 = NaN (the OCP Microscaling Formats specification, MXFP4).
#pragma once

#include "common.cuh"

namespace bskv {
namespace dev {

constexpr int kFp4Block = 32;  // values per scale

// Two fp32 values to E2M1, round to nearest even, saturating to +-6; `lo` in bits 0-3.
__device__ __forceinline__ uint32_t cvt_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\t"
      "mov.b32 %0, {t, 0, 0, 0};\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}

// The eight E2M1 values of a word as f16 pairs: r[i] holds byte i (low nibble in the low half).
__device__ __forceinline__ void cvt_e2m1x8(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// The four E2M1 values of the low two bytes of a word as f16 pairs.
__device__ __forceinline__ void cvt_e2m1x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// Scale code of a block whose largest magnitude has the fp32 bits `top` (sign cleared):
// 2^(floor(log2 max) - 2), so that the largest value lands in [4, 8) and rounds to 4 or 6;
// 0 (2^-127) below 2^-125; 255 (NaN) when the block holds an infinity or a NaN.
__device__ __forceinline__ uint32_t e8m0_of_max(uint32_t top) {
  const uint32_t e = top >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 2^(127 - code) for code <= 252 (what e8m0_of_max gives for finite blocks).
__device__ __forceinline__ float e8m0_inverse(uint32_t code) {
  return __uint_as_float((254u - code) << 23);
}
// 2^(code - 127), exactly (code 0 is an fp32 subnormal); NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t code) {
  return __uint_as_float(code == 255u ? 0x7fffffffu : code == 0u ? 0x00400000u : code << 23);
}

// Page and slot of token `pos` of request `b` through a device page table; false when the
// request, position or page is out of range.
__device__ __forceinline__ bool page_slot(const int32_t* indptr, const int32_t* indices,
                                          int32_t batch, int32_t page_size, int64_t num_pages,
                                          int32_t b, int32_t pos, int32_t& page, int32_t& slot) {
  if (b < 0 || b >= batch || pos < 0) return false;
  const int64_t at = int64_t(__ldg(indptr + b)) + pos / page_size;
  if (at >= __ldg(indptr + b + 1)) return false;
  page = __ldg(indices + at);
  slot = pos % page_size;
  return page >= 0 && page < num_pages;
}

}  // namespace dev
}  // namespace bskv
