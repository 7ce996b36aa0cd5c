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

// (a & 0x0f0f0f0f) | (b & 0xf0f0f0f0) in one instruction (written out, the compiler narrows the
// masks to the bits it knows and needs two).
__device__ __forceinline__ uint32_t nibbles(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, 0x0f0f0f0f, 0xE4;" : "=r"(r) : "r"(a), "r"(b));
  return r;
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

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// The scales 2^(code - 127) of the codes in a word's bytes as fp32, exactly; NaN for 255.
template <int NB>
__device__ __forceinline__ void scales_of(uint32_t w, float (&f)[NB]) {
#pragma unroll
  for (int i = 0; i < NB; i += 2) {
    uint32_t pair;  // bf16 has fp32's exponents
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %0, lo;\n\t}" : "=r"(pair) : "r"(i ? w >> 16 : w));
    f[i] = __uint_as_float(pair << 16);
    f[i + 1] = __uint_as_float(pair & 0xffff0000u);
  }
}

// Scale codes of row `row` of a shared-memory tile (2 bytes for D = 64).
template <int D>
__device__ __forceinline__ uint32_t scale_word(const uint8_t* s, int row) {
  if constexpr (D == 128) return *reinterpret_cast<const uint32_t*>(s + 4 * row);
  else return *reinterpret_cast<const uint16_t*>(s + 2 * row);
}

__device__ __forceinline__ int exponent_of(float x) {
  return int(__float_as_uint(x) >> 23) - 127;
}
__device__ __forceinline__ float pow2(int k) { return __uint_as_float(uint32_t(k + 127) << 23); }

__device__ __forceinline__ float max_over_rows(float x) {  // lanes of equal lane & 3
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float sum_over_rows(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// The B fragments of a query row of D = 32 NB values for products over NB 32-value blocks: lane
// (g, t) holds values 32 b + 8 t .. + 7 of row g as four f16 pairs per block b. bf16 rows are
// multiplied by the power of two that puts their largest magnitude into [2^14, 2^15) (exact:
// values below 2^-29 of it may lose low bits to f16's subnormals); returns its inverse. `negate`
// flips the row's signs.
template <typename T, int NB>
__device__ __forceinline__ float load_q_f16(const T* row, bool live, bool negate, int lane,
                                            uint32_t (&q)[NB][4]) {
  const int t = lane & 3;
  uint4 x[NB];
#pragma unroll
  for (int blk = 0; blk < NB; ++blk)
    x[blk] = live ? __ldg(reinterpret_cast<const uint4*>(row + 32 * blk + 8 * t)) : make_uint4(0, 0, 0, 0);
  if constexpr (__is_same(T, __half)) {
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      const uint32_t sign = negate ? 0x80008000u : 0u;
      q[blk][0] = x[blk].x ^ sign;
      q[blk][1] = x[blk].y ^ sign;
      q[blk][2] = x[blk].z ^ sign;
      q[blk][3] = x[blk].w ^ sign;
    }
    return 1.f;
  } else {
    uint32_t top = 0;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      const uint32_t w[4] = {x[blk].x, x[blk].y, x[blk].z, x[blk].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = int(top >> 7);
    const int k = e == 255 ? 0 : min(141 - e, 126);
    const float f = negate ? -pow2(k) : pow2(k);
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      const uint32_t w[4] = {x[blk].x, x[blk].y, x[blk].z, x[blk].w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        q[blk][i] = pack_half2(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
    }
    return pow2(-k);
  }
}

}  // namespace dev
}  // namespace bskv
