// The 4-bit pools' format: E2M1 codes with an E4M3 scale for every 16 channels.
//
// A page of B tokens is B * D * 9/16 bytes in lines of 144: the codes of 256 / D
// consecutive tokens (128 bytes), then their 16 scales. One contiguous run per
// page is one bulk copy; a line of 9 x 16 bytes puts the same 16-byte piece of
// consecutive lines into different shared memory banks.
#pragma once

#include "common.cuh"

namespace pkv {

constexpr int kFp4Line = 144;
constexpr int kFp4Group = 16;  // channels that share a scale

// Byte offsets inside a page of token t's codes and of its scales.
template <int D>
__host__ __device__ constexpr int fp4_codes_at(int t) {
  return D == 256 ? t * kFp4Line : (t >> 1) * kFp4Line + (t & 1) * 64;
}
template <int D>
__host__ __device__ constexpr int fp4_scales_at(int t) {
  return D == 256 ? t * kFp4Line + 128 : (t >> 1) * kFp4Line + 128 + (t & 1) * 8;
}

// The eight E2M1 codes of w as four f16x2, byte after byte, low code first (exact).
__device__ __forceinline__ void e2m1x8_f16x2(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

// Eight fp32 -> a word of E2M1 codes, the first in its lowest four bits (nearest, ties
// to the even code, saturating).
__device__ __forceinline__ uint32_t e2m1x8_of(const float (&x)[8]) {
  uint32_t d;
  asm("{\n\t.reg .b8 a, b, c, e;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 e, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, e};\n\t}"
      : "=r"(d)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return d;
}

// The two E4M3 codes in the low 16 bits of w as f16x2 (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2_lo(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w)));
  return h;
}

// One E4M3 code as fp32 (exact; NaN stays NaN).
__device__ __forceinline__ float e4m3_f32(uint8_t x) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(x)));
  return __low2float(*reinterpret_cast<__half2*>(&h));
}

// How rows of `per` 8-channel pieces are dealt to threads: a CTA has whole rows, `rows` of
// them side by side, so that a thread's piece is the same in every one it has (its head,
// its scales) and the row is found without a division.
struct RowsOfCta {
  uint32_t per, rows, inverse;  // inverse: of per, for a product in the place of a division

  static constexpr int kThreads = 256;  // or one row, up to 1024

  explicit RowsOfCta(int per_row)
      : per(per_row), rows(per_row < kThreads ? kThreads / per_row : 1),
        inverse((1u << 16) / per_row + 1) {}
  int threads() const { return static_cast<int>((rows * per + 31) / 32 * 32); }

  // The row of the CTA's that thread tid has a piece of, `rows` or more for none. (Below
  // 256 threads tid * per is below 2^16, so that the rounded-up inverse is exact.)
  __device__ __forceinline__ uint32_t row_of(uint32_t tid) const {
    return rows == 1 ? (tid >= per ? 1 : 0) : (tid * inverse) >> 16;
  }
};

}  // namespace pkv
