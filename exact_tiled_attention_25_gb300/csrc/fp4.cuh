// 4-bit cache rows: e2m1 codes and one bfloat16 descale per row.
//
// A code is a sign bit and a magnitude of 0, 0.5, 1, 1.5, 2, 3, 4 or 6; element 2 i of a
// row is the low half of byte i.  A row x of d values is held as
//     s = amax|x| / 6 rounded up to bfloat16 (at least 2^-100; 0 for a row of zeros),
//     code = e2m1_rn(x / s),      value = code * s.
// Rounding s up keeps every quotient within 6, so no value is cut off; what the eight bits
// of s cost is part of the step of the codes, which are taken relative to the s that is
// stored.  A row that holds an infinity or a NaN gets s = NaN and codes of 0: it reads
// back as NaN instead of as some finite number.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sm103_prims.cuh"

namespace attn {

constexpr float kMinRowDescale = 0x1p-100f;   // 1 / s and the quotients' residuals stay normal numbers

// Eight float32 -> a word of eight codes (element 0 in the lowest four bits), round to nearest even, largest 6.
__device__ __forceinline__ uint32_t e2m1_word(const float (&x)[8]) {
  uint32_t w;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(w)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return w;
}

// The eight codes of a word as four pairs of float16 (exact), element 2 i in the low half.
__device__ __forceinline__ void e2m1_halves(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ float bf16_bits(uint32_t b) { return __uint_as_float(b << 16); }

// The descale of a row whose largest magnitude has these float32 bits (as an integer, so
// that infinities and NaNs win).
__device__ __forceinline__ float row_descale(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return __uint_as_float(0x7FFF0000u);
  if (amax_bits == 0u) return 0.f;
  const uint32_t up = (__float_as_uint(__fdiv_rn(__uint_as_float(amax_bits), 6.f)) + 0xFFFFu) & 0xFFFF0000u;
  return fmaxf(__uint_as_float(up), kMinRowDescale);
}

}  // namespace attn
