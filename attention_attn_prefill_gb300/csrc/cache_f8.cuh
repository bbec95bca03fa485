// The 8-bit paged cache: number format and layout of a record (one page of one KV head).
//
// The 16 tokens of a page share a scale for their keys and one for their values: a power of two, 2^e, with the
// smallest e >= -124 for which no finite value exceeds 448 2^e.  A value's code is x 2^-e rounded to e4m3 (4
// significant bits, largest number 448), nearest even, and stands for the code times 2^e.  A power of two takes
// nothing from a floating-point code's precision, which does not depend on where in its range a number lies; it
// makes every stored value a bf16 number exactly, and lets a page's codes move to a larger scale without a second
// rounding, but for numbers that fall below 2^-6 of the new scale's unit.  NaN and infinities become NaN.
//
// Record of 32 d + 16 bytes, in the order in which the decode kernel's lanes (lane = 4 g + t of a warp) take it, as
// wide loads without bank conflicts:
//   [0, 16 d)      K codes.  Row (i, j) of 512 bytes: 16-byte word of lane 4 g + t holds channels
//                  64 j + 16 t .. + 15 of token 8 i + g.
//   [16 d, 32 d)   V codes.  B = min(16, d / 8) bytes a lane: row (b1, b0, h) holds at lane 4 g + t channels
//                  8 B h + B g .. + B - 1 of token 8 b1 + 2 t + b0.
//   [32 d, + 16)   f32 scale of the keys, f32 scale of the values, 8 bytes unused
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace attn {
namespace f8 {

constexpr int PAGE = 16;
constexpr uint32_t LEAST = 3;  // biased exponent of the smallest scale, 2^-124

template <int D>
struct Record {
  static constexpr int VB = D / 8 < 16 ? D / 8 : 16;  // bytes of a token that a lane holds in a V row
  static constexpr int VH = D / (8 * VB);             // V rows a token
  static constexpr int KJ = D / 64;                   // K rows a token
  static constexpr int K_OFF = 0;
  static constexpr int V_OFF = 16 * D;
  static constexpr int S_OFF = 32 * D;
  static constexpr int BYTES = 32 * D + 16;
};

// Biased exponent of the scale for a largest magnitude (the bits of a finite bf16 without its sign): 448 is
// 1.75 2^8, so a mantissa past 0.75 takes the next power.
__device__ __forceinline__ uint32_t scale_exponent(uint32_t most) {
  const uint32_t e = (most + 0x1fu) >> 7;
  return e < LEAST + 8 ? LEAST : e - 8;
}
__device__ __forceinline__ float pow2(uint32_t biased) { return __uint_as_float(biased << 23); }

// two floats -> two codes, `lo` in the lower byte
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

// the two codes in the lower half of w as fp16 numbers, the lower byte in the lower half
__device__ __forceinline__ uint32_t halves2(uint32_t w) {
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(d) : "r"(w));
  return d;
}
// those in the upper half
__device__ __forceinline__ uint32_t halves2_upper(uint32_t w) {
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(d) : "r"(w));
  return d;
}

}  // namespace f8
}  // namespace attn
