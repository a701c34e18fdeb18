// Microscaled 4-bit floating point, shared by its kernels.
//
// A row of K values (K a multiple of 32) is stored as K/2 data bytes and
// `scale pitch` scale bytes. Data: e2m1 codes (sign, two exponent bits, one
// mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), the value of
// even index in a byte's low half. Scales: one byte b for every 32 values, the
// power of two 2^(b - 127), 255 for not-a-number; padded with zeros to a
// multiple of 16 bytes, so that a row's scales of 512 values are one aligned
// 16-byte vector.
//
// Quantisation of 32 values with largest magnitude m: b = floor(log2 m) - 2 +
// 127, at least 0 (the largest e2m1 value is 6 = 1.5 * 2^2, so m * 2^(127-b)
// lies in [4, 8)); each value times 2^(127-b), which is exact in fp32, is
// rounded to the nearest e2m1 value, ties to the code with an even mantissa
// bit, above 6 to 6. A block that holds an infinity or a NaN gets b = 255: all
// of it stands for NaN.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace stm {
namespace mx4 {

constexpr int kBlock = 32;      // values per scale
constexpr int kScaleNaN = 255;

__host__ __device__ constexpr inline int64_t scale_pitch(int64_t K) { return round_up(ceil_div(K, kBlock), 16); }

// Scale byte of a block whose largest magnitude has the fp32 bits m (sign
// cleared). Magnitude bits order like the values, and NaN's are the largest.
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
  const int e = (int)(m >> 23);
  return e == 255 ? kScaleNaN : (uint32_t)max(e - 2, 0);
}

// 2^(127 - b) for a finite block's scale byte b (0 <= b <= 252); 0 for NaN.
__device__ __forceinline__ float inverse_scale(uint32_t b) {
  return b == kScaleNaN ? 0.f : __uint_as_float((254u - b) << 23);
}

// 2^(b - 127); NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == kScaleNaN ? 0x7fffffffu : b << 23);
}

// Eight fp32 values to eight codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t pack8(const float* f) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// Eight codes to fp32.
__device__ __forceinline__ void unpack8(uint32_t w, float* f) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

}  // namespace mx4
}  // namespace stm
