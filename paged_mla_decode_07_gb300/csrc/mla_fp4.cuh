// FP4 cache rows: 400 bytes per token.
//
//   bytes [0, 256)    64 words of eight 4-bit codes (E2M1: 0, 1/2, 1, 3/2, 2, 3, 4, 6 and a sign)
//   bytes [256, 272)  16 scale bytes, byte s for dims 32 s .. 32 s + 31: 2^(byte - 127)
//   bytes [272, 400)  64 bf16 RoPE values
//
// Word w holds dims 8 w .. 8 w + 7: bits 4 i .. 4 i + 2 are the magnitude of dim
// i, bit 8 i + 7 the sign of dim i and bit 8 i + 3 that of dim 4 + i (i < 4).
// With the signs at the places that they have in a word of four 8-bit floats,
// eight codes become eight such floats with two byte permutations and five
// logical instructions (the plain order would take four and seven).
//
// Scales are 2^-13 .. 2^13 (bytes 114 .. 140; other bytes are read as the
// nearest of these): then every value code * scale is an E5M2 number, so
// products over FP4 rows take the rows as 8-bit operands, exactly, and no bytes
// that a row may hold make a latent value that is not finite.
#pragma once

#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {

constexpr int kFp4RowBytes = 400;
constexpr int kFp4ScaleOffset = 256;
constexpr int kFp4RopeOffset = 272;
constexpr int kFp4ScaleMin = 114, kFp4ScaleMax = 140;

// Smallest e with amax <= 6 * 2^e (clamped): amax = 1.f * 2^x is at most 6 * 2^(x - 2) where 1.f <= 1.5.
__device__ __forceinline__ int fp4_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 129 + ((u & 0x7fffffu) > 0x400000u ? 1 : 0);
  return min(max(e, kFp4ScaleMin - 127), kFp4ScaleMax - 127);
}

// Eight floats -> eight E2M1 codes (nearest even, saturated at 6; NaN: 6), code i at bits 4 i.
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight codes, code i at bits 4 i, with their signs moved to the places of a row's word.
__device__ __forceinline__ uint32_t fp4_word(uint32_t w) {
  auto spread = [](uint32_t h) {  // bits 3, 7, 11, 15 -> 3, 11, 19, 27
    h = (h | (h << 8)) & 0x00880088u;
    return (h | (h << 4)) & 0x08080808u;
  };
  return (w & 0x77777777u) | (spread(w & 0x8888u) << 4) | spread((w >> 16) & 0x8888u);
}

// The clamped scale of a byte, from 0 (2^-13) to 26 (2^13).
__device__ __forceinline__ uint32_t fp4_scale_index(uint32_t byte) {
  return static_cast<uint32_t>(min(max(static_cast<int>(byte), kFp4ScaleMin), kFp4ScaleMax) - kFp4ScaleMin);
}

// Word of a row -> its eight values as fp32, each times `scale`.
__device__ __forceinline__ void fp4_floats(uint32_t w, float scale, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // the code's three bits as the lowest exponent bits and the first mantissa bit of a float: 2^-126 of its value
    const uint32_t mag = ((w >> (4 * i)) & 7u) << 22;
    const uint32_t sign = (w >> (i < 4 ? 8 * i + 7 : 8 * (i - 4) + 3)) << 31;
    v[i] = __uint_as_float(mag | sign) * 8.507059173023462e37f * scale;
  }
}

// Word of a row -> two words of four E5M2 values (dims 0..3 and 4..7), each
// times the scale of `lut`, whose two words hold the eight magnitudes.
__device__ __forceinline__ uint2 fp4_lut(uint32_t scale_index) {
  // 0, 1/2, 1, 3/2 and 2, 3, 4, 6 at 2^-13; a binade up is 4 more in every byte (0 stays 0)
  return make_uint2(0x0a080400u + scale_index * 0x04040400u, 0x12100e0cu + scale_index * 0x04040404u);
}
__device__ __forceinline__ uint2 fp4_e5m2(uint32_t w, uint2 lut) {
  const uint32_t sel = w & 0x77777777u;
  uint2 r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r.x) : "r"(lut.x), "r"(lut.y), "r"(sel));
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r.y) : "r"(lut.x), "r"(lut.y), "r"(sel >> 16));
  r.x |= w & 0x80808080u;
  r.y |= (w << 4) & 0x80808080u;
  return r;
}

}  // namespace mla
