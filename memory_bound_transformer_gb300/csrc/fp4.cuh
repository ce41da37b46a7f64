// The 4-bit paged KV cache's number format (sm_103a conversions).
//
// A value is e2m1(code) * e4m3(scale byte) * g: a 4-bit code per value (sign,
// two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), one e4m3
// scale per 16 neighbouring channels of a token's head, and the tensor's fp32
// scale g. A (block, KV head) of a K or V pool is 9 d bytes: the codes of its
// 16 tokens [16][d / 2] (channel 2j in the low half of byte j), then their
// scales [16][d / 16].
#pragma once

#include "common.cuh"

namespace mbt {

constexpr int kFp4Group = 16;                                   // channels per scale
__host__ __device__ constexpr int fp4_unit_bytes(int d) { return kBlockTokens * (d / 2 + d / kFp4Group); }

// Two fp32 values to e2m1 codes, nearest (ties to even), saturating at 6: the
// first in the low half of the byte.
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float lo, float hi) {
  uint16_t r;
  asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n cvt.u16.u8 %0, t;\n}\n" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}

// The eight e2m1 codes of a word as four FP16 pairs, exactly: pair j holds the
// codes of byte j (low half of the byte in the low half of the pair).
__device__ __forceinline__ void e2m1x8_to_h2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

// The same for the four codes of a 16-bit word.
__device__ __forceinline__ void e2m1x4_to_h2(uint32_t w, uint32_t (&h)[2]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %2;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n}\n"
      : "=r"(h[0]), "=r"(h[1]) : "r"(w));
}

__device__ __forceinline__ float2 h2_to_float2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace mbt
