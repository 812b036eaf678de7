// qsa_kv4.cuh -- the 4-bit cache format shared by its writer and its readers:
// a row (token, KV head, K or V) of 80 bytes, 64 of e2m1 codes (value 2i in
// the low half of byte i), 8 e4m3 scales of 16 values each, the fp32 row scale,
// 4 zero bytes.  The last 16 bytes are the row's scale chunk.
#pragma once

#include "qsa_kv8.cuh"

namespace qsa {

constexpr int kKv4Codes = 64;     // bytes of codes
constexpr int kKv4Chunk = 16;     // bytes of the scale chunk behind them
constexpr float kE2m1Max = 6.0f;  // codes 0 0.5 1 1.5 2 3 4 6, bit 3 the sign

// The eight e2m1 codes of a word as four f16 pairs: pair i holds byte i's low code, then its high one.  Exact.
__device__ __forceinline__ void e2m1_to_f16(uint32_t w, uint32_t& p0, uint32_t& p1, uint32_t& p2, uint32_t& p3) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(p0), "=r"(p1), "=r"(p2), "=r"(p3)
      : "r"(w));
}
// Eight fp32 values as e2m1 codes (value i in nibble i), to nearest even, saturating at 6.
__device__ __forceinline__ uint32_t f32_to_e2m1(const float (&x)[8]) {
  uint32_t w;
  asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(w)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return w;
}
// Products of f16 pairs.
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

}  // namespace qsa
