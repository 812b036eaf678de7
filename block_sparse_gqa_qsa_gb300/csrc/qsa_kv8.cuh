// qsa_kv8.cuh -- the 8-bit cache format shared by its writer and its reader:
// e4m3 codes (conversions by the hardware's cvt) and the range of block scales.
#pragma once

#include "qsa_device.cuh"

namespace qsa {

constexpr float kE4m3Max = 448.0f;
constexpr float kScaleLo = 3.552713678800501e-15f;  // 2^-48
constexpr float kScaleHi = 2.81474976710656e14f;    // 2^48

// A stored scale as the kernels read it: inside [2^-48, 2^48], NaN as the lower bound (fmaxf returns the
// number of a number and a NaN).
__device__ __forceinline__ float read_scale(float s) { return fminf(fmaxf(s, kScaleLo), kScaleHi); }

// Four e4m3 codes (bytes 0..3 of w) as two f16 pairs; every code is an exact f16 value.
__device__ __forceinline__ void e4m3_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// Four fp32 values as e4m3 codes (byte i = xi), to nearest even; NaN gives NaN, larger values saturate at 448.
__device__ __forceinline__ uint32_t f32_to_e4m3(float x0, float x1, float x2, float x3) {
  uint32_t w;
  asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n"
      " mov.b32 %0, {a, b};\n}\n"
      : "=r"(w)
      : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
  return w;
}

}  // namespace qsa
