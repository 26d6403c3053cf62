// Device helpers of the microscaled 4-bit cache: 16 E2M1 elements share one E4M3 scale, a tensor
// one float scale. Element 2j of a record sits in the low half of code byte j, element 2j + 1 in
// the high half.
#pragma once

#include "mx_walk.cuh"
#include "tq_device.cuh"

namespace tq {
namespace mx {

constexpr int kBlock = 16; // elements that share a scale

// The four (low, high) element pairs of a code word as fp16 pairs (exact).
__device__ __forceinline__ void e2m1_to_h2(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n"
      ".reg .b8 b0, b1, b2, b3;\n"
      "mov.b32 {b0, b1, b2, b3}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n"
      "}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// Two E4M3 bytes (low 16 bits of w) as an fp16 pair (exact; 0x7F and 0xFF are NaN).
__device__ __forceinline__ uint32_t e4m3_to_h2(uint32_t w) {
  uint32_t r;
  asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(r) : "r"(w));
  return r;
}

__device__ __forceinline__ float e4m3_to_float(uint32_t byte) {
  const uint32_t h = e4m3_to_h2(byte & 0xFFu);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}

// v >= 0 to E4M3, to nearest with ties to even, saturating at 448.
__device__ __forceinline__ uint32_t float_to_e4m3(float v) {
  uint32_t r;
  asm("{\n.reg .b16 t;\ncvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\ncvt.u32.u16 %0, t;\n}" : "=r"(r) : "f"(0.0f), "f"(v));
  return r & 0xFFu;
}

// Eight values to E2M1 codes of one word, to nearest with ties to even, saturating at 6.
__device__ __forceinline__ uint32_t float_to_e2m1(const float *v) {
  uint32_t r;
  asm("{\n"
      ".reg .b8 b0, b1, b2, b3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      "mov.b32 %0, {b0, b1, b2, b3};\n"
      "}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

} // namespace mx
} // namespace tq
