// Device helpers of 4-bit matrices: codes and scales to values and back.
#pragma once

#include "zero_ops_device.cuh"

namespace zk {

constexpr int kScaleTile = 512;  // bytes of scales of 128 rows, four blocks each

// Eight values to codes, the first in the lowest four bits (nearest, ties to
// the even code, beyond 6 to 6).
__device__ __forceinline__ uint32_t to_codes8(const float v[8]) {
  uint32_t r;
  asm("{ .reg .b8 a, b, c, d;\n"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      "mov.b32 %0, {a, b, c, d}; }"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
__device__ __forceinline__ void from_codes8(uint32_t codes, float v[8]) {
  uint32_t h[4];
  asm("{ .reg .b8 a, b, c, d;\n"
      "mov.b32 {a, b, c, d}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n"
      "cvt.rn.f16x2.e2m1x2 %3, d; }"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.f32.f16 %0, lo; cvt.f32.f16 %1, hi; }"
        : "=f"(v[2 * i]), "=f"(v[2 * i + 1])
        : "r"(h[i]));
}
// E4M3, nearest, beyond 448 to 448; and back.
__device__ __forceinline__ uint32_t to_e4m3(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
  return r & 0xFFu;
}
__device__ __forceinline__ float from_e4m3(uint32_t byte) {
  uint32_t h;
  float f;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)byte));
  asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.f32.f16 %0, lo; }" : "=f"(f) : "r"(h));
  return f;
}

// What a scale byte stands for, times g.
template <bool NV>
__device__ __forceinline__ float scale_value(uint32_t byte, float g) {
  if (NV) return byte == 0x7Fu ? __uint_as_float(0x7FC00000u) : __fmul_rn(from_e4m3(byte), g);
  if (byte == 0xFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

}  // namespace zk
