// The 4-bit cache format and its conversions (sm_103a).
//
// 16 consecutive dims of one token's head row are 16 E2M1 codes (two a byte, the lower dim in the low
// nibble) and one E4M3 scale; a code's value is e2m1 * scale * (one fp32 scale per kv head).  A
// (block, head) page holds the codes of its 16 tokens, then their scales: 9 d contiguous bytes, which
// the tile kernel moves as one bulk copy and the rows kernel as 16-byte cp.async pieces.  The scale belongs to the token, so storing a token never
// re-encodes its neighbours.  e2m1 * e4m3 has at most six significant bits and lies in
// [2^-10, 2688]: exact in f16.
#pragma once

#include "pa_device.cuh"

namespace pa {

template <int D>
struct Fp4Page {
  static constexpr int kCodeRow = D / 2;                 // code bytes of one token
  static constexpr int kScaleRow = D / 16;               // scale bytes of one token
  static constexpr int kCodeBytes = 16 * kCodeRow;
  static constexpr int kBytes = kCodeBytes + 16 * kScaleRow;  // 9 d
  static_assert(kBytes % 16 == 0, "a page is a whole number of 16-byte pieces");
};

// Eight E2M1 codes (nibble i = code i) -> four f16 pairs (codes 2i, 2i + 1), exactly.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Eight floats -> eight E2M1 codes (to nearest even, saturating at +-6; a NaN becomes 6).
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float* f) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return w;
}

}  // namespace pa
