// packed.cuh -- the 4-bit latent row and the instructions that read and write it.
//
// A row of 512 latents takes 288 bytes: 256 bytes of e2m1 codes (latent 2k in the low nibble
// of byte k, 2k + 1 in the high one), then one e4m3 scale for each group of 16 latents:
//   c[i] = unit * scale[i / 16] * code[i],   code in +-{0, 0.5, 1, 1.5, 2, 3, 4, 6},
// unit a power of two that the caller chooses for the whole cache.  A product scale * code has
// at most six significant bits and lies in +-[2^-10, 2688]: exact in fp16 and in bf16.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace mla {
namespace packed {

constexpr int kGroup = 16;                            // latents per scale
constexpr int kCodeBytes = kLatent / 2;               // 256
constexpr int kScaleBytes = kLatent / kGroup;         // 32
constexpr int kRowBytes = kCodeBytes + kScaleBytes;   // 288
constexpr int kPageBytes = kPageTokens * kRowBytes;   // 18,432

// The four bytes of w, each a pair of e2m1 codes (low nibble first), as four pairs of fp16.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
// Two e4m3 scales (the low 16 bits) as a pair of fp16 (every e4m3 value is exact in fp16).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(v));
  return r;
}
// Two floats to e4m3, nearest even, at most 448; lo in the low byte.
__device__ __forceinline__ uint32_t f32_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Eight floats to e2m1, nearest with ties to even, at most 6 in size; the first in the lowest nibble.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// Round to nearest; subnormal operands and results are kept.
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Power-of-two check of a caller's unit: finite, positive, one significant bit, and far enough
// from the ends of the range that it and its reciprocal keep a row's values normal.
inline bool valid_unit(float unit) {
  uint32_t bits;
  __builtin_memcpy(&bits, &unit, 4);
  const uint32_t e = bits >> 23;
  return (bits & 0x7FFFFFu) == 0 && e >= 127 - 64 && e <= 127 + 64;
}

}  // namespace packed
}  // namespace mla
