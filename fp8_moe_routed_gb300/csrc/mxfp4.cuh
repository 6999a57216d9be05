// mxfp4.cuh -- OCP microscaled FP4: e2m1 elements in blocks of 32 along K, each
// with a power-of-two scale (e8m0).
//
//   X = 2^(floor(log2 amax) - 2), not below 2^-127;  code = e2m1(v / X), round to
//   nearest even, saturating at +-6;  scale byte = log2 X + 127.
// 2 is the largest exponent of e2m1 (4 and 6). A block with an infinity or a NaN
// gets the scale byte 0xFF (NaN): everything computed from it is NaN instead of a
// plausible number. v / X is exact (a power of two), so codes have one right value.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace fp8moe {

constexpr int kMxBlock = 32;
constexpr int kMxWord = 128;      // K values whose four scale bytes share a 32-bit word
constexpr uint32_t kMxNan = 0xFFu;

// Scale byte of a block whose largest magnitude has these bf16 bits. As integers
// the bits of magnitudes are ordered like the values, with infinity and NaN last,
// and their upper eight bits are the biased exponent floor(log2) + 127.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 7;
  return e == 0xFFu ? kMxNan : e > 2u ? e - 2u : 0u;
}

// 1 / X for a scale byte (<= 252 when not NaN): 2^(127 - byte), a normal number. A NaN
// byte gives some number: the caller does not use the codes.
__device__ __forceinline__ float mx_inv_scale(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// X itself: 2^(byte - 127); byte 0 is the subnormal 2^-127, 0xFF is NaN.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return byte == kMxNan ? __uint_as_float(0x7FFFFFFFu)
                        : byte ? __uint_as_float(byte << 23) : __uint_as_float(1u << 22);
}

// Eight f32 -> eight e2m1 codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float2 (&f)[4]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r) : "f"(f[0].x), "f"(f[0].y), "f"(f[1].x), "f"(f[1].y), "f"(f[2].x), "f"(f[2].y),
        "f"(f[3].x), "f"(f[3].y));
  return r;
}

// Eight e2m1 codes -> four f16 pairs (exact), lowest code first.
__device__ __forceinline__ void e2m1x8_to_f16x2x4(uint32_t v, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(v));
}

}  // namespace fp8moe
