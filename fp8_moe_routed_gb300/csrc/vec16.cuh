// vec16.cuh -- 16 bytes of bf16 or f32 values as pairs of f32 registers and back, and
// the packed f32 arithmetic on such pairs (one instruction for two values). Each is rounded
// like the scalar operation, but a product whose sum follows may be joined with it into one
// rounding, although both ask for their own: where that rounding matters, the product is
// taken by a scalar operation, which is never joined.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "ptx.cuh"

namespace fp8moe {

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  mul_f32x2(a.x, a.y, b.x, b.y, d.x, d.y);
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// kN values = kP pairs in 16 bytes.
template <typename T> struct Vec;
template <> struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8, kP = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float2 (&f)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(bf16lo_to_f32(w[i]), bf16hi_to_f32(w[i]));
  }
  static __device__ __forceinline__ uint4 pack(const float2 (&f)[4]) {
    return make_uint4(f32x2_to_bf16x2(f[0].x, f[0].y), f32x2_to_bf16x2(f[1].x, f[1].y),
                      f32x2_to_bf16x2(f[2].x, f[2].y), f32x2_to_bf16x2(f[3].x, f[3].y));
  }
};
template <> struct Vec<float> {
  static constexpr int kN = 4, kP = 2;
  static __device__ __forceinline__ void unpack(const uint4& v, float2 (&f)[2]) {
    f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  static __device__ __forceinline__ uint4 pack(const float2 (&f)[2]) {
    return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                      __float_as_uint(f[1].y));
  }
};

}  // namespace fp8moe
