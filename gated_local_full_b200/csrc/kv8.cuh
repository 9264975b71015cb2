// The 8-bit formats of the quantised paged cache.
//
// A block's codes of one KV head and of K or V share one float32 scale:
//   scale = max |x| / top, kept at least as large as before while the block
//           fills (0 below 2^-107, well before 1 / scale and what the
//           attention makes of a scale leave float32; NaN when a value is not
//           finite);
//   code  = round_to_format(x * (1 / scale)), value = code * scale.
// scale, 1 / scale and the products are single float32 roundings, so a host or
// another kernel that follows the formula gets the same codes. The one step
// that loses information is the rounding to the format: int8 whole numbers in
// [-127, 127] (symmetric, so that -x has the code of x negated), or e4m3
// (largest 448), both to nearest with ties to even.
#pragma once

#include <cuda_fp16.h>

#include "oda_internal.cuh"

namespace oda {

constexpr int kInt8 = ODA_KV8_INT8, kE4m3 = ODA_KV8_E4M3;

template <int FMT>
struct Fmt8;

template <>
struct Fmt8<kInt8> {
  static constexpr float kTop = 127.f;
  // four codes -> two f16 pairs, exactly: a byte xored with 0x80 under the
  // exponent of 1024 is 1024 + 128 + code
  static __device__ __forceinline__ void to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));   // 1152
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias);
    __half2 y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
    lo = *reinterpret_cast<uint32_t*>(&x);
    hi = *reinterpret_cast<uint32_t*>(&y);
  }
  // four float32 within +-127 -> four codes: added to 1.5 * 2^23 they are rounded to
  // whole numbers, ties to even, in the sum's low byte
  static __device__ __forceinline__ uint32_t pack(float x, float y, float z, float w) {
    const uint32_t a = __byte_perm(__float_as_uint(__fadd_rn(x, 0x1.8p23f)),
                                   __float_as_uint(__fadd_rn(y, 0x1.8p23f)), 0x0040);
    const uint32_t b = __byte_perm(__float_as_uint(__fadd_rn(z, 0x1.8p23f)),
                                   __float_as_uint(__fadd_rn(w, 0x1.8p23f)), 0x0040);
    return __byte_perm(a, b, 0x5410);
  }
};

template <>
struct Fmt8<kE4m3> {
  static constexpr float kTop = 448.f;
  static __device__ __forceinline__ void to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y, float z, float w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(r)
        : "f"(x), "f"(y), "f"(z), "f"(w));
    return r;
  }
};

// Four codes -> four float32, exactly.
template <int FMT>
__device__ __forceinline__ float4 codes_to_f32(uint32_t w) {
  uint32_t lo, hi;
  Fmt8<FMT>::to_f16(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<__half2*>(&hi));
  return make_float4(a.x, a.y, b.x, b.y);
}

}  // namespace oda
