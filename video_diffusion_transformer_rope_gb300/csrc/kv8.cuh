// Device helpers of the 8-bit cache: e4m3 codes of 16-token blocks with a power of two as scale.
//
// A value is code * 2^e.  With e in [-15, 7] it is exact in bf16 and in fp16: the largest is 448 * 2^7 = 57344, the
// smallest step 2^-9 * 2^-15 = 2^-24, fp16's own.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

namespace vdx {

constexpr int kBlock8 = 16;
constexpr int kMinExp8 = -15, kMaxExp8 = 7;

// The least e in range with amax <= 448 * 2^e = 1.75 * 2^(8 + e); amax >= 0, infinity included.
__device__ __forceinline__ int block_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kMinExp8), kMaxExp8);
}
__device__ __forceinline__ int scale_exponent(uint8_t byte) {
  return min(max(static_cast<int>(byte) - 127, kMinExp8), kMaxExp8);
}
__device__ __forceinline__ float two_to(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// 2^e as both halves of a pair of fp16; e >= -14 is normal, -15 the subnormal 2^-15.
__device__ __forceinline__ uint32_t half_two_to(int e) {
  return e > kMinExp8 ? static_cast<uint32_t>(e + 15) << 10 : 0x200u;
}

// Two floats to codes, nearest even, clamped to 448; the first in the low byte.
__device__ __forceinline__ uint32_t encode2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  return encode2(a, b) | (encode2(c, d) << 16);
}
// The two codes of the low (kHigh: high) half of w as a pair of fp16, exactly.
template <bool kHigh>
__device__ __forceinline__ uint32_t decode2(uint32_t w) {
  uint32_t r;
  if (kHigh)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Four codes as two pairs of T times a power of two, exactly: `scale` is pair_two_to<T>(e).  NaN codes come out as NaN in
// fp16 and as 480 in bf16; any_nan(top) tells whether there was one among the codes of all calls that shared `top`, 0 at first.
template <typename T>
__device__ __forceinline__ uint32_t pair_two_to(int e);
template <>
__device__ __forceinline__ uint32_t pair_two_to<__half>(int e) {
  return half_two_to(e) * 0x10001u;
}
template <>
__device__ __forceinline__ uint32_t pair_two_to<__nv_bfloat16>(int e) {
  return static_cast<uint32_t>(e + 120 + 127) * 0x800080u;       // times the 2^120 that decode4 leaves out
}
template <typename T>
__device__ __forceinline__ void decode4(uint32_t w, uint32_t scale, uint32_t& lo, uint32_t& hi, uint32_t& top);
template <>
__device__ __forceinline__ void decode4<__half>(uint32_t w, uint32_t scale, uint32_t& lo, uint32_t& hi, uint32_t&) {
  lo = half2_mul(decode2<false>(w), scale);
  hi = half2_mul(decode2<true>(w), scale);
}
// A code's exponent and mantissa, moved to where bf16 has its own, are its value times 2^-120 (subnormals too).
template <>
__device__ __forceinline__ void decode4<__nv_bfloat16>(uint32_t w, uint32_t scale, uint32_t& lo, uint32_t& hi, uint32_t& top) {
  const uint32_t h[2] = {__byte_perm(w, 0u, 0x1404), __byte_perm(w, 0u, 0x3424)};
  uint32_t m[2], r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    m[i] = (h[i] & 0x7f007f00u) >> 4;
    const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&m[i]), *reinterpret_cast<const __nv_bfloat162*>(&scale));
    r[i] = *reinterpret_cast<const uint32_t*>(&v) | (h[i] & 0x80008000u);
  }
  top = __vimax3_u16x2(top, m[0], m[1]);               // NaN put in its place here costs 4 for each pair: a 480p frame's weights 310 us, not 299
  lo = r[0];
  hi = r[1];
}
__device__ __forceinline__ bool any_nan(uint32_t top) { return max(top & 0xffffu, top >> 16) == 0x7f0u; }
__device__ __forceinline__ void decode8(const uint2& x, float (&f)[8]) {
  const uint32_t h[4] = {decode2<false>(x.x), decode2<true>(x.x), decode2<false>(x.y), decode2<true>(x.y)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

}  // namespace vdx
