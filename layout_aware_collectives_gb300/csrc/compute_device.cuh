// Device helpers shared by the feed-forward unit's kernels: bf16 and e4m3
// conversions, the block scale, and the gate activations.
#pragma once

#include <math_constants.h>
#include <stdint.h>

#include "compute_internal.h"

namespace tide {

// The kernels ahead on the stream have ended and their writes are there; the
// next one may begin its set-up.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// Two floats to packed bf16, to nearest even: `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint16_t to_bf16(float v) { return (uint16_t)pack_bf16(v, 0.0f); }

// The largest finite magnitude e4m3 holds is 448 = 1.75 * 2^8.  The block
// scale is the smallest power of two >= 2^-126 that brings `amax`, the
// block's largest finite magnitude, to 448 or below; 1 for a block of zeros.
// Being a power of two it rounds nothing: a value's only rounding is e4m3's
// own, and code * scale is exact in bf16 (4 significant bits; below 2^-126
// it may round as any bf16 subnormal does).
__device__ __forceinline__ uint32_t scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  if (b == 0) return 127;
  const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)(e < 1 ? 1 : e);
}
__device__ __forceinline__ float exponent_value(uint32_t e) { return __uint_as_float(e << 23); }
// 1 / 2^(e - 127), exact: e is within [1, 247].
__device__ __forceinline__ float exponent_inverse(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// A scale that is a power of two, at least 2^-126, as itself; any other as NaN.
__device__ __forceinline__ float power_of_two(float s) {
  const uint32_t b = __float_as_uint(s), e = b >> 23;
  return (b & 0x7fffffu) == 0 && e - 1u < 254u ? s : CUDART_NAN_F;
}
// The same as an exponent byte (E8M0, whose 255 is NaN) in all four bytes.
__device__ __forceinline__ uint32_t exponent_bytes(float s) {
  const uint32_t b = __float_as_uint(s), e = b >> 23;
  return ((b & 0x7fffffu) == 0 && e - 1u < 254u ? e : 255u) * 0x01010101u;
}

// Two 32-bit operations as one instruction: c += (a, b) * w.
__device__ __forceinline__ void fma2(uint64_t& c, uint32_t a, uint32_t b, uint64_t w) {
  asm("{ .reg .b64 v; mov.b64 v, {%1, %2}; fma.rn.f32x2 %0, v, %3, %0; }" : "+l"(c) : "r"(a), "r"(b), "l"(w));
}
// c += (a, b) * v * w, in this order.
__device__ __forceinline__ void mul_fma2(uint64_t& c, uint32_t a, uint32_t b, uint64_t v, uint64_t w) {
  asm("{ .reg .b64 t; mov.b64 t, {%1, %2}; mul.rn.f32x2 t, t, %3; fma.rn.f32x2 %0, t, %4, %0; }"
      : "+l"(c)
      : "r"(a), "r"(b), "l"(v), "l"(w));
}
__device__ __forceinline__ uint64_t twice(float v) {
  const uint32_t b = __float_as_uint(v);
  return ((uint64_t)b << 32) | b;
}

// Neither zero, subnormal, infinite nor NaN.
__device__ __forceinline__ bool normal(float v) { return (__float_as_uint(v) & 0x7fffffffu) - 0x800000u < 0x7f000000u; }

// A block's two scales may have a product that fp32 does not hold where it
// holds the result.  So the block's sum v, a multiple of 2^-18 below 2^25, is
// multiplied by one scale w and then, in the multiply-add, by the other, x: v w
// stays a normal number for w within 2^-100 and 2^100.  Outside, w leaves a
// power of two to x.  Returns it, 1 within.  No branches: this stands in every
// block's way.
__device__ __forceinline__ float leave_power(float& w) {
  const float m = fabsf(w);
  const bool high = m > 0x1p100f, low = m < 0x1p-100f;
  w *= high ? 0x1p-27f : low ? 0x1p49f : 1.0f;
  return high ? 0x1p27f : low ? 0x1p-49f : 1.0f;
}
// x takes it.  Past fp32 the largest number does: v w x is past it too, or v is 0.
__device__ __forceinline__ float take_power(float x, float power) {
  const float r = x * power;
  return fabsf(x) < CUDART_INF_F ? fminf(fmaxf(r, -0x1.fffffep127f), 0x1.fffffep127f) : r;
}

// A block's largest magnitude is taken with fmaxf, which passes over NaN.  If
// it is infinite, infinities are made NaN (which is what their codes are)
// and the maximum is taken again: so finite blocks pay for no checks.
__device__ __forceinline__ float no_infinity(float v) { return fabsf(v) < CUDART_INF_F ? v : CUDART_NAN_F; }

// Two scaled values to e4m3, to nearest even, NaN to NaN.
__device__ __forceinline__ uint16_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  return (uint32_t)pack_e4m3(a, b) | ((uint32_t)pack_e4m3(c, d) << 16);
}

// Two e4m3 codes to float (exact: every e4m3 value is an f16 value).
__device__ __forceinline__ float2 e4m3_values(uint16_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  float2 f;
  asm("{ .reg .f16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h; }"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// sigmoid(v) from e = exp(-|v|): 1 or e over 1 + e.  exp(-v) itself passes
// 2^126 at v = -87.3, where __fdividef gives 0, and then fp32's range, both while
// e is still a normal number.
struct Sigmoid {
  float over, under;
};
__device__ __forceinline__ Sigmoid sigmoid(float v) {
  const float e = __expf(-fabsf(v));
  return Sigmoid{v < 0.0f ? e : 1.0f, 1.0f + e};
}

// The tanh form of GELU is g * sigmoid(2 z), z = sqrt(2/pi) (g + 0.044715 g^3),
// since 0.5 (1 + tanh z) = sigmoid(2 z).  Past |g| = 64 the sigmoid is 0 or 1
// in 32 bits; the clamp keeps the cube and the square there finite.
__device__ __forceinline__ float gelu_clamp(float g) { return fminf(fmaxf(g, -64.0f), 64.0f); }
__device__ __forceinline__ float gelu_sigmoid(float c) {
  const Sigmoid s = sigmoid(2.0f * 0.7978845608028654f * (c + 0.044715f * c * c * c));
  return __fdividef(s.over, s.under);
}

// Gate activations, in 32 bits.
template <int ACT>
__device__ __forceinline__ float activation(float g) {
  if (ACT == TIDE_ACT_SILU) {
    const Sigmoid s = sigmoid(g);
    return __fdividef(g * s.over, s.under);
  }
  return g * gelu_sigmoid(gelu_clamp(g));
}

// act(g) and its derivative.
template <int ACT>
__device__ __forceinline__ float2 activation_grad(float g) {
  if (ACT == TIDE_ACT_SILU) {
    const Sigmoid q = sigmoid(g);
    const float s = __fdividef(q.over, q.under);
    return make_float2(g * s, s * (1.0f + g * (1.0f - s)));
  }
  const float c = gelu_clamp(g);
  const float s = gelu_sigmoid(c);
  const float dz = 0.7978845608028654f * (1.0f + 3.0f * 0.044715f * c * c);
  // 2 g alone may pass fp32's range; its factors are 0 long before
  return make_float2(g * s, s + 2.0f * (g * (s * (1.0f - s) * dz)));
}

}  // namespace tide
