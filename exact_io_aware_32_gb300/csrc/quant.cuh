// Values to E4M3 codes of value / factor, as the stores into an 8-bit cache make them.
#pragma once
#include <cstdint>

namespace fa {

// x / f for an E4M3 code, rounded once: the quotient rounded to odd (24 bits, the
// last one set when something was cut off) rounds to the code's 4 bits as the
// exact quotient would, ties among them. q = x / f to within one last place by
// one correction of x * (1 / f); the remainder x - q f is exact and its sign
// says on which side of q the quotient lies: an odd neighbour of q (or q, if
// odd) on that side has no tie between it and the quotient.
__device__ __forceinline__ float quotient_odd(float x, float f, float inv) {
  const float q0 = x * inv;
  const float q = fmaf(fmaf(-q0, f, x), inv, q0);
  const float r = fmaf(-q, f, x);
  const uint32_t b = __float_as_uint(q);
  const uint32_t odd = (b - ((b ^ __float_as_uint(r)) >> 31)) | 1u;  // towards zero when r's sign is the other one
  const float y = r != 0.f ? __uint_as_float(odd) : q;
  return fabsf(q0) < 512.f ? y : q0;  // past the largest code, infinite or NaN: as it is
}

// Four values to E4M3 codes, nearest even, +-448 beyond, NaN for NaN.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
      " mov.b32 %0, {lo, hi};\n}\n"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Factors far from 1, where the remainder or 1 / f would leave the normal range: f and the values are first multiplied by
// a power of two, 2^120 or 2^-110. f, subnormal or not, stays exact so. A value that overflows is 2^100 factors or more,
// the largest code; one that is rounded is below 2^-100 factors, code zero.
struct Factor {
  float f, inv, scale;
};
__device__ __forceinline__ Factor factor_of(float f) {
  const float scale = f <= 0x1p-100f ? 0x1p120f : f >= 0x1p100f ? 0x1p-110f : 1.0f;
  return {f * scale, 1.0f / (f * scale), scale};
}

// Four bf16 values as codes, each quotient rounded to odd first.
static __device__ __noinline__ uint32_t quantise4_exact(uint32_t lo, uint32_t hi, float f, float inv, float scale) {
  float x[4] = {__uint_as_float(lo << 16), __uint_as_float(lo & 0xffff0000u), __uint_as_float(hi << 16),
                __uint_as_float(hi & 0xffff0000u)};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = quotient_odd(x[i] * scale, f, inv);
  return e4m3x4(x[0], x[1], x[2], x[3]);
}

// The same. x * (1 / f) is within two last places of the quotient, so its code is the quotient's unless a tie of two
// codes lies that near: the 20 bits that a normal code drops within two of 0x80000. Those, and values below the normal
// codes, whose ties lie elsewhere, go the exact way. (All values that way: 27 us for 15523 tokens of 8 heads of 128,
// bound by its 14 instructions a value; a correctly truncated division for each: 58 us.)
__device__ __forceinline__ uint32_t quantise4(uint32_t lo, uint32_t hi, const Factor& s) {
  const float x[4] = {__uint_as_float(lo << 16), __uint_as_float(lo & 0xffff0000u), __uint_as_float(hi << 16),
                      __uint_as_float(hi & 0xffff0000u)};
  float q[4];
  bool exact = s.scale != 1.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[i] = x[i] * s.inv;
    exact |= ((__float_as_uint(q[i]) - 0x7FFFEu) & 0xFFFFFu) <= 4u || fabsf(q[i]) < 0x1p-6f;
  }
  return exact ? quantise4_exact(lo, hi, s.f, s.inv, s.scale) : e4m3x4(q[0], q[1], q[2], q[3]);
}

}  // namespace fa
