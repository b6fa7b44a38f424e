// int8 codes of rows: s = max|x| / 127 (float32, IEEE division), q = x / s to the
// nearest whole number, ties to even, within [-127, 127]. A row of zeros has s = 0 and
// q = 0; a row with an infinity or a NaN has s = NaN and q = 0, so that every product
// of it is NaN.
#pragma once
#include "mm.h"

namespace moe {

// max|x| travels as the bits of |x|, which order as the values do, with infinities and
// NaN above them: no value is dropped, as fmaxf drops NaN.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t amax8(const float (&v)[8], uint32_t m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_u32(m, abs_bits(v[i]));
  return m;
}
struct RowScale {
  float s, r;   // the scale, and 1 / s (0 where every code is 0, infinite where s is
                // subnormal and so far off amax / 127 that a code may pass 127)
};
__device__ __forceinline__ RowScale row_scale(uint32_t amax) {
  RowScale q;
  const bool finite = amax < 0x7F800000u;
  q.s = finite ? __uint_as_float(amax) / 127.0f : __uint_as_float(0x7FC00000u);
  q.r = !finite || q.s == 0.0f ? 0.0f
        : q.s < 1.17549435e-38f ? __uint_as_float(0x7F800000u)
                                : 1.0f / q.s;
  return q;
}
// The code of v. v r is within 2^-22 of the float32 quotient v / s, relative (r rounds
// once, the product once, the quotient once: 1.5 x 2^-23), so within 127 x 2^-22 < 3.1e-5
// of it: where it is further than that from the middle of two whole numbers, both round
// to the same one. Otherwise (and where r is infinite, so
// that v r is no number or infinite) `near` is set and the caller divides. A division takes about ten
// instructions, this takes three.
__device__ __forceinline__ float code_near(float v, float r, bool& near) {
  const float p = v * r, q = rintf(p);
  near |= !(__builtin_fabsf(p - q) < 0.5f - 3.2e-5f);
  return q;
}
__device__ __forceinline__ float code_exact(float v, float s) {
  return __builtin_fminf(__builtin_fmaxf(rintf(v / s), -127.0f), 127.0f);
}
__device__ __forceinline__ uint32_t pack_codes(float a, float b, float c, float d) {
  const uint32_t x = static_cast<uint32_t>(static_cast<int>(a)) & 0xFFu,
                 y = static_cast<uint32_t>(static_cast<int>(b)) & 0xFFu,
                 z = static_cast<uint32_t>(static_cast<int>(c)) & 0xFFu,
                 w = static_cast<uint32_t>(static_cast<int>(d));
  return x | (y << 8) | (z << 16) | (w << 24);
}
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const RowScale& s) {
  float q[8];
  bool near = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = code_near(v[i], s.r, near);
  if (s.r == 0.0f) {   // uniform over a row: zeros, or no numbers
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = 0.0f;
  } else if (near) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = code_exact(v[i], s.s);
  }
  return make_uint2(pack_codes(q[0], q[1], q[2], q[3]), pack_codes(q[4], q[5], q[6], q[7]));
}

}  // namespace moe
