// int8 codes of rows: s = max|x| / 127 (float32, IEEE division), q = x / s to the
// nearest whole number, ties to even, within [-127, 127]. A row of zeros has s = 0 and
// q = 0; a row with an infinity or a NaN has s = NaN and q = 0, so that every product
// of it is NaN.
#pragma once
#include "norm_rows.h"

namespace moe {

// max|x| travels as the bits of |x|, which order as the values do, with infinities and
// NaN above them: no value is dropped, as fmaxf drops NaN.
__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The largest |x| of eight values as float32 bits. 16-bit values are compared as they are
// stored, two at a time.
template <class T, bool F32>
__device__ __forceinline__ uint32_t amax8(const Row8<T, F32>& x, uint32_t m) {
  if constexpr (F32) {
    const uint32_t w[8] = {x.lo.x, x.lo.y, x.lo.z, x.lo.w, x.hi.x, x.hi.y, x.hi.z, x.hi.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_u32(m, w[i] & 0x7FFFFFFFu);
    return m;
  } else {
    typedef __attribute__((__vector_size__(2 * sizeof(uint16_t)))) uint16_t u16x2_t;
    auto mx = [](uint32_t a, uint32_t b) {
      return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a),
                                                                    __builtin_bit_cast(u16x2_t, b)));
    };
    const uint32_t w = mx(mx(x.lo.x & 0x7FFF7FFFu, x.lo.y & 0x7FFF7FFFu), mx(x.lo.z & 0x7FFF7FFFu, x.lo.w & 0x7FFF7FFFu));
    float a, b;
    unpack2<T>(max_u32(w & 0xFFFFu, w >> 16), a, b);
    return max_u32(m, __float_as_uint(a));
  }
}

struct RowScale {
  float s, r;   // the scale, and about 1 / s (0 where every code is 0, infinite where s is
                // subnormal and so far off amax / 127 that a code may pass 127)
};
__device__ __forceinline__ RowScale row_scale(uint32_t amax) {
  RowScale q;
  const bool finite = amax < 0x7F800000u;
  q.s = finite ? __uint_as_float(amax) / 127.0f : __uint_as_float(0x7FC00000u);
  q.r = !finite || q.s == 0.0f ? 0.0f
        : q.s < 1.17549435e-38f ? __uint_as_float(0x7F800000u)
                                : __builtin_amdgcn_rcpf(q.s);
  return q;
}
__device__ __forceinline__ float code_exact(float v, float s) {
  return __builtin_fminf(__builtin_fmaxf(rintf(v / s), -127.0f), 127.0f);
}
// Codes of eight values of one row. v r is within 2^-22 of the float32 quotient v / s,
// relative (r is off by 2^-23, the quotient rounds once, 2^-24; the fma does not round
// v r), so within 127 x 2^-22 < 3.1e-5 of it: where v r is further than that from the
// middle of two whole numbers, both round to the same one. That number is the low byte of
// v r + 1.5 x 2^23, whose last place is 1. Otherwise, for about one value in 16000, the
// eight are divided, at about ten instructions each instead of five.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const RowScale& s) {
  constexpr float kBig = 12582912.0f;
  uint32_t t[8];
  float off = 0.0f;   // the furthest from a whole number
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float b = __builtin_fmaf(v[i], s.r, kBig);
    off = __builtin_fmaxf(off, __builtin_fabsf(__builtin_fmaf(v[i], s.r, kBig - b)));
    t[i] = __float_as_uint(b);
  }
  if (s.r == 0.0f) return make_uint2(0, 0);   // uniform over a row: zeros, or no numbers
  if (!(off < 0.5f - 3.2e-5f) || __builtin_isinf(s.r)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = static_cast<uint32_t>(static_cast<int>(code_exact(v[i], s.s)));
  }
  auto pack = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {   // their low bytes
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0C0C0400u), __builtin_amdgcn_perm(b, a, 0x0C0C0400u),
                                 0x05040100u);
  };
  return make_uint2(pack(t[0], t[1], t[2], t[3]), pack(t[4], t[5], t[6], t[7]));
}

}  // namespace moe
