#pragma once
#include <cstdint>

namespace w4a8 {

// Codes of four values in units of the scale, |v * inv| < 2^21: rint of the
// exact product (ties to even) by one fused multiply-add into the unit range of
// 1.5 * 2^23, whose low byte is then the code.
__device__ __forceinline__ uint32_t pack_codes(const float* v, float inv) {
  constexpr float kMagic = 12582912.0f;
  const uint32_t c0 = __float_as_uint(fmaf(v[0], inv, kMagic)), c1 = __float_as_uint(fmaf(v[1], inv, kMagic));
  const uint32_t c2 = __float_as_uint(fmaf(v[2], inv, kMagic)), c3 = __float_as_uint(fmaf(v[3], inv, kMagic));
  return __byte_perm(__byte_perm(c0, c1, 0x0040), __byte_perm(c2, c3, 0x0040), 0x5410);
}

// x / s for r = 1 / s (IEEE): the product by the reciprocal, corrected by its
// remainder (Markstein 1990, "Computation of elementary functions on the IBM
// RISC System/6000 processor"). A quotient midway between two codes comes out
// as that, and goes to the even one; x * r alone lands on either side. (r = 0
// gives 0.)
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, s, x), r, q);
}

}  // namespace w4a8
