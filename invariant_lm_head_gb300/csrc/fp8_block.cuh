// e4m3 values of a block under one fp32 scale, each rounded once.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace lmh {

// A block's quotient x * 448 / a in parts that stay clear of overflow and
// underflow: with a = am * 2^e (1 <= am < 2), c = 448 * 2^-e and r = 1 / am
// rounded to nearest, y = x * c is exact wherever q does not round to zero, and
// y / am is corrected from y * r by its exact remainder (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// IBM J. Res. Dev. 34(1), 1990). It is taken from -y and -r: a zero's remainder
// is +0 either way, and +0 * -r is the zero whose addition keeps the quotient's
// sign (-0 * 448 / a is -0).
struct BlockScale {
  float neg_c, am, neg_r, scale;
};

// A block that holds an infinity or a NaN (passed on in a): every q becomes NaN.
__device__ __forceinline__ BlockScale block_scale_nan(float a) {
  BlockScale s;
  s.scale = a;
  s.neg_c = 0.f;
  s.am = 1.f;
  s.neg_r = __uint_as_float(0x7fffffffu);
  return s;
}

// a: the largest |x|, a normal fp32 number.
__device__ __forceinline__ BlockScale block_scale(float a) {
  BlockScale s;
  const uint32_t ab = __float_as_uint(a);
  const int e = static_cast<int>(ab >> 23) - 127;
  const float am = __uint_as_float((ab & 0x007fffffu) | 0x3f800000u);
  s.neg_c = -448.f * __uint_as_float(static_cast<uint32_t>(127 - (e < 127 ? e : 126)) << 23);
  if (e == 127) s.neg_c *= 0.5f;
  s.am = am;
  s.neg_r = -__frcp_rn(am);
  s.scale = __fdiv_rn(a, 448.f);
  return s;
}

// Two quotients to a pair of e4m3 bytes (low half first).
__device__ __forceinline__ uint32_t quantize2(f32x2 x, const BlockScale& s) {
  const f32x2 neg_y = f2_mul(x, f2_pack(s.neg_c, s.neg_c));
  const f32x2 neg_r = f2_pack(s.neg_r, s.neg_r);
  const f32x2 q0 = f2_mul(neg_y, neg_r);
  const f32x2 neg_rem = f2_fma(q0, f2_pack(s.am, s.am), neg_y);
  float lo, hi;
  f2_unpack(f2_fma(neg_rem, neg_r, q0), lo, hi);
  uint16_t out;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(out) : "f"(hi), "f"(lo));
  return out;
}

}  // namespace lmh
