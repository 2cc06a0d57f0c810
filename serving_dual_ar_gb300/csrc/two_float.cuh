// Arithmetic on unevaluated sums of two floats (about 44 bits), for results that
// are rounded to few bits at once and must not depend on the order of a sum.
#pragma once

#include "s2_common.cuh"

namespace s2 {

// Unevaluated sums hi + lo of two floats (Dekker 1971; Knuth's two-sum).
S2_DEV Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
S2_DEV Two quick_two(float a, float b) {   // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
S2_DEV Two two_prod(float a, float b) {
  const float p = __fmul_rn(a, b);
  return {p, __fmaf_rn(a, b, -p)};
}
S2_DEV Two add(Two a, Two b) {
  Two s = two_sum(a.hi, b.hi);
  return quick_two(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
S2_DEV Two mul(Two a, float b) {
  const Two p = two_prod(a.hi, b);
  return {p.hi, __fmaf_rn(a.lo, b, p.lo)};
}
// hi + lo rounded to odd at 24 bits: rounding that to the few bits of e4m3
// gives what rounding hi + lo itself gives, also next to a tie.
S2_DEV float round_odd(Two a) {
  uint32_t u = __float_as_uint(a.hi);
  if (a.lo != 0.f && (u & 0x7f800000u) != 0x7f800000u) {
    if ((a.lo < 0.f) != (a.hi < 0.f)) --u;
    u |= 1u;
  }
  return __uint_as_float(u);
}

}  // namespace s2
