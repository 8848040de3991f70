// Cosine and sine of an fp64 angle, for the rotary positions' tables.  Plain C++ (host and
// device); the host build is checked against 64-bit-mantissa arithmetic by tests/test_cos_sin.py.
#pragma once

#include <stdint.h>

#ifndef AWQ_HOST_DEVICE
#define AWQ_HOST_DEVICE __host__ __device__
#endif

namespace awq {

// x = n pi/2 + r, |r| <= pi/4 (a little more for |x| past 2^31), then the Taylor series of
// r: the first terms left out are r^17/17! and r^18/18!, 2^-53.8 of the sine and 2^-58 of the
// cosine at most.  With the roundings both are good to 2^-51 of themselves for |x| up to 2^31 (worst
// of 8 million found: 2^-52; with two terms fewer the sine had 2^-45), so
// one in 2^26 at most rounds to the other fp32 neighbour than the exact value does.
AWQ_HOST_DEVICE inline void cos_sin(double x, double &cosine, double &sine) {
  const double n = __builtin_rint(x * 0x1.45f306dc9c883p-1);          // 2/pi
  double r = __builtin_fma(-n, 0x1.921fb54442d18p0, x);                // pi/2 in two parts
  r = __builtin_fma(-n, 0x1.1a62633145c07p-54, r);
  const double r2 = r * r;
  double s = __builtin_fma(r2, -1.0 / 1307674368000.0, 1.0 / 6227020800.0);
  s = __builtin_fma(r2, s, -1.0 / 39916800.0);
  s = __builtin_fma(r2, s, 1.0 / 362880.0);
  s = __builtin_fma(r2, s, -1.0 / 5040.0);
  s = __builtin_fma(r2, s, 1.0 / 120.0);
  s = __builtin_fma(r2, s, -1.0 / 6.0);
  s = __builtin_fma(r * r2, s, r);
  double c = __builtin_fma(r2, 1.0 / 20922789888000.0, -1.0 / 87178291200.0);
  c = __builtin_fma(r2, c, 1.0 / 479001600.0);
  c = __builtin_fma(r2, c, -1.0 / 3628800.0);
  c = __builtin_fma(r2, c, 1.0 / 40320.0);
  c = __builtin_fma(r2, c, -1.0 / 720.0);
  c = __builtin_fma(r2, c, 1.0 / 24.0);
  c = __builtin_fma(r2, c, -0.5);
  c = __builtin_fma(r2, c, 1.0);
  const int quarter = (int)(int64_t)n & 3;
  const double a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
  cosine = quarter == 1 || quarter == 2 ? -a : a;
  sine = quarter & 2 ? -b : b;
}

}  // namespace awq
