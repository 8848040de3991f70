// Host build of the rotary positions' cosine and sine (cos_sin.h) against the C library's of
// 64-bit mantissas: prints the largest errors, relative to the value or, where that is smaller,
// to 2^-25 (below it the angle's own reduction counts, absolutely).  Built and run by
// tests/test_cos_sin.py.
#include <cmath>
#include <cstdio>
#include <random>
#define AWQ_HOST_DEVICE
#include "cos_sin.h"
int main() {
  static_assert(sizeof(long double) > 8, "a mantissa of 64 bits");
  const double half_pi = 1.5707963267948966;
  std::mt19937_64 rng(1);
  std::uniform_real_distribution<double> u(0.0, 1.0);
  long double worst[2] = {0, 0};
  double at[2] = {0, 0};
  auto look = [&](double x) {
    double c, s;
    awq::cos_sin(x, c, s);
    const long double want[2] = {cosl(x), sinl(x)}, got[2] = {c, s};
    for (int i = 0; i < 2; ++i) {
      const long double e = fabsl(got[i] - want[i]) / fmaxl(fabsl(want[i]), 0x1p-25L);
      if (e > worst[i]) worst[i] = e, at[i] = x;
    }
  };
  look(0.0);
  for (int i = 0; i < 2000000; ++i) {
    const double sign = i & 1 ? -1.0 : 1.0;
    look(sign * std::exp2(u(rng) * 61 - 30));                                       // any size up to 2^31
    look(sign * (double)(int64_t)(u(rng) * 2147483648.0) * std::exp2(-14 * u(rng)));  // a position times a frequency
    look(sign * ((int)(u(rng) * 1e6) + 0.5 + 1e-6 * u(rng)) * half_pi);              // the reduction's ends
    look((double)(int)(u(rng) * 1e9) * half_pi);                                     // near zeros
  }
  for (int r = 0; r < 200000; ++r) look(half_pi / 2 * (r - 100000) / 100000.0);
  std::printf("%.6Lg %.17g\n%.6Lg %.17g\n", worst[0], at[0], worst[1], at[1]);
  return 0;
}
