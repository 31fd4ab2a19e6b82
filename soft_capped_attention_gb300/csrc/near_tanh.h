// Three terms of tanh near zero, fitted on the host (plain C++).
#pragma once

#include <math.h>

namespace capattn {

// tanh(u) = u (a0 + a1 w + a2 w^2), w = u^2, for |u| <= kNearTanh: tanh(u) / u
// interpolated at the three Chebyshev nodes of w in [0, kNearTanh^2], then with both
// scales folded in: cap tanh(in X) = X (c0 + z (c1 + z c2)), z = X^2.  Relative error
// 1.9e-8, below the five terms' 2.7e-8 (it grows with the range's sixth power: 1.05e-7
// for |u| <= 0.2, a step of fp32 more than either).
constexpr double kNearTanh = 0.15;
inline void near_tanh_fit(double cap, double in, float c[3]) {
  const double pi = 3.14159265358979323846, half = 0.5 * kNearTanh * kNearTanh;
  double w[3], f[3];
  for (int i = 0; i < 3; ++i) {
    w[i] = half * (1.0 + cos((2 * i + 1) * pi / 6.0));
    f[i] = tanh(sqrt(w[i])) / sqrt(w[i]);
  }
  // Newton's divided differences, multiplied out
  const double d01 = (f[1] - f[0]) / (w[1] - w[0]), d12 = (f[2] - f[1]) / (w[2] - w[1]);
  const double d012 = (d12 - d01) / (w[2] - w[0]);
  const double a[3] = {f[0] - d01 * w[0] + d012 * w[0] * w[1], d01 - d012 * (w[0] + w[1]), d012};
  double s = cap * in;
  for (int i = 0; i < 3; ++i, s *= in * in) c[i] = (float)(a[i] * s);
}

}  // namespace capattn
