// A polynomial of the soft-sign cap near zero, fitted on the host (plain C++).
#pragma once

#include <math.h>

namespace capattn {

// s / (1 + |s| / cap) = X (c0 + |X| (c1 + |X| (c2 + .. + |X| c6))), s = sm_scale X, for
// w = |s| / cap <= kNearSoftSign: 1 / (1 + w) interpolated at the seven Chebyshev nodes of
// [0, kNearSoftSign], then with both scales folded in.  Relative error 2.2e-8 (the pole at
// w = -1 lies 6.7 half-ranges from the middle: a factor of 13 a term).
constexpr double kNearSoftSign = 0.35;
inline void near_soft_sign_fit(double cap, double sm_scale, float c[7]) {
  const double pi = 3.14159265358979323846, half = 0.5 * kNearSoftSign;
  double w[7], d[7], a[7] = {0, 0, 0, 0, 0, 0, 0};
  for (int i = 0; i < 7; ++i) {
    w[i] = half * (1.0 + cos((2 * i + 1) * pi / 14.0));
    d[i] = 1.0 / (1.0 + w[i]);
  }
  // Newton's divided differences, then multiplied out from the last node on
  for (int k = 1; k < 7; ++k)
    for (int i = 6; i >= k; --i) d[i] = (d[i] - d[i - 1]) / (w[i] - w[i - k]);
  for (int i = 6; i >= 0; --i) {
    for (int j = 6; j > 0; --j) a[j] = a[j - 1] - w[i] * a[j];
    a[0] = d[i] - w[i] * a[0];
  }
  double s = sm_scale;
  for (int i = 0; i < 7; ++i, s *= fabs(sm_scale) / cap) c[i] = (float)(a[i] * s);
}

}  // namespace capattn
