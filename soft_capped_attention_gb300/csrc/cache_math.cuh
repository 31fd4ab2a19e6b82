// The caps in fp32 for the calls whose fp32 results (a log-sum-exp, summed
// weights) are read as numbers: each form keeps its relative accuracy near zero,
// where an absolute error of the cap would become a relative error of exp(t).
//
//   tanh      : cap tanh(s / cap)
//   soft_sign : s / (1 + |s| / cap)
//   alsc      : out (sigma(d + ab) - sigma(ab)), d = alpha s / cap.  With
//               E = e^{-|d|} - 1 the difference of the two sigmoids is
//                 d >= 0 : -E (1 - sb) / (1 + e^{-ab} (1 + E))
//                 d <  0 :  E sb       / (1 + e^{ab}  (1 + E))
//               (sb = sigma(ab)), without the cancellation of the two
//               sigmoids: subtracting them costs up to 1e-5 of the score.
#pragma once

#include "cache_internal.h"

namespace capattn {

template <int METHOD>
__device__ __forceinline__ float exact_cap(float s, const ExactCap& k) {
  if constexpr (METHOD == CAPATTN_CAP_TANH) {
    return k.cap * tanhf(s * k.inv_cap);
  } else if constexpr (METHOD == CAPATTN_CAP_SOFT_SIGN) {
    return s / (1.0f + fabsf(s) * k.inv_cap);
  } else if constexpr (METHOD == CAPATTN_CAP_ALSC) {
    const float d = s * k.a;
    const float e = expm1f(-fabsf(d));
    const bool up = d >= 0.f;
    const float num = up ? -k.one_minus_sb : k.sb;
    const float den = up ? k.emb : k.eb;
    return k.out * (e * num / fmaf(den, 1.0f + e, 1.0f));
  } else {
    return s;
  }
}

}  // namespace capattn
