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
//
// Raw scores small against the cap (|s / cap| <= 1/2 for tanh, |d| <= 1/2 for
// alsc, which is where scores usually are) take a polynomial on the FMA pipe,
// two at a time, when a whole warp's scores are in its range; its relative error
// is about 1e-7.
#pragma once

#include "cache_internal.h"
#include "softmax_elem.cuh"

namespace capattn {

// cap(s), s = sm_scale X, with library functions.
template <int METHOD>
__device__ __forceinline__ float exact_cap(float s, const ExactCap& k) {
  if constexpr (METHOD == CAPATTN_CAP_TANH) {
    return k.cap * tanhf(s * k.inv_cap);
  } else if constexpr (METHOD == CAPATTN_CAP_SOFT_SIGN) {
    return s / (1.0f + fabsf(s) * k.inv_cap);
  } else if constexpr (METHOD == CAPATTN_CAP_ALSC) {
    const float d = s * k.alsc.a;
    const float e = expm1f(-fabsf(d));
    const bool up = d >= 0.f;
    const float num = up ? -k.alsc.one_minus_sb : k.alsc.sb;
    const float den = up ? k.alsc.emb : k.alsc.eb;
    return k.alsc.out * (e * num / fmaf(den, 1.0f + e, 1.0f));
  } else {
    return s;
  }
}

constexpr bool has_poly(int method) { return method == CAPATTN_CAP_TANH || method == CAPATTN_CAP_ALSC; }

// cap(sm_scale X) of two raw scores inside the polynomial's range.
template <int METHOD>
__device__ __forceinline__ F2 poly_cap2(F2 X, const ExactCap& k) {
  if constexpr (METHOD == CAPATTN_CAP_TANH) {
    const F2 z = f2_mul(X, X);
    F2 q = f2_fma(f2(k.poly[4], k.poly[4]), z, f2(k.poly[3], k.poly[3]));
    q = f2_fma(q, z, f2(k.poly[2], k.poly[2]));
    q = f2_fma(q, z, f2(k.poly[1], k.poly[1]));
    q = f2_fma(q, z, f2(k.poly[0], k.poly[0]));
    return f2_mul(X, q);
  } else {
    F2 q = f2_fma(f2(k.poly[6], k.poly[6]), X, f2(k.poly[5], k.poly[5]));
#pragma unroll
    for (int i = 4; i >= 0; --i) q = f2_fma(q, X, f2(k.poly[i], k.poly[i]));
    return f2_mul(X, q);
  }
}

// cap(sm_scale X) of one raw score of any size: near zero the polynomial, else
// exp2 and a reciprocal, which cancel nothing there.
template <int METHOD>
__device__ __forceinline__ float any_cap(float X, const ExactCap& k) {
  const float s = X * k.sm_scale;
  if constexpr (METHOD == CAPATTN_CAP_TANH || METHOD == CAPATTN_CAP_ALSC) {
    if (k.xmax == 0.f) return exact_cap<METHOD>(s, k);
    float near, unused, far;
    const float xc = fminf(fmaxf(X, -k.xmax), k.xmax);
    f2_split(poly_cap2<METHOD>(f2(xc, xc), k), near, unused);
    if constexpr (METHOD == CAPATTN_CAP_TANH) {
      const float e = ex2_approx(fabsf(s) * (k.inv_cap * 2.0f * kL2E));
      far = copysignf(k.cap * (1.0f - 2.0f * rcp_approx(1.0f + e)), s);
    } else {
      const float d = s * k.alsc.a;
      const float x = ex2_approx(-fabsf(d) * kL2E);
      const bool up = d >= 0.f;
      far = k.alsc.out * ((1.0f - x) * (up ? k.alsc.one_minus_sb : -k.alsc.sb)) * rcp_approx(fmaf(up ? k.alsc.emb : k.alsc.eb, x, 1.0f));
    }
    return fabsf(X) <= k.xmax ? near : far;
  } else if constexpr (METHOD == CAPATTN_CAP_SOFT_SIGN) {
    return s * rcp_approx(fmaf(fabsf(s), k.inv_cap, 1.0f));
  } else {
    return s;
  }
}

}  // namespace capattn
