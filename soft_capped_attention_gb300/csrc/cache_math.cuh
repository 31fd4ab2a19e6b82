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

// 32 lanes x 32 bits, 32 consecutive columns per thread, and the largest |x| of them
// (NaN apart) by the same load.
__device__ __forceinline__ float tmem_ld32_absmax(uint32_t taddr, uint32_t (&r)[32]) {
  float top;
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.abs.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(top)
      : "r"(taddr)
      : "memory");
  return top;
}

}  // namespace capattn
