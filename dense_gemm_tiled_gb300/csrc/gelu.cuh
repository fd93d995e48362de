#pragma once
// The gelu x Phi(x) and its derivative Phi(x) + x phi(x) of one or two fp32
// values, for results in 16 bits and in 32 (the microscaled storage's elementwise
// kernels and the fused products' epilogues).
#include "mx_format.cuh"

namespace gb300 {
namespace {

// 16-bit types.  For a pair x, given as n = -|x|: c = erfc(|x| / sqrt 2) / 2 =
// Phi(-|x|) and e = exp(-x^2 / 2), which the gelu and its derivative share:
//   erfc(z) = t (a1 + t (a2 + ... )) exp(-z^2),  t = 1 / (1 + p z),
// within 1.5e-7 (M. Abramowitz and I. Stegun, "Handbook of Mathematical
// Functions", 7.1.26), which the rounding to 16 bits covers but in the far tail:
// 0.3 % of gelu(-5.7) = -3e-8, 1.2 % of gelu(-8.5) = -8e-17.  A value costs an
// exponential, a reciprocal and five paired operations; with erff and expf, the
// forward and backward pass at 16384 x 5632 bf16 took 465 us against 232 with
// scalar operations of this form.
__device__ __forceinline__ f32x2 normal_tail2_over_e(f32x2 n, f32x2& e) {  // c / e
  float a, b;
  unpair(fma2(n, pair(-0.3275911f * 0.70710678f), pair(1.f)), a, b);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
  const f32x2 t = pair(a, b);
  unpair(mul2(mul2(n, n), pair(-0.72134752f)), a, b);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
  e = pair(a, b);
  f32x2 c = fma2(t, pair(0.5f * 1.061405429f), pair(0.5f * -1.453152027f));
  c = fma2(t, c, pair(0.5f * 1.421413741f));
  c = fma2(t, c, pair(0.5f * -0.284496736f));
  c = fma2(t, c, pair(0.5f * 0.254829592f));
  return mul2(t, c);
}
__device__ __forceinline__ f32x2 normal_tail2(f32x2 n, f32x2& e) {
  const f32x2 c = normal_tail2_over_e(n, e);
  return mul2(c, e);
}
// -|x|, not below -64 (where c and e are 0 already), so that an infinity meets no
// 0; a NaN stays one
__device__ __forceinline__ float minus_abs(float x) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(-fabsf(x)), "f"(-64.f));
  return r;
}

// v -> act(v) (0 none, 1 relu: v where v > 0, else 0, 2 gelu).  The gelu as max(x, 0) -
// |x| Phi(-|x|): for 16-bit results from the form above, for fp32 ones from normcdff,
// within a few ulp in both tails.
template <typename T, int N>
__device__ __forceinline__ void act_of(float (&v)[N], int act) {
  if (act == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = v[i] > 0.f ? v[i] : 0.f;
  } else if (act == 2) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float m0 = v[i] > 0.f ? v[i] : 0.f, m1 = v[i + 1] > 0.f ? v[i + 1] : 0.f;
      if constexpr (sizeof(T) == 4) {
        const float n0 = minus_abs(v[i]), n1 = minus_abs(v[i + 1]);
        v[i] = __fmaf_rn(n0, normcdff(n0), m0);
        v[i + 1] = __fmaf_rn(n1, normcdff(n1), m1);
      } else {
        const f32x2 n = pair(minus_abs(v[i]), minus_abs(v[i + 1]));
        f32x2 e;
        const f32x2 c = normal_tail2(n, e);
        unpair(fma2(n, c, pair(m0, m1)), v[i], v[i + 1]);
      }
    }
  }
}

// d *= act'(x).  relu: d where x > 0, else 0 (whatever d is); gelu: h = Phi(-|x|) -
// |x| phi(x) where x < 0, else 1 - h.
template <typename T, int N>
__device__ __forceinline__ void slope_of(float (&d)[N], const float (&x)[N], int act) {
  if (act == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = x[i] > 0.f ? d[i] : 0.f;
  } else if (act == 2) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = i; k < i + 2; ++k) {
          const float n = minus_abs(x[k]);
          const float h = __fmaf_rn(n * 0.39894228f, expf(-0.5f * n * n), normcdff(n));
          d[k] *= x[k] < 0.f ? h : 1.f - h;
        }
      } else {
        const f32x2 n = pair(minus_abs(x[i]), minus_abs(x[i + 1]));
        f32x2 e;
        const f32x2 c = normal_tail2_over_e(n, e);
        const f32x2 h = mul2(fma2(n, pair(0.39894228f), c), e);
        float h0, h1, g0, g1;
        unpair(h, h0, h1);
        unpair(fma2(h, pair(-1.f), pair(1.f)), g0, g1);
        unpair(mul2(pair(d[i], d[i + 1]), pair(x[i] < 0.f ? h0 : g0, x[i + 1] < 0.f ? h1 : g1)), d[i],
               d[i + 1]);
      }
    }
  }
}

}  // namespace
}  // namespace gb300
