// The scores of pkv_attention_scored, shared by its decode and prefill kernels:
// the tanh cap's forms and its parameters.
#pragma once

#include "pkv_device.cuh"

namespace pkv {
namespace dev {

// From the raw product s = q.K to a logit in log2 units: s * lin without a cap
// (lin = scale * log2(e)); with one, cap2 * tanh(x), x = s * k, k = scale /
// cap, cap2 = cap * log2(e).
struct ScoreParams {
  float lin, k, mul, cap2;  // mul = 2 log2(e) k
  bool cap;
};
__device__ __forceinline__ ScoreParams score_params(const AttnArgs& a) {
  ScoreParams p;
  p.cap = a.score.softcap > 0.f;
  p.lin = a.scale * kLog2e;
  p.k = p.cap ? a.scale / a.score.softcap : 0.f;
  p.mul = 2.f * kLog2e * p.k;
  p.cap2 = a.score.softcap * kLog2e;
  return p;
}

// The cap's forms.  Up to |x| = 1/2, s times a polynomial of degree 3 in s^2
// whose coefficients hold the powers of k, two values at a time: fitted to
// tanh(x) / x with constant term 1 for the smallest largest relative error
// (6.4e-7; 7.2e-7 as computed), relative so that a cap far above the logits
// leaves them their precision.  Past that the identity tanh(x) = 1 - 2 / (1 +
// e^(2x)): one exponential, whose overflow and underflow give +-1, and one
// reciprocal, an absolute error of about 2^-22 of the cap.  Where k is so small
// or large that a power of it or of s could leave fp32's range (a cap of a
// hundred thousand), capped_poly serves |x| <= 1: x times a degree-6 polynomial
// in x^2 of the same kind (5.5e-8; 1.6e-7 as computed).
struct CapForm {
  f32x2 a[4];   // pairs: formed at each use they cost two moves an operation
  float limit;  // largest s^2; -1: k not in range
};
__device__ __forceinline__ CapForm cap_form(const ScoreParams& sp) {
  CapForm c;
  const float k2 = sp.k * sp.k;
  const bool in_range = sp.k >= 0x1p-20f && sp.k <= 0x1p20f;
  const float a[4] = {sp.lin, sp.lin * -0.33328161f * k2, sp.lin * 0.13205360f * k2 * k2,
                      sp.lin * -0.04475065f * k2 * k2 * k2};
#pragma unroll
  for (int n = 0; n < 4; ++n) c.a[n] = pair(a[n], a[n]);
  c.limit = in_range ? 0.25f / k2 : -1.f;
  return c;
}
__device__ __forceinline__ float capped_poly(float s, const ScoreParams& p) {
  const float x = s * p.k, u = x * x;
  float c = fmaf(0.0010582346f, u, -0.0062592492f);
  c = fmaf(c, u, 0.0203596614f);
  c = fmaf(c, u, -0.0534986593f);
  c = fmaf(c, u, 0.1332640797f);
  c = fmaf(c, u, -0.3333298564f);
  return s * p.lin * fmaf(c, u, 1.f);
}
// s -> cap2 * tanh(x) + nm, by one form (0: the cubic, 1: exponential); the
// largest s^2 max'ed into big (form 0).
template <int kForm, int kN>
__device__ __forceinline__ void cap_values(float (&s)[kN], const ScoreParams& sp,
                                           const CapForm& cf, float nm, float& big) {
  if (kForm == 1) {
    const float c2 = sp.cap2 + nm;
#pragma unroll
    for (int i = 0; i < kN; ++i)
      s[i] = fmaf(-2.f * sp.cap2, fast_rcp(1.f + fast_exp2(s[i] * sp.mul)), c2);
    return;
  }
  const f32x2 nm2 = pair(nm, nm);
  float m0 = 0.f, m1 = 0.f;
#pragma unroll
  for (int i = 0; i < kN / 2; ++i) {
    const f32x2 v = pair(s[2 * i], s[2 * i + 1]), w = mul2(v, v);
    float w0, w1;
    split(w, w0, w1);
    if (i & 1) m1 = max3f(m1, w0, w1); else m0 = max3f(m0, w0, w1);
    const f32x2 q = fma2(fma2(fma2(w, cf.a[3], cf.a[2]), w, cf.a[1]), w, cf.a[0]);
    split(fma2(v, q, nm2), s[2 * i], s[2 * i + 1]);
  }
  big = max3f(big, m0, m1);
}

// Fixed-reference softmax.  A capped logit lies within +-cap2 (log2 units), and
// a row's own bias term at most max_bias above it.  With the reference cap2 / 2
// + max_bias, exp2(y - reference) is at most 2^(cap2 / 2), and at least 2^(-3/2
// cap2) for the key of that bias: inside fp32's and bf16's exponents for cap2 <=
// 80 (caps up to 55) with room for the sums.  No maximum is looked for then and
// nothing is rescaled.  (k: the cubic form's range.)
constexpr float kFixedCap2 = 80.f;
inline bool fixed_reference(const AttnArgs& a) {
  const float k = a.score.softcap > 0.f ? a.scale / a.score.softcap : 0.f;
  return a.score.softcap * kLog2e <= kFixedCap2 && k >= 0x1p-20f && k <= 0x1p20f;
}
// The largest -slope2 * |pos - j| over the keys first <= j <= last that a row at
// pos sees (its own among them).
__device__ __forceinline__ float max_bias(float slope2, int pos, int first, int last) {
  return -fminf(0.f, slope2) * (float)max(pos - first, last - pos);
}

}  // namespace dev
}  // namespace pkv
