// The scores of pkv_attention_scored, shared by its decode and prefill kernels:
// the tanh cap's forms and the fixed reference.
#pragma once

#include "pkv_device.cuh"

namespace pkv {
namespace dev {

// From the raw product s = q.K to a logit in log2 units: s * lin without a cap
// (lin = scale * log2(e)); with one, cap2 * tanh(x), x = s * k, k = scale /
// cap, cap2 = cap * log2(e), in one of these forms:
//   kDeg2, kDeg3: for |x| up to 1/4, 1/2, s times a polynomial in s^2 whose
//     coefficients hold the powers of k, two values at a time: fitted to
//     tanh(x) / x with constant term 1 for the smallest largest relative error
//     (5.5e-7 and 7.2e-7 as computed), relative so that a cap far above the
//     logits leaves them their precision;
//   kExp: the identity tanh(x) = 1 - 2 / (1 + e^(2x)): one exponential, whose
//     overflow and underflow give +-1, and one reciprocal, an absolute error of
//     about 2^-22 of the cap.
// Where k is so small or large that a power of it or of s could leave fp32's
// range (a cap of a hundred thousand; limits -1), capped_poly serves |x| <= 1: x
// times a degree-6 polynomial in x^2 of the same kind (1.6e-7 as computed).
enum Form { kDeg2, kDeg3, kExp };
__device__ __forceinline__ float capped_poly(float s, const ScoreArgs& p) {
  const float x = s * p.k, u = x * x;
  float c = fmaf(0.0010582346f, u, -0.0062592492f);
  c = fmaf(c, u, 0.0203596614f);
  c = fmaf(c, u, -0.0534986593f);
  c = fmaf(c, u, 0.1332640797f);
  c = fmaf(c, u, -0.3333298564f);
  return s * p.lin * fmaf(c, u, 1.f);
}
// s -> cap2 * tanh(x) + nm by one form; the largest s^2 max'ed into big (not
// kExp).
template <Form kForm, int kN>
__device__ __forceinline__ void cap_values(float (&s)[kN], const ScoreArgs& sp, float nm,
                                           float& big) {
  if (kForm == kExp) {
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
    const f32x2 q = kForm == kDeg2
                        ? fma2(fma2(w, sp.deg2[2], sp.deg2[1]), w, sp.deg2[0])
                        : fma2(fma2(fma2(w, sp.deg3[3], sp.deg3[2]), w, sp.deg3[1]), w,
                               sp.deg3[0]);
    split(fma2(v, q, nm2), s[2 * i], s[2 * i + 1]);
  }
  big = max3f(big, m0, m1);
}

// Fixed-reference softmax.  A capped logit lies within +-cap2 (log2 units), and
// the bias is counted from the row's visible key that has the most of it (see
// bias_from), where it is zero.  The weight exp2 of the sum is then between
// 2^-cap2 and 2^cap2 at that key and lower at the others, so that no maximum is
// looked for and nothing is rescaled.  What cap2 <= 80 (caps up to 55) leaves of
// fp32's exponents (bf16 has the same):
//   below: a row's largest weight is at least 2^-80, and exp2 flushes below
//     2^-126, so that a key further along the bias counts down to 2^-46 of it
//     (2^19 keys less than that are 2^-27 of the sum), and the products of the
//     largest with V keep all their bits for |V| >= 2^-46;
//   above: a sum of 2^19 weights of 2^80 is 2^99: |V| up to 2^28.
// (With half of cap2 more, the weights begin at 2^-120: at cap 55.4, with scores
// at the cap's lower end, a bias loses all beyond six binades, 1.4% of a row's
// weight at a slope of 0.02, and an output of V around 2^-30 is 78% off.)
constexpr float kFixedCap2 = 80.f;
inline bool fixed_reference(const ScoredArgs& a) {
  return a.score.softcap > 0.f && a.score.cap2 <= kFixedCap2 && a.score.limit3 > 0.f;
}
// The distance that the bias of a row at pos is counted from, -slope2 * (|pos -
// j| - from): its own (0), or, with a bias that grows with distance, the farthest
// of the keys first .. last that it sees.  Distances are whole numbers below
// 2^20, so that their difference is exact and the bias never positive, however
// steep the slope (a bias and its largest value, rounded one by one, are 2^12
// apart at a slope of 10^8).
__device__ __forceinline__ float bias_from(float slope2, int pos, int first, int last) {
  return slope2 < 0.f ? (float)max(pos - first, last - pos) : 0.f;
}

// Whether a scored call's prefill items are single query heads: where even so
// they leave a quarter of the SMs idle, two heads of an item would only wait
// for each other.  (One prompt, us a call, single and in pairs, at 1/4, 3/4, 1 and
// 1 1/2 items an SM; without a cap and with a bias within 1 us of these:
//   16 heads over 2, cap 50:  14.8 16.9 | 22.4 25.0 | 28.4 29.4 | 44.4 37.6
//   32 over 8:                13.2 15.1 | 16.7 19.0 | 20.4 21.2 | 30.1 25.6
//   64 over 8:                12.7 14.3 | 14.1 16.2 | 17.8 17.5 | 21.1 19.4
//   32 over 1:                13.4 15.5 | 16.7 19.2 | 20.3 21.6 | 29.8 25.6.)
__device__ __forceinline__ bool single_head_items(const AttnArgs& a, int n_pre, int sms) {
  return (long long)n_pre * a.hq * 4 <= 3LL * sms;
}

}  // namespace dev
}  // namespace pkv
