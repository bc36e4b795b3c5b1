// Score modifiers of the *_mod entry points: softcap, distance bias and first
// visible keys.  Scores live in the exp2 domain (natural score x log2 e), so
//     capped:  c log2e tanh(s / c)          (s = raw * scale, c the cap)
//     biased:  - slope_h log2e |p - t|
#pragma once

#include <cfloat>
#include <cmath>

#include "common.cuh"

namespace pkv {

constexpr float kLog2e = 1.4426950408889634f;

// Device-side form of the modifiers (host constants folded once per call).
struct ScoreMod {
  float cap_log2 = 0.f;        // c log2e (0: no cap)
  float raw_to_x = 0.f;        // raw score -> s / c, the argument of tanh
  const float* slopes = nullptr;     // [num_q_heads], natural units
  const int32_t* first_keys = nullptr;   // decode: [batch]; prefill: [total_q]
  const int32_t* prefix_lens = nullptr;  // prefill only: [batch]
};

// `raw_scale` takes a raw q . k to the natural score (scale, and an FP8 cache's K scale).
inline ScoreMod make_score_mod(float raw_scale, float softcap, const float* slopes, const int32_t* first_keys,
                               const int32_t* prefix_lens) {
  ScoreMod m;
  if (softcap > 0.f) {
    m.cap_log2 = softcap * kLog2e;
    m.raw_to_x = fmaxf(fminf(raw_scale / softcap, FLT_MAX), -FLT_MAX);
  }
  m.slopes = slopes;
  m.first_keys = first_keys;
  m.prefix_lens = prefix_lens;
  return m;
}

// 0 or in [1e-30, 1e30], where c log2e and scale / c stay inside fp32 (a NaN fails both).
inline bool softcap_valid(float softcap) { return softcap == 0.f || (softcap >= 1e-30f && softcap <= 1e30f); }

// Scales at which a distance bias may be held in raw score units, slope / scale
// per key (one operation per score less than after scaling): far enough from
// fp32's ends that slope / scale times a distance below 2^31 stays inside for
// slopes below 2^33.  At 1e-37 a slope of 0.5 left it from 68 keys of distance on.
inline bool raw_bias_scale(float scale) { return scale >= 0x1p-64f && scale <= 0x1p64f; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(x) = 1 - 2 / (1 + e^2x), whose error is absolute, about 2^-22.  Overflow
// of e^2x gives 1, underflow -1, a NaN stays one.
__device__ __forceinline__ float tanh_by_exp_abs(float x) {
  return 1.f - __fdividef(2.f, 1.f + ex2(x * (2.f * kLog2e)));
}

// The same with the first four terms of the series below 1/4, so that the error
// is relative (1.2e-6) and a large cap costs no accuracy.
__device__ __forceinline__ float tanh_by_exp(float x) {
  const float y = x * x;
  const float series = x * fmaf(y, fmaf(y, fmaf(y, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
  return fabsf(x) < 0.25f ? series : tanh_by_exp_abs(x);
}

// Caps (x log2 e) up to which the absolute error will do: 2^-22 of it is 1.2e-4.
constexpr float kAbsCapLog2 = 512.f;

}  // namespace pkv
