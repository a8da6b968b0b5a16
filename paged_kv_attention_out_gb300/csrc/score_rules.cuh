// score_rules.cuh - what a score goes through between Q K^T and the softmax in
// the calls with score rules (decode and extend): a soft cap, a bias linear in
// the distance, and which keys a query sees.
#pragma once

#include <math.h>
#include <stdint.h>

#include "pkv_common.cuh"

namespace pkv {

// Bits of a kernel's compile-time rules: kRuleRanges (visible keys follow a
// window and a prefix) is set in every kernel with rules.
constexpr int kRuleRanges = 1;
constexpr int kRuleCap = 2;
constexpr int kRuleBias = 4;

// tanh on |x| <= kTanhPoly as an odd polynomial of degree nine, fitted here
// (iteratively reweighted least squares on Chebyshev nodes) with the linear
// coefficient held at one: relative error 1.2e-7, 1.9e-7 evaluated in fp32.
constexpr float kTanhPoly = 0.625f;
constexpr float kTanh3 = -0.3333234190940857f;
constexpr float kTanh5 = 0.13308174908161163f;
constexpr float kTanh7 = -0.051947902888059616f;
constexpr float kTanh9 = 0.015195372514426708f;

// The same on |x| <= kTanhNear with degree five (relative error 4.9e-7): the
// prefill softmax uses it for tiles whose every score is that near zero.
constexpr float kTanhNear = 0.25f;
constexpr double kTanhNear3 = -0.33324571;
constexpr double kTanhNear5 = 0.12876421;

__device__ __forceinline__ float rule_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rule_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh x = 1 - 2 / (1 + e^2x), or the polynomial near zero, where that form
// would cancel: relative error below 2^-20 everywhere, so a cap of any size
// keeps the scores' own precision.
__device__ __forceinline__ float rule_tanh_far(float x) {
  return 1.f - 2.f * rule_rcp(1.f + rule_exp2(x * (2.f * kLog2e)));
}

__device__ __forceinline__ float rule_tanh(float x) {
  const float u = x * x;
  const float p = fmaf(fmaf(fmaf(kTanh9, u, kTanh7), u, kTanh5), u, kTanh3);
  const float near = fmaf(x * u, p, x);
  return fabsf(x) <= kTanhPoly ? near : rule_tanh_far(x);
}

// `near` also bounds the capped score itself (kNearLog2, log2 units): the
// prefill softmax takes a bound of a row's scores for their maximum.
constexpr float kNearLog2 = 16.f;

// The rules of one call, as the kernels take them.
struct ScoreRules {
  float cap_in;    // scale / cap: x = cap_in * q.k
  float cap_log2;  // cap * log2(e): the capped score in log2 units is cap_log2 tanh x
  const float *alibi_slopes;   // [Hq], or null
  // cap_log2 tanh(cap_in s) = s (c1 + s^2 (c3 + s^2 c5)) for |s| <= near
  float near, c1, c3, c5;
  int32_t window;              // > 0: keys at a distance below it; 0: no window
  const int32_t *prefix_lens;  // [batch], or null: first keys that every query sees
};

}  // namespace pkv
