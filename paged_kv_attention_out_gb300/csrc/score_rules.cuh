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

// tanh x = 1 - 2 / (1 + e^2x): an absolute error of 1.2e-7 whatever x. A capped
// score is off by that times the cap (0.09 under a cap of 1e6), so it is for
// |x| > kTanhPoly, or for caps of up to 100.
__device__ __forceinline__ float rule_tanh_far(float x) {
  return 1.f - 2.f * rule_rcp(1.f + rule_exp2(x * (2.f * kLog2e)));
}

// That, or the polynomial near zero: relative error below 2^-20 everywhere, so
// a cap of any size keeps the scores' own precision.
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

// The key tiles of a block of queries whose first one is at position t0, in
// the order walked: tiles 0 .. pre - 1 hold the always visible prefix, tile v
// >= pre of the walk is tile v + gap of the request.
constexpr int kRuleTile = 128;  // keys
struct TileWalk {
  int pre, gap;
};
__device__ __forceinline__ TileWalk tile_walk(int t0, int window, int prefix) {
  const int first = window > 0 ? max(0, t0 - window + 1) / kRuleTile : 0;
  TileWalk w;
  w.pre = min((prefix + kRuleTile - 1) / kRuleTile, first);
  w.gap = first - w.pre;
  return w;
}

// The request's always visible keys, within its row.
__device__ __forceinline__ int rule_prefix(const int32_t *prefix_lens, int r, int seq) {
  return prefix_lens ? min(max(prefix_lens[r], 0), seq) : 0;
}

// Columns 32 w .. 32 w + 31 of a tile that a row sees, one bit each: those in
// lo .. hi and those below pre.
__device__ __forceinline__ uint32_t below_bits(int n) {  // the n lowest bits, 0 <= n clipped
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}
__device__ __forceinline__ uint32_t seen_bits(int lo, int hi, int pre, int w) {
  return (below_bits(hi + 1 - 32 * w) & ~below_bits(lo - 32 * w)) | below_bits(pre - 32 * w);
}

// The prefill softmax's part of the rules (a row of kRuleTile scores a thread).
// A tile is near if a bound of each row's scores comes with the loads (the
// largest absolute raw score of each 32 columns under a cap, the largest raw
// one under a bias alone), every raw score is in the short polynomial's range,
// no column is masked and the bias is not so steep that the bound would be far
// off. Its scores are then computed within the exponential's argument, in pairs
// on the FMA pipe:
//   y = s (c1 + u (c3 + u c5)) [+ slope cc] + (row terms - m),   u = s^2
// three packed instructions more per pair for a cap, one for a bias, and the
// reference m is that bound (at most 2 kNearLog2 + kNearBias above the row's
// maximum, so nothing that counts underflows). Other tiles take the general
// way: every score in place, masked, then its true maximum.
constexpr float kNearBias = 46.f;  // most a bias may change within 32 columns, log2 units

template <bool kCap, bool kBias>
__device__ __forceinline__ void near_pair(float s0, float s1, int cc, float scale_log2,
                                          float slope, float row, const ScoreRules &rules,
                                          float &y0, float &y1) {
  const float2 s = make_float2(s0, s1);
  float2 t = make_float2(row, row);
  if constexpr (kBias) t = __ffma2_rn(make_float2(slope, slope), make_float2(cc, cc + 1), t);
  float2 p = make_float2(scale_log2, scale_log2);
  if constexpr (kCap) {
    const float2 u = __fmul2_rn(s, s);
    p = __ffma2_rn(u, make_float2(rules.c5, rules.c5), make_float2(rules.c3, rules.c3));
    p = __ffma2_rn(u, p, make_float2(rules.c1, rules.c1));
  }
  p = __ffma2_rn(s, p, t);
  y0 = p.x;
  y1 = p.y;
}

// All scores of a tile in log2 units, in place, without the bias; top: the
// largest absolute raw score of the thread's row. The polynomial (in pairs on the
// FMA pipe) where it holds for all of a warp's rows. Otherwise the exponential
// form, alone where a cap is so small that 1.2e-7 of it is less than a score's
// fp32 sum is off by, else with the polynomial score by score, since a tile with
// a large score holds small ones too: each(f) puts f of the raw scores into v. Its
// short loop keeps these two out of the unrolled code, which every tile passes:
// 4 chunks of up to 2048 tokens over up to 8192 keys, 32/8 heads of 128, window
// 4096, cap 50, raw scores up to 5 / 15 / 30 / 60: 190 / 258 / 252 / 364 us; all
// unrolled 195 / 262 / 257 / 372, score by score alone 195 / 263 / 260 / 484.
constexpr float kFarCapLog2 = 144.3f;  // caps of up to 100: off by at most 1.2e-5

template <typename Each>
__device__ __forceinline__ void cap_scores(float (&v)[kRuleTile], float top,
                                           const ScoreRules &rules, Each each) {
  if (__all_sync(0xffffffffu, top * rules.cap_in <= kTanhPoly)) {
#pragma unroll
    for (int cc = 0; cc < kRuleTile; cc += 2) {
      const float2 x = __fmul2_rn(make_float2(v[cc], v[cc + 1]),
                                  make_float2(rules.cap_in, rules.cap_in));
      const float2 u = __fmul2_rn(x, x);
      float2 p = __ffma2_rn(u, make_float2(kTanh9, kTanh9), make_float2(kTanh7, kTanh7));
      p = __ffma2_rn(u, p, make_float2(kTanh5, kTanh5));
      p = __ffma2_rn(u, p, make_float2(kTanh3, kTanh3));
      p = __ffma2_rn(__fmul2_rn(x, u), p, x);
      p = __fmul2_rn(p, make_float2(rules.cap_log2, rules.cap_log2));
      v[cc] = p.x;
      v[cc + 1] = p.y;
    }
  } else if (rules.cap_log2 <= kFarCapLog2) {
    each([&](float s) { return rules.cap_log2 * rule_tanh_far(s * rules.cap_in); });
  } else {
    each([&](float s) { return rules.cap_log2 * rule_tanh(s * rules.cap_in); });
  }
}

// Scores in log2 units less slope times the distance, for the row whose query
// is at column t of the tile (t < 0 or past its end for most). A row's
// -slope t is the same for the whole tile: it is returned, not added, unless
// the tile holds keys behind some row's query (ahead), whose distance is cc - t.
template <bool kScaled>
__device__ __forceinline__ float bias_scores(float (&v)[kRuleTile], float scale_log2, float slope,
                                             int t, bool ahead) {
  const float ft = static_cast<float>(t);
  if (ahead) {
#pragma unroll
    for (int cc = 0; cc < kRuleTile; ++cc)
      v[cc] = fmaf(-slope, fabsf(ft - cc), kScaled ? v[cc] : v[cc] * scale_log2);
    return 0.f;
  }
#pragma unroll
  for (int cc = 0; cc < kRuleTile; ++cc)
    v[cc] = fmaf(slope, cc, kScaled ? v[cc] : v[cc] * scale_log2);
  return -slope * ft;
}

}  // namespace pkv
