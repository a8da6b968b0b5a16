// extend_direct.cuh - the variants of direct_tc.cuh for extend under score rules
// (always with two softmax groups: a block of one query tile is walked by both).
#pragma once

#include "direct_tc.cuh"

namespace pkv {
namespace direct {

template <int D, int kRules>
cudaError_t launch_rules_kv(const DirectArgs &a, bool tma,
                            const CUtensorMap &km, const CUtensorMap &vm, const CUtensorMap &qm,
                            cudaStream_t stream) {
  return tma ? launch<D, 2, true, kRules>(a, km, vm, qm, stream)
             : launch<D, 2, false, kRules>(a, km, vm, qm, stream);
}

template <int D>
cudaError_t launch_rules(const DirectArgs &a, bool tma,
                         const CUtensorMap &km, const CUtensorMap &vm, const CUtensorMap &qm,
                         cudaStream_t stream) {
  const bool cap = a.rules.cap_log2 > 0.f, bias = a.rules.alibi_slopes != nullptr;
  if (cap && bias)
    return launch_rules_kv<D, kRuleRanges | kRuleCap | kRuleBias>(a, tma, km, vm, qm, stream);
  if (cap) return launch_rules_kv<D, kRuleRanges | kRuleCap>(a, tma, km, vm, qm, stream);
  if (bias) return launch_rules_kv<D, kRuleRanges | kRuleBias>(a, tma, km, vm, qm, stream);
  return launch_rules_kv<D, kRuleRanges>(a, tma, km, vm, qm, stream);
}

cudaError_t launch_rules_128(const DirectArgs &a, bool tma,
                             const CUtensorMap &km, const CUtensorMap &vm, const CUtensorMap &qm,
                             cudaStream_t stream);
cudaError_t launch_rules_64(const DirectArgs &a, bool tma,
                            const CUtensorMap &km, const CUtensorMap &vm, const CUtensorMap &qm,
                            cudaStream_t stream);

}  // namespace direct
}  // namespace pkv
