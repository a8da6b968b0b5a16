// extend_direct.cu - extend under score rules with few query blocks: plan and
// launch of the kernel in direct_tc.cuh.
//
// Against the gather and attention of extend.cu: no copy of the keys, and the
// work is shared out by key tiles instead of whole blocks, so a call with fewer
// blocks than SMs, or with a long prefix and a short chunk, fills the GPU.
#include "extend_direct.cuh"

namespace pkv {

bool extend_direct_plan(int32_t batch, int32_t total_q, int32_t hq, int32_t hkv, int32_t d,
                        int32_t max_seq, int32_t sm_count, DirectPlan *plan) {
  const int32_t tpb = 2 * (direct::kM / (hq / hkv));
  const int64_t blocks = (static_cast<int64_t>(total_q) + tpb - 1) / tpb + batch;
  if (batch > direct::kMaxRuleRequests || blocks > direct::kMaxRuleBlocks) return false;
  *plan = direct::plan(static_cast<int32_t>(blocks), 2, hkv, d, max_seq, sm_count);
  return true;
}

cudaError_t launch_extend_direct(const PoolGeom &g, int32_t layer, const void *q,
                                 const int32_t *qo_indptr, void *o, float *lse,
                                 const int32_t *page_table, int64_t table_stride,
                                 const int32_t *table_idx, const int32_t *seq_lens, int32_t batch,
                                 int32_t total_q, int32_t hq, float scale, const ScoreRules &rules,
                                 const DirectPlan &plan, void *workspace, unsigned *err,
                                 cudaStream_t stream) {
  direct::DirectArgs a;
  CUtensorMap km{}, vm{}, qm{};
  bool tma;
  if (!direct::direct_args(&a, &km, &vm, &qm, &tma, g, layer, q, qo_indptr, o, lse, page_table,
                           table_stride, table_idx, seq_lens, batch, total_q, hq, scale, plan,
                           workspace, err))
    return cudaErrorInvalidValue;
  a.rules = rules;
  return g.d == 128 ? direct::launch_rules_128(a, tma, km, vm, qm, stream)
                    : direct::launch_rules_64(a, tma, km, vm, qm, stream);
}

}  // namespace pkv
