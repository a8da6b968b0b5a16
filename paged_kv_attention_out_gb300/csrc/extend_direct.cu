// extend_direct.cu - extend under score rules with few query blocks: plan and
// launch of the kernel in direct_tc.cuh.
//
// Against the gather and attention of extend.cu: no copy of the keys, and the
// work is shared out by key tiles instead of whole blocks, so a call with fewer
// blocks than SMs, or with a long prefix and a short chunk, fills the GPU. With
// enough blocks the gathered form is the faster one: its K/V tiles come by
// large boxes, and its softmax keeps less state.
#include "extend_direct.cuh"

namespace pkv {

// Which of the two forms takes less time, in microseconds, by their measured
// parts: the longest block (T key tiles, by the hint) bounds the gathered form
// while there are fewer (block, kv head) pairs N than SMs, the direct one shares
// the tiles out evenly, at more per tile and with a merge; a hint bounds the
// longest row, the others are taken to be half as long and more. (Direct /
// gathered, 32/8 heads of 128, page size 16, distance bias: 1 request of one
// token over 800 keys 16.3 / 18.4, 4 over up to 800 21.2 / 18.1, over 1400 21.1 /
// 26.2; 8 over up to 1400 23.8 / 28.6, up to 2000 24.7 / 35.9; 4 of up to 200
// over up to 1400 33.7 / 31.1, up to 2900 42.1 / 54.3; 8 of up to 200 over up to
// 1400 48.7 / 35.3. Cap 50 and window 4096: 1 of 1000 over 3000 keys 61 / 49; 4
// of up to 2048 over up to 8192 251 / 190.)
static bool direct_is_faster(int64_t pairs, int64_t tiles, int64_t sms) {
  const double gathered = 12.0 + 1.5 * tiles * ((pairs + sms - 1) / sms);
  const double direct = 21.5 + 1.5 * static_cast<double>(pairs) * tiles / sms;
  return direct < gathered;
}

// A call whose blocks have a group each and no more key tiles than this takes
// the direct form for its one launch (8/8 heads of 64, distance bias: 2 of 48
// over up to 200 keys 9.4 us against 11.1 gathered, 400 keys 12.1 / 13.6, 800
// 15.4 / 17.2; 32/8 of 128: 13.3 / 14.0, 18.6 / 16.8, 23.5 / 22.6).
constexpr int kOneLaunchTiles = 3;

static int64_t block_bound(int32_t batch, int32_t total_q, int32_t tpb) {
  return (static_cast<int64_t>(total_q) + tpb - 1) / tpb + batch;
}

size_t extend_direct_workspace(int32_t batch, int32_t total_q, int32_t hq, int32_t hkv, int32_t d,
                               int32_t max_seq, int32_t sm_count) {
  const int64_t blocks = block_bound(batch, total_q, 2 * (direct::kM / (hq / hkv)));
  return direct::plan(static_cast<int32_t>(std::min<int64_t>(blocks, direct::kMaxRuleBlocks)), 2,
                      hkv, d, max_seq, 0, sm_count)
      .workspace_bytes;
}

bool extend_direct_plan(int32_t batch, int32_t total_q, int32_t hq, int32_t hkv, int32_t d,
                        int32_t max_seq, int32_t window, int32_t sm_count, DirectPlan *plan) {
  const int32_t tpb = 2 * (direct::kM / (hq / hkv));
  const int64_t blocks = block_bound(batch, total_q, tpb);
  if (batch > direct::kMaxRuleRequests || blocks > direct::kMaxRuleBlocks) return false;
  // key tiles of a block: all up to the longest request's, or the window's
  int64_t tiles = (static_cast<int64_t>(max_seq) + direct::kN - 1) / direct::kN;
  if (window > 0)
    tiles = std::min<int64_t>(tiles, (static_cast<int64_t>(window) + tpb) / direct::kN + 2);
  const int64_t busy = std::max<int64_t>(batch, (static_cast<int64_t>(total_q) + tpb - 1) / tpb);
  *plan = direct::plan(static_cast<int32_t>(blocks), 2, hkv, d, max_seq, tiles, sm_count);
  return (plan->whole && tiles <= kOneLaunchTiles) ||
         direct_is_faster(busy * hkv, tiles, sm_count > 0 ? sm_count : 1);
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
