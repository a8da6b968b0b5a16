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

// What the host knows of a call.
struct Sizes {
  double batch, total_q, keys;  // keys: bound on the requests' keys together
  double blocks;                // query blocks that hold tokens, about
  double tiles;                 // key tiles of the longest block
  bool one_tile;                // a request's tokens fit one query tile, on the average
  double hkv, d, sms;
};

// Which of the two forms takes less time, in microseconds, by their measured
// parts. Gathered: every key is copied (at 5 TB/s; a few us of it are hidden),
// then the longest block's tiles, or all tiles by the SMs, at 1.5 each. Direct:
// all tiles and four for each block's beginning and end, shared out evenly, at
// the copy rate's 1.5 a tile for one query tile and the softmax's 2.2 for two.
// (Direct / gathered, 32/8 heads of 128, page size 16; distance bias: 1 request
// of one token over 800 keys 16.3 / 18.4, 4 over up to 800 21.2 / 18.1, 8 over up
// to 1400 23.8 / 28.6; 64 over up to 16000 316 / 922; 32 of up to 16 over up to
// 4000 68 / 125; 8 of up to 200 over up to 1400 48.7 / 35.3, 4 over up to 2900
// 42.1 / 54.3; 4 of up to 512 over up to 16000 177 / 245. Cap 50 and window 4096:
// that 89 / 81, 64 of one token over up to 16000 184 / 495, 1 of 1000 over 3000
// 62 / 49, 4 of up to 2048 over up to 8192 251 / 191.)
static bool direct_is_faster(const Sizes &z) {
  const double mean = std::max(
      1.0, std::min(z.tiles, (z.keys - z.total_q / 2) / (z.batch * direct::kN)));
  const double waves = z.blocks * z.hkv / z.sms;
  const double copied = 8.0 * z.batch * mean * direct::kN * z.hkv * z.d;  // bytes, both ways
  const double gathered =
      12.0 + std::max(0.0, copied / 5e6 - 4.0) + 1.5 * std::max(z.tiles, mean * waves);
  const double direct =
      z.one_tile ? 21.5 + 1.5 * (mean + 4) * waves : 26.0 + 2.2 * (mean + 4) * waves;
  return direct < gathered;
}

// A call whose blocks have a group each takes the direct form with one query
// tile to a block (both softmax groups walk it), or with two where those do not
// fit but the key tiles are no more than kOneLaunchTiles: one launch, no shares,
// no copy. (Blocks of one tile, direct / of two / gathered, distance bias: 1 of
// 200 tokens over 1000 keys, 32/8 heads of 128, 18.4 / 24.8 / 23.8 us; 4 of up to
// 200 over up to 1600, 16/16 of 64, 18.3 / 30.2 / 29.3; 2 of up to 300 over up to
// 1500, 32/8 of 128, 23.8 / 34.8 / 32.5; 2 of 48 over up to 200, 8/8 of 64, 9.4 /
// 9.4 / 11.1. Of two: 3 tiles 12.1 / 13.6 gathered, 4 13.3 / 14.0, 7 23.5 / 22.6.
// Shared out, one tile to a block is the slower: 4 of up to 512 over up to 16000
// 224 / 176.)
constexpr int kOneLaunchTiles = 3;

static int64_t block_bound(int32_t batch, int32_t total_q, int32_t tpb) {
  return (static_cast<int64_t>(total_q) + tpb - 1) / tpb + batch;
}

size_t extend_direct_workspace(int32_t batch, int32_t total_q, int32_t hq, int32_t hkv, int32_t d,
                               int32_t max_seq, int32_t sm_count) {
  const int64_t blocks = block_bound(batch, total_q, 2 * (direct::kM / (hq / hkv)));
  return direct::plan(static_cast<int32_t>(std::min<int64_t>(blocks, direct::kMaxRuleBlocks)), 2, 2,
                      hkv, d, max_seq, 0, sm_count)
      .workspace_bytes;
}

bool extend_direct_plan(int32_t batch, int32_t total_q, int32_t hq, int32_t hkv, int32_t d,
                        int32_t max_seq, int64_t max_total_keys, int32_t window,
                        int32_t sm_count, DirectPlan *plan) {
  const int32_t tpt = direct::kM / (hq / hkv), tpb = 2 * tpt;
  if (batch > direct::kMaxRuleRequests) return false;
  int64_t tiles = 0;
  for (int32_t n = 1; n <= 2; ++n) {  // query tiles to a block
    const int64_t blocks = block_bound(batch, total_q, n * tpt);
    if (blocks > direct::kMaxRuleBlocks) continue;
    // key tiles of a block: all up to the longest request's, or the window's
    tiles = (static_cast<int64_t>(max_seq) + direct::kN - 1) / direct::kN;
    if (window > 0)
      tiles = std::min<int64_t>(tiles,
                                (static_cast<int64_t>(window) + n * tpt) / direct::kN + 2);
    *plan = direct::plan(static_cast<int32_t>(blocks), 2, n, hkv, d, max_seq, tiles, sm_count);
    if (plan->whole && (n == 1 || tiles <= kOneLaunchTiles)) return true;
  }
  if (block_bound(batch, total_q, tpb) > direct::kMaxRuleBlocks) return false;
  Sizes z;
  z.batch = batch;
  z.total_q = total_q;
  z.keys = static_cast<double>(batch) * max_seq;
  if (max_total_keys >= 1) z.keys = std::min(z.keys, static_cast<double>(max_total_keys));
  z.blocks = std::max<double>(batch, (static_cast<int64_t>(total_q) + tpb - 1) / tpb);
  z.tiles = static_cast<double>(tiles);
  z.one_tile = total_q <= static_cast<int64_t>(batch) * tpt;
  z.hkv = hkv;
  z.d = d;
  z.sms = sm_count > 0 ? sm_count : 1;
  return direct_is_faster(z);
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
