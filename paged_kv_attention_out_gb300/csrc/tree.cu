// tree.cu - attention of a tree of drafted tokens over the paged cache.
//
// Mathematics. Request r has c_r drafted tokens, stored as the last c_r of its
// seq_lens[r] keys (p_r = seq_lens[r] - c_r cached ones before them). Token j
// sees every cached key, and of the drafted ones itself and its ancestors by
// parents[] (a parent is an earlier token, -1 the last cached one): a row mask
// that touches only the key tiles which hold drafted keys. The kernel is in
// direct_tc.cuh. 16 requests with up to 32768 keys, 32/8 heads of 128, page
// size 16: 144 us for 16 drafts each (0.95 of the copy rate), 169-174 for 64.
#include "direct_tc.cuh"

namespace pkv {
namespace {

using namespace direct;

template <int D>
cudaError_t launch_d(const DirectArgs &a, const DirectPlan &plan, bool tma, const CUtensorMap &km,
                     const CUtensorMap &vm, const CUtensorMap &qm, cudaStream_t stream) {
  if (plan.query_tiles == 1)
    return tma ? launch<D, 1, true, 0>(a, km, vm, qm, stream)
               : launch<D, 1, false, 0>(a, km, vm, qm, stream);
  return tma ? launch<D, 2, true, 0>(a, km, vm, qm, stream)
             : launch<D, 2, false, 0>(a, km, vm, qm, stream);
}

// Blocks per request.
int32_t tree_blocks(int32_t hq, int32_t hkv, int32_t max_tree, int32_t tiles_per_block) {
  const int32_t tpb = tiles_per_block * (kM / (hq / hkv));
  return (max_tree + tpb - 1) / tpb;
}

}  // namespace

// One query tile where it holds a request's drafts, or where every query tile
// can have a group of its own and the keys, which its other tiles read again,
// stay in L2; otherwise two. (64 drafts, blocks of one / two tiles, page size 16;
// 32/8 heads of 128: 1 request of 520 keys 12.9 / 18.6 us, of 1400 18.3 / 18.9, 4
// of up to 900 15.8 / 22.9, 2 of up to 2900 20.3 / 25.4, 8 of up to 2900 32.6 /
// 32.4; 28/4 of 64: 4 of up to 2900 18.4 / 21.7.)
constexpr int64_t kReadTwice = 64 << 20;

DirectPlan tree_plan(int32_t batch, int32_t hq, int32_t hkv, int32_t d, int32_t max_tree,
                     int32_t max_seq, int32_t sm_count) {
  const int64_t tiles = (static_cast<int64_t>(max_seq) + kN - 1) / kN;
  auto plan = [&](int32_t query_tiles, int32_t tiles_per_block) {
    return direct::plan(batch * tree_blocks(hq, hkv, max_tree, tiles_per_block), query_tiles,
                        tiles_per_block, hkv, d, max_seq, tiles, sm_count);
  };
  const DirectPlan one = plan(1, 1);
  if (max_tree <= kM / (hq / hkv)) return one;
  const DirectPlan two = plan(2, 2);
  const int64_t kv_bytes = 4 * batch * tiles * kN * hkv * d;
  const bool few = one.max_blocks * static_cast<int64_t>(hkv) <= sm_count && kv_bytes <= kReadTwice;
  DirectPlan p = one.whole || few ? one : two;
  p.workspace_bytes = std::max(one.workspace_bytes, two.workspace_bytes);  // (grows with the sizes)
  return p;
}

cudaError_t launch_tree(const PoolGeom &g, int32_t layer, const void *q, const int32_t *qo_indptr,
                        const int32_t *parents, void *o, float *lse, const int32_t *page_table,
                        int64_t table_stride, const int32_t *table_idx, const int32_t *seq_lens,
                        int32_t batch, int32_t total_q, int32_t hq, float scale, int32_t max_tree,
                        const DirectPlan &plan, void *workspace, unsigned *err,
                        cudaStream_t stream) {
  DirectArgs a;
  CUtensorMap km{}, vm{}, qm{};
  bool tma;
  if (!direct_args(&a, &km, &vm, &qm, &tma, g, layer, q, qo_indptr, o, lse, page_table,
                   table_stride, table_idx, seq_lens, batch, total_q, hq, scale, plan, workspace,
                   err))
    return cudaErrorInvalidValue;
  a.parents = parents;
  a.max_tree = max_tree;
  a.blocks_per_req = tree_blocks(hq, g.hkv, max_tree, plan.tiles_per_block);
  a.read_once = a.blocks_per_req == 1;
  return g.d == 128 ? launch_d<128>(a, plan, tma, km, vm, qm, stream)
                    : launch_d<64>(a, plan, tma, km, vm, qm, stream);
}

}  // namespace pkv
