// direct_tc.cuh - attention of a few query blocks per request over the paged
// cache, on tcgen05 / TMEM, its K/V read straight from the pool. Two uses: a
// tree of drafted tokens (tree.cu) and extend under score rules when there are
// few blocks (extend_direct.cu); kRules = 0 is the tree, otherwise the rules'
// bits (score_rules.cuh).
//
// A query block is up to kQT x (128 / g) tokens of one request x the g query
// heads of one kv head. It walks the key tiles that hold a key some of its
// tokens see: S = scale Q K^T, masked; o = softmax(S) V; lse = log sum exp S.
// The running maximum and sum of each row stay in registers while the keys
// stream by once.
//
// What bounds it. K/V is read once per block of 128 or 256 rows: 2 * rows FLOPs
// per byte, so memory up to a hundred rows or so, and near the softmax's rate
// at 256.
//
// Schedule. The unit of work is a 128-key tile of one query block, with a cost
// of its own where two query tiles share it. Group i of G = SMs / Hkv groups
// takes the i-th equal share of the cost of all units, in (block, key) order;
// the Hkv CTAs of a group walk the same share, one kv head each, so the pieces
// of a token's K (V) row are read at about the same time. Every group has the
// same work whatever the requests' lengths are, and only its first and last
// block can be shared with a neighbour: those go out as fp32 partial states
// (slot 2 i of the workspace for a block begun by an earlier group, 2 i + 1
// for one that goes on in the next) and a second kernel merges them; every
// other block is written directly.
//
// A call with few, short blocks gives each its own group instead: no share to
// find, no partial state, no second kernel.
//
// Roles of a CTA (kQT = 1 or 2 query tiles of 128 rows):
//   warps 0 .. 4 kQT - 1  softmax: one query row per thread (TMEM lane)
//   next warp             TMEM allocation and the MMAs. The warp stays together
//       and one elected lane issues, so that descriptors and loop state are in
//       uniform registers: a lone thread took 60 clocks an MMA or commit, which
//       made this warp the bound.
//   the rest              producers: the Q tiles by TMA, then K and V tiles
//       alternately into a ring of slots; kTma: three warps, TMA boxes of a
//       power of two of rows that divides the page size, the box holding the
//       request's last key by 16-byte cp.async with zero fill, so that no
//       stale bits behind it reach P V; otherwise three or four warps of
//       cp.async.
// With one query tile the scores are double buffered, S(j + 1) is computed
// while the softmax works on S(j); with two, the tiles take turns. A block of
// the two-tile kernel whose tokens fit one tile is walked by both softmax
// groups, each taking every other key tile with a state of its own (m, l, O),
// which the first group joins at the end of the segment.
// Every hand-off is an mbarrier; every wait is bounded (tc_common.cuh).
#pragma once

#include <cuda.h>
#include <math.h>

#include <algorithm>

#include "pkv_common.cuh"
#include "pkv_internal.h"
#include "score_rules.cuh"
#include "tc_common.cuh"
#include "tensor_map.h"

namespace pkv {
namespace direct {

constexpr int kM = 128;  // query rows per tile (= TMEM lanes)
constexpr int kN = kRuleTile;  // keys per K/V tile
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 0;    // score buffers at 0 and 128
constexpr uint32_t kTmemO = 256;  // O_x at 256 + 128 x
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr int kMaxTree = PKV_MAX_TREE_TOKENS;
constexpr int kMaskWords = kMaxTree / 32;
constexpr int kMinTiles = 4;    // smallest share of a group, in key tiles
constexpr int kBlockTiles = 2;  // cost of a block's prologue and epilogue, in key tiles
// Cost of a key tile for a block of one and of two query tiles. At D = 128
// both are near the tile's 64 KB at the copy rate (64 drafts: 171, 170, 169 and
// 176 us for 1:1, 5:6, 3:4 and 3:5; 33 drafts: 153, 155, 155 and 163); at 64
// two tiles' softmax takes longer than 32 KB do (107, 117, 111 us for 3:5, 5:6
// and 3:4; 33 drafts: 88, 106, 99).
struct TileCost {
  int one, two;
};
constexpr TileCost tile_cost(int d) { return d == 128 ? TileCost{5, 6} : TileCost{3, 5}; }
constexpr int kMergeRows = 32;

// Producer warps; warp w issues every kProducerWarps-th K or V tile. A warp
// takes longer to issue a tile's copies than their bytes take (boxes of 16
// rows one lane after the other, or 64 row pieces per lane), so several work
// at a time: twelve warps of a CTA cost no more registers than ten (a softmax
// thread holds a whole score row). Page size 16, one query tile: 185 us with
// one TMA warp, 147 with three.
constexpr int producer_warps(int query_tiles, bool tma) {
  return tma || query_tiles == 2 ? 3 : 4;
}

// Registers per thread of the two-tile kernel's warpgroups: of 384 x 168 at
// launch, the MMA and producer warps give up what the eight softmax warps take.
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * 168, "registers of the launch");
static_assert(producer_warps(2, true) == 3 && producer_warps(2, false) == 3,
              "three whole warpgroups");

template <int D, int kQT>
struct DirectSmem {
  static constexpr int kQBytes = kM * D * 2;   // one query tile
  static constexpr int kSlotBytes = kN * D * 2;  // one K or V tile
  static constexpr int kSlots = D == 128 ? (kQT == 2 ? 5 : 6) : 8;
  static constexpr int kQ = 0;
  static constexpr int kRing = kQT * kQBytes;
  static constexpr int kBars = kRing + kSlots * kSlotBytes;
  // + barriers + alignment slack; the ring keeps a second CTA off the SM, so
  // that one 512-column TMEM allocation is all there is
  static constexpr int kTotal = kBars + 32 * 8 + 1024;
  static_assert(kTotal <= 227 * 1024 - 1792, "shared memory (with the static arrays)");
  static_assert(kTotal > 114 * 1024, "one CTA per SM");
  // A warp that waits for unit u's slot has issued unit u - warps, so unit u -
  // warps - slots is consumed, and with it every unit up to two before it (K
  // tiles are consumed ahead of the V tile before them): unit u - 2 slots among
  // them, without which the parity waited for could be an older phase's.
  static_assert(producer_warps(kQT, true) <= kSlots - 2 && producer_warps(kQT, false) <= kSlots - 2,
                "producer warps run too far ahead of the ring");
};

enum : int {
  kBarFull = 0,       // [8] producers: the slot's tile landed
  kBarEmpty = 8,      // [8] MMA: every MMA reading the slot done
  kBarSFull = 16,     // [2] MMA: score buffer ready
  kBarPFull = 18,     // [2] softmax: P written over the score buffer
  kBarPvDone = 20,    // MMA (one query tile): the tile's P V done
  kBarOFull = 21,     // [2] MMA: O_x final
  kBarOEmpty = 23,    // [2] softmax: O_x read out
  kBarQFull = 25,     // producer: Q landed
  kBarQEmpty = 26,    // MMA: every S of the segment done
  kBarState = 27,     // softmax group 1: its state of a shared query tile is in shared memory
  kBarTeardown = 28,
};

struct DirectArgs {
  const __nv_bfloat16 *k_plane;  // this layer's K rows [slots][Hkv * D]
  const __nv_bfloat16 *v_plane;
  int64_t slots;
  int32_t page_size;
  int32_t hkv;
  const int32_t *qo_indptr;
  const int32_t *parents;  // tree
  __nv_bfloat16 *o;
  float *lse;
  const int32_t *page_table;
  int64_t table_stride;
  const int32_t *table_idx;
  const int32_t *seq_lens;
  int32_t batch;
  int32_t total_q;
  int32_t hq;
  int32_t group;
  int32_t tokens_per_tile;
  int32_t tokens_per_block;  // one or two query tiles' (kQT = 2)
  int32_t max_tree;        // tree
  int32_t blocks_per_req;  // tree
  int32_t read_once;       // no K/V byte is read by more than one block
  int32_t max_blocks;  // entries of `table`
  int32_t groups;
  int32_t whole;       // group i takes block i (groups = max_blocks), nothing is shared or merged
  TileCost cost;
  int32_t box;           // rows of a K/V TMA box (kTma)
  float scale_log2;      // |scale| log2(e) (log2(e) for scale 0), > 0
  int32_t q_mode;        // 0: scores as they are, 1: negated (scale < 0), 2: zero (scale 0)
  float *part_o;         // [2 groups][Hkv][D / 4][rows] float4
  float *part_lse;       // [2 groups][Hkv][rows]
  // per block: its first and last group (-1, -1 if nothing is merged), its
  // first token and number of tokens
  int4 *table;
  ScoreRules rules;  // extend
  unsigned *err;
};

// Most requests, and blocks in all (max_blocks), of a call under rules: one
// thread each finds a request's blocks, and a block's request.
constexpr int kMaxRuleRequests = 256;
constexpr int kMaxRuleBlocks = 352;

// The call's blocks. Tree: a fixed number per request. Rules: block first[r]
// is the first of request r (count from 0 in shared memory).
struct Blocks {
  const uint16_t *first;
  int count;
};

// One query block: up to kQT tokens_per_tile tokens of one request.
struct Block {
  int req, sub, t_base, tokens, p, c, seq, tiles;
  int prefix, lo;  // rules: keys below `prefix` and from `lo` on are seen by some token
  TileWalk walk;   // rules: which key tiles those are
  int cost;   // of a key tile
  int extra;  // of the block's prologue and epilogue, added to its first tile's
};

// What is wrong with a request's tables (0: nothing).
template <int kRules>
__device__ __forceinline__ unsigned bad_request(const DirectArgs &a, int r, int beg, int end,
                                                int seq) {
  unsigned bad = 0;
  const int row = a.table_idx ? a.table_idx[r] : r;
  if (beg < 0 || end < beg || end > a.total_q || (seq >= 0 && seq < end - beg)) bad |= kErrIndptr;
  if (seq < 0 || seq > a.table_stride * a.page_size) bad |= kErrSeqLen;
  if (row < 0) bad |= kErrTableIdx;
  if (kRules == 0 && !(bad & kErrIndptr) && end - beg > a.max_tree) bad |= kErrTree;
  return bad;
}

// Block b of the call, tiles = 0 if there is nothing to compute. Keys behind
// the block's last token (and, under rules, outside what its tokens see) are
// of no interest to it.
template <int kQT, int kRules>
__device__ __forceinline__ Block load_block(const DirectArgs &a, const Blocks &blocks, int b,
                                            bool report) {
  Block k{};
  if constexpr (kRules == 0) {
    k.req = b / a.blocks_per_req;
    k.sub = b - k.req * a.blocks_per_req;
  } else {
    int hi = a.batch - 1;  // the last request that begins at or before block b
    while (k.req < hi) {
      const int mid = (k.req + hi + 1) / 2;
      if (blocks.first[mid] <= b)
        k.req = mid;
      else
        hi = mid - 1;
    }
    k.sub = b - blocks.first[k.req];
  }
  const int beg = a.qo_indptr[k.req], end = a.qo_indptr[k.req + 1];
  k.seq = a.seq_lens[k.req];
  k.c = end - beg;
  k.p = k.seq - k.c;
  const int tpb = a.tokens_per_block;
  const unsigned bad = bad_request<kRules>(a, k.req, beg, end, k.seq);
  if (bad) {
    if (report && k.sub == 0) flag_error(a.err, bad);
    k.tiles = 0;
    return k;
  }
  k.t_base = beg + k.sub * tpb;
  k.tokens = min(tpb, k.c - k.sub * tpb);
  k.cost = k.tokens <= a.tokens_per_tile ? a.cost.one : a.cost.two;
  k.extra = kBlockTiles * a.cost.one;
  if (k.tokens <= 0) return k;
  const int t0 = k.p + k.sub * tpb;
  k.tiles = (t0 + k.tokens + kN - 1) / kN;
  if constexpr (kRules != 0) {
    k.prefix = rule_prefix(a.rules.prefix_lens, k.req, k.seq);
    k.lo = a.rules.window > 0 ? max(0, t0 - a.rules.window + 1) : 0;
    k.walk = tile_walk(t0, a.rules.window, k.prefix);
    k.tiles = max(k.tiles, (k.prefix + kN - 1) / kN) - k.walk.gap;
  }
  return k;
}

// First key of the block's tile v.
template <int kRules>
__device__ __forceinline__ int tile_key(const TileWalk &w, int v) {
  return (kRules != 0 && v >= w.pre ? v + w.gap : v) * kN;
}

// Quotients of non-negative numbers, in 32 bits where they fit (a 64-bit
// division takes a tenth of a microsecond, and several lie on the way to the
// first load).
__device__ __forceinline__ long long div_down(long long x, long long y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}
__device__ __forceinline__ long long div_up(long long x, long long y) {
  return div_down(x + y - 1, y);
}

// A CTA's walk over its share of the tiles; every role keeps its own copy.
struct Walk {
  int block;      // of the next segment
  int skip;       // tiles of it that belong to an earlier group
  long long left;  // cost of the share from the next tile on
};

struct Segment {
  Block b;
  int tile0, n;   // key tiles tile0 .. tile0 + n - 1
  bool whole;     // the block's every tile: written directly
  int slot;       // of its partial state otherwise
};

template <int kQT, int kRules>
__device__ __forceinline__ bool next_segment(const DirectArgs &a, const Blocks &blocks, Walk &w,
                                             Segment &s) {
  while (w.block < blocks.count && w.left > 0) {
    s.b = load_block<kQT, kRules>(a, blocks, w.block, false);
    ++w.block;
    s.tile0 = w.skip;
    w.skip = 0;
    if (s.tile0 >= s.b.tiles) continue;
    // the tiles that begin within the share (the second begins extra later)
    const long long extra = s.tile0 == 0 ? s.b.extra : 0;
    const long long n = w.left > extra ? div_up(w.left - extra, s.b.cost) : 0;
    s.n = static_cast<int>(min(static_cast<long long>(s.b.tiles - s.tile0), n > 1 ? n : 1ll));
    s.whole = s.n == s.b.tiles;
    s.slot = 2 * static_cast<int>(blockIdx.y) + (s.tile0 == 0 ? 1 : 0);
    w.left -= extra + static_cast<long long>(s.n) * s.b.cost;
    return true;
  }
  return false;
}

// Whether the two softmax groups of the two-tile kernel share the block's one
// query tile (group x takes key tiles x, x + 2, ..) or have a tile each.
__device__ __forceinline__ bool shared_tile(const DirectArgs &a, const Segment &s) {
  return s.b.tokens <= a.tokens_per_tile && s.n > 1;
}

// Key tiles that softmax group x walks of the segment (two-tile kernel): its
// share of them, or all that may hold a key its query tile's tokens see.
template <int kRules>
__device__ __forceinline__ int tiles_of(const DirectArgs &a, const Segment &s, int tpb, int x) {
  if (shared_tile(a, s)) return (s.n + 1 - x) / 2;
  const int tok = min(a.tokens_per_tile, s.b.tokens - x * a.tokens_per_tile);
  if (tok <= 0) return 0;
  int end = (s.b.p + s.b.sub * tpb + x * a.tokens_per_tile + tok + kN - 1) / kN;
  if (kRules != 0) end = max(end, (s.b.prefix + kN - 1) / kN) - s.b.walk.gap;
  return max(0, min(s.n, end - s.tile0));
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}

template <int D, int kQT, bool kTma, int kRules>
__global__ void __launch_bounds__((4 * kQT + 1 + producer_warps(kQT, kTma)) * 32, 1)
    direct_kernel(const __grid_constant__ CUtensorMap k_map,
                const __grid_constant__ CUtensorMap v_map,
                const __grid_constant__ CUtensorMap q_map, const DirectArgs a) {
  using S = DirectSmem<D, kQT>;
  constexpr int kSlots = S::kSlots;
  constexpr int kSoftmaxWarps = 4 * kQT;
  constexpr int kMmaWarp = kSoftmaxWarps;
  constexpr int kProducerWarp0 = kMmaWarp + 1;
  constexpr int kProducerWarps = producer_warps(kQT, kTma);
  constexpr int kThreads = (kSoftmaxWarps + 1 + kProducerWarps) * 32;
  constexpr int kHalves = D / 64;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ long long s_scan[kThreads / 32];
  __shared__ Walk s_walk;
  __shared__ float2 s_state[kQT == 2 ? kM : 1];  // (m, l) of group 1's rows (shared query tile)
  // Tree: a copy of the request's parents for each softmax group (root: 255).
  // Rules: the first block of each request.
  __shared__ uint8_t s_parents[kRules == 0 ? kQT : 1][kRules == 0 ? kMaxTree : 4];
  __shared__ uint16_t s_first[kRules == 0 ? 1 : kMaxRuleRequests];
  constexpr bool kCap = (kRules & kRuleCap) != 0;
  constexpr bool kBias = (kRules & kRuleBias) != 0;
  static_assert(kRules == 0 || kThreads >= kMaxRuleBlocks, "a thread per block");
  const int tid = threadIdx.x;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (uniform for the compiler, too)
  const int lane = tid & 31;
  const int kvh = blockIdx.x;
  const int tpt = a.tokens_per_tile;
  const int tpb = a.tokens_per_block;

  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_addr(smem);
  const uint32_t bars = sbase + S::kBars;
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  volatile int *abort = &s_abort;

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(bar(kBarFull + i), 32);  // the lanes of the warp that fills it
      mbar_init(bar(kBarEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarSFull + i), 1);
      mbar_init(bar(kBarPFull + i), 128);
      mbar_init(bar(kBarOFull + i), 1);
      mbar_init(bar(kBarOEmpty + i), 128);
    }
    mbar_init(bar(kBarPvDone), 1);
    mbar_init(bar(kBarQFull), 1);
    mbar_init(bar(kBarQEmpty), 1);
    mbar_init(bar(kBarState), 128);
    mbar_init(bar(kBarTeardown), 1);
    s_abort = 0;
    s_walk = Walk{0, 0, 0};
    mbar_init_fence();
  }
  {
    // rows group * tpt .. 127 of a query tile are never loaded: zero them once
    const int pad_rows = kM - a.group * tpt;
    for (int i = tid; i < kQT * kHalves * pad_rows * 8; i += kThreads) {
      const int chunk = i & 7, row = (i >> 3) % pad_rows, region = (i >> 3) / pad_rows;
      *reinterpret_cast<uint4 *>(smem + S::kQ + region * (kM * 128) + (kM - pad_rows + row) * 128 +
                                 chunk * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_async_shared();
  }
  if (warp == kMmaWarp) tmem_alloc(smem_addr(&s_tmem), kTmemCols);

  Blocks blocks{s_first, a.batch * a.blocks_per_req};
  grid_dependency_wait();  // pool, q and tables may come from the previous kernel
  grid_dependents_launch();
  {
    // The share of this CTA's group: the total cost of all blocks, then the
    // block that holds the share's beginning. Thread t of a round takes block
    // base + t.
    const bool lead = blockIdx.x == 0 && blockIdx.y == 0;
    auto scan = [&](long long v, long long &total) {  // inclusive, over the CTA
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += u;
      }
      __syncthreads();  // s_scan of the previous round is read
      if (lane == 31) s_scan[warp] = v;
      __syncthreads();
      long long before = 0, all = 0;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) {
        before += w < warp ? s_scan[w] : 0;
        all += s_scan[w];
      }
      total = all;
      return v + before;
    };
    long long total = 0, round;
    if constexpr (kRules != 0) {
      int n = 0;  // blocks of request tid
      if (tid < a.batch) {
        const int beg = a.qo_indptr[tid], end = a.qo_indptr[tid + 1];
        const unsigned bad = bad_request<kRules>(a, tid, beg, end, a.seq_lens[tid]);
        if (bad && lead) flag_error(a.err, bad);
        n = bad ? 0 : (end - beg + tpb - 1) / tpb;
      }
      const long long end = scan(n, round);
      // malformed tables can hold more blocks than the call has tokens for (and
      // `table` entries): those past the bound, all of requests behind the
      // first malformed pair, are left out
      const long long most = a.max_blocks;
      if (tid < a.batch) s_first[tid] = static_cast<uint16_t>(min(end - n, most));
      blocks.count = static_cast<int>(min(round, most));
      __syncthreads();
    }
    if (a.whole) {  // block i is all that group i has
      const int b = static_cast<int>(blockIdx.y);
      blocks.count = min(blocks.count, b + 1);
      if (tid == 0) {
        if (kRules == 0 && blockIdx.x == 0) load_block<kQT, kRules>(a, blocks, b, true);
        s_walk = Walk{b, 0, 0x7fffffff};
      }
    } else {
      const int nblocks = blocks.count;
      struct Cost {
        int tiles, unit, extra, t_base, tokens;
      };
      auto cost_of = [&](int b, bool report, Cost &c) -> long long {
        c = Cost{0, 1, 0, 0, 0};
        if (b >= nblocks) return 0;
        const Block k = load_block<kQT, kRules>(a, blocks, b, kRules == 0 && report);
        if (k.tiles == 0) return 0;
        c = Cost{k.tiles, k.cost, k.extra, k.t_base, k.tokens};
        return k.extra + static_cast<long long>(k.tiles) * k.cost;
      };
      Cost unit0, unit;
      const long long mine = cost_of(tid, lead, unit0);
      const long long first_end = scan(mine, round);
      const long long first_total = round;
      total = round;
      for (int b0 = kThreads; b0 < nblocks; b0 += kThreads) {
        scan(cost_of(b0 + tid, lead, unit), round);
        total += round;
      }
      // at least one tile begins in every share that a block covers
      const int least = max(kMinTiles * a.cost.one, kBlockTiles * a.cost.one + a.cost.two);
      const long long per = max(static_cast<long long>(least), div_up(total, a.groups));
      const long long lo = per * blockIdx.y;
      const long long hi = min(total, lo + per);
      long long base = 0;
      for (int b0 = 0; b0 < nblocks && (lead || base <= lo); b0 += kThreads) {
        const int b = b0 + tid;
        long long cost = mine;
        unit = unit0;
        if (b0 > 0) cost = cost_of(b, false, unit);
        long long end = first_end;
        round = first_total;
        if (b0 > 0) end = scan(cost, round);
        end += base;
        const long long start = end - cost;
        if (cost > 0 && start <= lo && lo < end && lo < hi) {
          // the first tile that begins in the share
          const long long first =
              lo > start ? max(1ll, div_up(max(0ll, lo - start - unit.extra), unit.unit)) : 0;
          const long long at = start + (first > 0 ? unit.extra : 0) + first * unit.unit;
          s_walk = Walk{b, static_cast<int>(first), hi - at};
        }
        if (lead && b < nblocks && a.groups > 1) {
          // which groups the block's tiles begin in (the merge reads this)
          int4 e = make_int4(-1, -1, unit.t_base, unit.tokens);
          if (cost > 0) {
            const long long last = unit.tiles > 1 ? end - unit.unit : start;
            const int g0 = static_cast<int>(div_down(start, per));
            const int g1 = static_cast<int>(div_down(last, per));
            if (g1 > g0) e.x = g0, e.y = g1;
          }
          a.table[b] = e;
        }
        base += round;
      }
      // entries of blocks that the call turned out not to have: the merge's grid
      // is sized by a host bound, and the workspace holds anything on entry
      if (lead && a.groups > 1)
        for (int b = nblocks + tid; b < a.max_blocks; b += kThreads)
          a.table[b] = make_int4(-1, -1, 0, 0);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s_tmem;
  Walk walk = s_walk;
  Segment sg;

  if (warp >= kMmaWarp) {
    // one warpgroup with two query tiles: the MMA warp and three producers
    if constexpr (kQT == 2) warpgroup_registers_dec<kOtherRegs>();
    if (warp >= kProducerWarp0) {
      // ------------------------------------------------------------ producers
      const int pw = warp - kProducerWarp0;
      const int64_t row_elems = static_cast<int64_t>(a.hkv) * D;
      const int64_t head_off = static_cast<int64_t>(kvh) * D;
      // K/V that one block reads is read once: its lines go first (page size
      // 64: 144.7 us against 150.2 with the default policy).
      const uint64_t kv_policy = a.read_once ? l2_evict_first_policy() : l2_evict_normal_policy();
      constexpr int kGroups = kTma ? 1 : kN / 32;  // boxes (keys) per lane and tile
      constexpr int kChunks = D / 8;
      constexpr int kKeysPerInstr = 32 / kChunks;
      const int ch = lane % kChunks;
      bool ok = true;
      uint32_t u0 = 0;  // ring unit (K and V tiles) of the segment's first tile
      uint32_t issued = 0;  // one past this warp's last unit
      int segs = 0;
      while (ok && next_segment<kQT, kRules>(a, blocks, walk, sg)) {
        const int row = a.table_idx ? a.table_idx[sg.b.req] : sg.b.req;
        const int32_t *pages = a.page_table + static_cast<int64_t>(row) * a.table_stride;
        // This lane's boxes of tile j (kTma: box `lane` of the tile; otherwise
        // one key of each 32): the page entry, loaded one of the warp's units
        // ahead and looked at only when the tile's copies are issued, and the
        // first pool row (-1 past the request or for a bad page).
        const int box = kTma ? a.box : 1;
        auto box_key = [&](int j, int g) -> int {
          const int at = kTma ? lane * box : g * 32 + lane;
          const int key = tile_key<kRules>(sg.b.walk, sg.tile0 + j) + at;
          if (kRules != 0 && key >= sg.b.prefix && key + box <= sg.b.lo) return -1;  // seen by none
          return at < kN && key < sg.b.seq ? key : -1;
        };
        auto load_entries = [&](int j, int (&e)[kGroups]) {
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            const int key = box_key(j, g);
            e[g] = key >= 0 ? __ldg(pages + key / a.page_size) : -1;
          }
        };
        auto first_row = [&](int j, int g, int ent) -> long long {
          const int key = box_key(j, g);
          if (key < 0) return -1;
          const long long s = static_cast<long long>(ent) * a.page_size + key % a.page_size;
          if (ent < 0 || s + box > a.slots) {
            flag_error(a.err, kErrPage);
            return -1;
          }
          return s;
        };
        // this warp's units of the segment: first, first + kProducerWarps, ..
        // (unit w holds K, or V if w is odd, of tile w / 2)
        const uint32_t n_units = 2u * static_cast<uint32_t>(sg.n);
        const uint32_t first =
            (static_cast<uint32_t>(pw) + kProducerWarps - u0 % kProducerWarps) % kProducerWarps;
        int next[kGroups];
        if (first < n_units) load_entries(static_cast<int>(first >> 1), next);
        if (pw == 0) {
          if (segs > 0) ok = mbar_wait_warp(bar(kBarQEmpty), (segs - 1) & 1, abort);
          if (ok && lane == 0) {
            // only tiles that hold tokens are loaded (and computed)
            const int nx = kQT == 2 && sg.b.tokens > tpt ? 2 : 1;
            const uint32_t box_bytes = static_cast<uint32_t>(a.group * tpt) * 128u;
            mbar_arrive_expect_tx(bar(kBarQFull), nx * kHalves * box_bytes);
            for (int x = 0; x < nx; ++x)
#pragma unroll
              for (int h = 0; h < kHalves; ++h)
                tma_load_3d(sbase + S::kQ + static_cast<uint32_t>(x * S::kQBytes + h * (kM * 128)),
                            &q_map, h * 64, kvh * a.group, sg.b.t_base + x * tpt, bar(kBarQFull));
          }
          __syncwarp();
          if (!ok) break;
        }
        ++segs;
        for (uint32_t w = first; w < n_units; w += kProducerWarps) {
          const int j = static_cast<int>(w >> 1), c = static_cast<int>(w & 1);
          const uint32_t u = u0 + w;
          const int key0 = tile_key<kRules>(sg.b.walk, sg.tile0 + j);
          long long cur[kGroups];
#pragma unroll
          for (int g = 0; g < kGroups; ++g) cur[g] = first_row(j, g, next[g]);
          if (w + kProducerWarps < n_units)
            load_entries(static_cast<int>((w + kProducerWarps) >> 1), next);
          const int st = static_cast<int>(u % kSlots);
          if (u >= kSlots &&
              !(ok = mbar_wait_warp(bar(kBarEmpty + st), ((u / kSlots) - 1) & 1, abort)))
            break;
          const uint32_t dst = sbase + S::kRing + st * S::kSlotBytes;
          const __nv_bfloat16 *plane = (c ? a.v_plane : a.k_plane) + head_off;
          if (kTma) {
            // boxes of live keys by TMA; the box of the last key and those
            // behind it (and bad pages) row by row, zeros where nothing is
            const int b_lane = lane * box;
            const bool in_tile = b_lane < kN;
            // (under rules, boxes with rows that no token sees are not live)
            const bool live = in_tile && cur[0] >= 0 && key0 + b_lane + box <= sg.b.seq &&
                              (kRules == 0 || key0 + b_lane >= sg.b.lo ||
                               key0 + b_lane + box <= sg.b.prefix);
            const unsigned live_mask = __ballot_sync(0xffffffffu, live);
            unsigned rest = __ballot_sync(0xffffffffu, in_tile && !live);
            if (lane == 0)
              mbar_expect_tx(bar(kBarFull + st),
                             static_cast<uint32_t>(__popc(live_mask) * box * D * 2));
            __syncwarp();
            if (live) {
#pragma unroll
              for (int h = 0; h < kHalves; ++h)
                tma_load_2d_hint(dst + static_cast<uint32_t>(h * (kN * 128) + b_lane * 128),
                                 c ? &v_map : &k_map, kvh * D + h * 64, static_cast<int>(cur[0]),
                                 bar(kBarFull + st), kv_policy);
            }
            const bool copied = rest != 0;
            while (rest) {
              const int src = __ffs(rest) - 1;
              rest &= rest - 1;
              const long long s0 = __shfl_sync(0xffffffffu, cur[0], src);
              for (int r = lane / kChunks; r < box; r += kKeysPerInstr) {
                const int kk = src * box + r;
                const bool in = s0 >= 0 && key0 + kk < sg.b.seq &&
                                (kRules == 0 || key0 + kk >= sg.b.lo || key0 + kk < sg.b.prefix);
                cp_async_16(dst + sw128_offset(kN, kk, ch * 8),
                            in ? plane + (s0 + r) * row_elems + ch * 8 : plane, in ? 16 : 0);
              }
            }
            if (copied) {  // landed, and visible to tcgen05.mma, before the arrival
              cp_async_wait_all();
              fence_async_shared();
            }
            mbar_arrive(bar(kBarFull + st));
          } else {
            // A lane knows the rows of four of the tile's keys; each copy takes
            // its row's address from the lane that does. Eight addresses are
            // exchanged before their copies: a copy keeps its place in the
            // program, a shuffle between two would delay the second.
            constexpr int kCopies = 32 / kKeysPerInstr;
            constexpr int kAhead = 8;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
              const bool in = cur[g] >= 0;
              const unsigned mask = __ballot_sync(0xffffffffu, in) >> (lane / kChunks);
              const uint64_t row_at =
                  reinterpret_cast<uint64_t>(in ? plane + cur[g] * row_elems : plane);
#pragma unroll
              for (int i0 = 0; i0 < kCopies; i0 += kAhead) {
                uint64_t src[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                  src[i] = __shfl_sync(0xffffffffu, row_at,
                                       (i0 + i) * kKeysPerInstr + lane / kChunks) +
                           ch * 16;
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                  cp_async_16_hint(
                      dst + sw128_offset(kN, g * 32 + (i0 + i) * kKeysPerInstr + lane / kChunks,
                                         ch * 8),
                      reinterpret_cast<const void *>(src[i]),
                      (mask >> ((i0 + i) * kKeysPerInstr)) & 1u ? 16 : 0, kv_policy);
              }
            }
          }
          if (!kTma) cp_async_mbar_arrive(bar(kBarFull + st));
          issued = u + 1;
        }
        u0 += n_units;
      }
      if (!ok) *abort = 1;
      cp_async_wait_all();
      if (*abort && lane == 0) {
        // every TMA copy this warp issued lands before the CTA can exit
        int never = 0;
        if (pw == 0 && segs > 0) mbar_wait(bar(kBarQFull), (segs - 1) & 1, &never);
        if (kTma)
          for (uint32_t t = issued > kSlots ? issued - kSlots : 0; t < issued; ++t)
            if (t % kProducerWarps == static_cast<uint32_t>(pw))
              mbar_wait(bar(kBarFull + t % kSlots), (t / kSlots) & 1, &never);
      }
    } else {
      // ------------------------------------------------------------ MMA issuer
      const bool issuer = elect_one();
      constexpr uint32_t idesc_qk = umma_idesc_bf16(kM, kN, 0, 0);
      constexpr uint32_t idesc_pv = umma_idesc_bf16(kM, D, 0, 1);
      const uint64_t dq0 = umma_desc_sw128(sbase + S::kQ, 16, 1024);
      const uint64_t dk0 = umma_desc_sw128(sbase + S::kRing, 16, 1024);
      const uint64_t dv0 = umma_desc_sw128(sbase + S::kRing, kN * 128, 1024);
      auto kstep = [](int ks) -> uint64_t {
        return static_cast<uint64_t>(((ks >> 2) * (kN * 128) + (ks & 3) * 32) >> 4);
      };
      auto slot_step = [](uint32_t u) -> uint64_t {
        return static_cast<uint64_t>((u % kSlots) * (S::kSlotBytes >> 4));
      };
      auto qk = [&](int x, int buf, uint32_t u) {  // scores of query tile x, K in unit u
        const uint64_t dq = dq0 + static_cast<uint64_t>((x * S::kQBytes) >> 4);
        const uint64_t dk = dk0 + slot_step(u);
        if (issuer) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            umma_bf16_ss(tmem + kTmemS + buf * kN, dq + kstep(ks), dk + kstep(ks), idesc_qk,
                         ks > 0 ? 1u : 0u);
          umma_commit(bar(kBarSFull + buf));
        }
      };
      auto pv = [&](int x, int buf, uint32_t u, bool first) {  // O_x (+)= P V, V in unit u
        const uint64_t dv = dv0 + slot_step(u);
        if (issuer) {
#pragma unroll
          for (int ks = 0; ks < kN / 16; ++ks)
            umma_bf16_ts(tmem + kTmemO + x * kN, tmem + kTmemS + buf * kN + ks * 8,
                         dv + ks * (2048 >> 4), idesc_pv, (!first || ks > 0) ? 1u : 0u);
        }
      };
      auto commit = [&](int i) {
        if (issuer) umma_commit(bar(i));
      };
      auto wait_unit = [&](uint32_t u) {
        const bool r = mbar_wait_uniform(bar(kBarFull + u % kSlots), (u / kSlots) & 1, abort);
        if (!kTma) fence_async_shared();  // cp.async wrote it, tcgen05.mma reads it
        tc_fence_after_sync();
        return r;
      };
      auto free_unit = [&](uint32_t u) { commit(kBarEmpty + static_cast<int>(u % kSlots)); };
      uint32_t u0 = 0;                // ring unit of the segment's first K tile
      uint32_t np0 = 0, np1 = 0;      // P tiles taken from score buffers 0 and 1
      uint32_t uses0 = 0, uses1 = 0;  // segments that used O_0, O_1
      int segs = 0;
      bool ok = true;
      while (ok && next_segment<kQT, kRules>(a, blocks, walk, sg)) {
        const int n = sg.n;
        if (!(ok = mbar_wait_uniform(bar(kBarQFull), segs & 1, abort))) break;
        ++segs;
        // One query tile: key tiles alternate between the score buffers, and
        // (two-tile kernel) between the softmax groups and their O.
        const bool alternate = kQT == 1 || shared_tile(a, sg);
        if (alternate) {
          for (int j = 0; ok && j < 2 && j < n; ++j) {
            if (!(ok = wait_unit(u0 + 2 * j))) break;
            qk(0, j, u0 + 2 * j);
            free_unit(u0 + 2 * j);
          }
          if (n <= 2 && ok) commit(kBarQEmpty);
          for (int j = 0; ok && j < n; ++j) {
            const int buf = j & 1;
            const int x = kQT == 2 ? buf : 0;
            uint32_t &np = buf ? np1 : np0;
            const uint32_t uses = x ? uses1 : uses0;
            const bool first = j <= x;  // of O_x
            if (first && uses > 0 &&
                !(ok = mbar_wait_uniform(bar(kBarOEmpty + x), (uses - 1) & 1, abort)))
              break;
            if (!(ok = mbar_wait_uniform(bar(kBarPFull + buf), np & 1, abort) &&
                       wait_unit(u0 + 2 * j + 1)))
              break;
            ++np;
            pv(x, buf, u0 + 2 * j + 1, first);
            free_unit(u0 + 2 * j + 1);
            if (kQT == 1) commit(kBarPvDone);
            if (kQT == 2 && j + 2 >= n) commit(kBarOFull + x);
            if (j + 2 < n) {
              if (!(ok = wait_unit(u0 + 2 * (j + 2)))) break;
              qk(0, buf, u0 + 2 * (j + 2));
              free_unit(u0 + 2 * (j + 2));
              if (j + 3 == n) commit(kBarQEmpty);
            }
          }
          if (kQT == 1 && ok) commit(kBarOFull);
          ++uses0;
          if (kQT == 2) ++uses1;
        } else {
          const int n0 = tiles_of<kRules>(a, sg, tpb, 0), n1 = tiles_of<kRules>(a, sg, tpb, 1);
          // score tile j of both query tiles, for those that walk it
          if (!(ok = wait_unit(u0))) break;
          if (n0 > 0) qk(0, 0, u0);
          if (n1 > 0) qk(1, 1, u0);
          free_unit(u0);
          if (n == 1) commit(kBarQEmpty);
          for (int j = 0; ok && j < n; ++j) {
            const uint32_t uk = u0 + 2 * (j + 1), uv = u0 + 2 * j + 1;
            const bool next = j + 1 < n;
            if (!(ok = wait_unit(uv))) break;
            if (j < n0) {
              if (j == 0 && uses0 > 0 &&
                  !(ok = mbar_wait_uniform(bar(kBarOEmpty), (uses0 - 1) & 1, abort)))
                break;
              if (!(ok = mbar_wait_uniform(bar(kBarPFull), np0 & 1, abort))) break;
              tc_fence_after_sync();
              ++np0;
              pv(0, 0, uv, j == 0);
              if (j == n0 - 1) commit(kBarOFull);
            }
            if (next && !(ok = wait_unit(uk))) break;
            if (next && j + 1 < n0) qk(0, 0, uk);
            if (j < n1) {
              if (j == 0 && uses1 > 0 &&
                  !(ok = mbar_wait_uniform(bar(kBarOEmpty + 1), (uses1 - 1) & 1, abort)))
                break;
              if (!(ok = mbar_wait_uniform(bar(kBarPFull + 1), np1 & 1, abort))) break;
              tc_fence_after_sync();
              ++np1;
              pv(1, 1, uv, j == 0);
              if (j == n1 - 1) commit(kBarOFull + 1);
            }
            free_unit(uv);
            if (next) {
              if (j + 1 < n1) qk(1, 1, uk);
              free_unit(uk);
            }
            if (j + 2 == n) commit(kBarQEmpty);
          }
          if (n0 > 0) ++uses0;
          if (n1 > 0) ++uses1;
        }
        u0 += 2 * static_cast<uint32_t>(n);
      }
      if (!ok) {
        *abort = 1;
        flag_error(a.err, kErrTimeout);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    if constexpr (kQT == 2) warpgroup_registers_inc<kSoftmaxRegs>();
    const int quarter = warp & 3;
    const int x = kQT == 2 ? warp >> 2 : 0;
    const int r = quarter * 32 + lane;  // row of the query tile == TMEM lane
    const int tt = r / a.group;         // token within the query tile
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t sbuf = tmem + lane_base + kTmemS + (kQT == 2 ? x * kN : 0);
    const uint32_t orow_t = tmem + lane_base + kTmemO + x * kN;
    uint32_t ns0 = 0, ns1 = 0;  // score tiles taken (per buffer with one query tile)
    uint32_t pv_tiles = 0;      // tiles before this segment (one query tile)
    uint32_t uses[2] = {0, 0};  // segments that used O_0, O_1
    uint32_t states = 0;        // shared query tiles so far
    bool ok = true;
    for (;;) {
      // The segment, looked at here for what the tile loop needs and loaded
      // again after it (a cache hit), so that a thread holding a whole score
      // row holds little else across the loop.
      Walk ahead_of = walk;
      if (!next_segment<kQT, kRules>(a, blocks, ahead_of, sg)) break;
      const bool shared = kQT == 2 && shared_tile(a, sg);
      const int xq = shared ? 0 : x;  // query tile
      const int n_x = kQT == 1 ? sg.n : tiles_of<kRules>(a, sg, tpb, x);
      const int first_draft = sg.b.p;  // tree
      // rules: last key (but for the prefix) of the tile's first token, of this row
      const int min_limit = sg.b.p + sg.b.sub * tpb + xq * tpt;
      const bool row_valid = tt < tpt && xq * tpt + tt < sg.b.tokens;
      const int limit = min_limit + (row_valid ? tt : 0);
      const int prefix = kRules != 0 ? sg.b.prefix : 0;
      const TileWalk tiles = kRules != 0 ? sg.b.walk : TileWalk{0, 0};
      // this group's tile j is tile first_tile + j * step of the block
      const int first_tile = sg.tile0 + (shared ? x : 0), step = shared ? 2 : 1;
      float slope = 0.f;  // of this row's head, log2 units per key
      if constexpr (kBias) slope = a.rules.alibi_slopes[kvh * a.group + r % a.group] * kLog2e;
      // This row's ancestors (bit i: drafted key i), if the segment reaches
      // the drafted keys. Every warp writes the request's parents (the same
      // ones) and reads back what it wrote; the group's other warps are done
      // with the last ones, since they were all waited for at that segment's
      // end (its final O takes every warp's P).
      uint32_t anc[kMaskWords];
#pragma unroll
      for (int w = 0; w < kMaskWords; ++w) anc[w] = 0;
      if (kRules == 0 && n_x > 0 && (sg.tile0 + sg.n) * kN > first_draft) {
        __syncwarp();  // the previous segment's are read
        for (int i = lane; i < sg.b.c; i += 32) {
          int par = a.parents[sg.b.t_base - sg.b.sub * tpb + i];
          if (par < -1 || par >= i) {  // not an earlier token: taken as a root
            flag_error(a.err, kErrTree);
            par = -1;
          }
          s_parents[x][i] = static_cast<uint8_t>(par < 0 ? 255 : par);
        }
        __syncwarp();
        if (row_valid) {
          // a parent is an earlier token: at most c steps (token 255 is
          // nobody's parent, so 255 can stand for the root)
          for (int i = sg.b.sub * tpb + xq * tpt + tt;;) {
#pragma unroll
            for (int w = 0; w < kMaskWords; ++w) anc[w] |= (i >> 5) == w ? 1u << (i & 31) : 0u;
            i = s_parents[x][i];
            if (i == 255) break;
          }
        }
        __syncwarp();
      }
      float m_used = -INFINITY, l = 0.f;
      for (int j = 0; ok && j < n_x; ++j) {
        const int buf = kQT == 1 ? (j & 1) : x;
        const uint32_t srow = sbuf + (kQT == 1 ? buf * kN : 0);
        uint32_t &ns = (kQT == 1 && buf) ? ns1 : ns0;
        if (!(ok = mbar_wait_warp(bar(kBarSFull + buf), ns & 1, abort))) break;
        ++ns;
        tc_fence_after_sync();
        float v[kN], mx0, mx1, mx2, mx3;
        if constexpr (kCap) {
          tmem_ld32_absmax(srow + 0, *reinterpret_cast<float(*)[32]>(&v[0]), mx0);
          tmem_ld32_absmax(srow + 32, *reinterpret_cast<float(*)[32]>(&v[32]), mx1);
          tmem_ld32_absmax(srow + 64, *reinterpret_cast<float(*)[32]>(&v[64]), mx2);
          tmem_ld32_absmax(srow + 96, *reinterpret_cast<float(*)[32]>(&v[96]), mx3);
        } else {
          tmem_ld32_max(srow + 0, *reinterpret_cast<float(*)[32]>(&v[0]), mx0);
          tmem_ld32_max(srow + 32, *reinterpret_cast<float(*)[32]>(&v[32]), mx1);
          tmem_ld32_max(srow + 64, *reinterpret_cast<float(*)[32]>(&v[64]), mx2);
          tmem_ld32_max(srow + 96, *reinterpret_cast<float(*)[32]>(&v[96]), mx3);
        }
        tmem_ld_wait();
        const int key0 = tile_key<kRules>(tiles, first_tile + j * step);
        // keys that some row may not see (uniform over the CTA or the group)
        const bool ahead = key0 + kN > (kRules == 0 ? first_draft : min_limit + 1);
        bool masked = ahead;
        bool near = false;    // rules: scores computed within the exponential's argument
        float row_add = 0.f;  // rules: what v, or the near form, leaves out of the row's scores
        float mul = a.scale_log2;
        if constexpr (kRules != 0) {
          const int window = a.rules.window;
          if (window > 0 && key0 < min_limit + tpt - window) masked = true;
          if (key0 + kN <= prefix) masked = false;
        }
        if constexpr (kCap || kBias) {
          const float top = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
          bool row_near = a.q_mode == 0;
          if constexpr (kCap) row_near = row_near && top <= a.rules.near;
          if constexpr (kBias) row_near = row_near && fabsf(slope) <= kNearBias / 31.f;
          near = !masked && !(kBias && ahead) && __all_sync(0xffffffffu, row_near);
          if (near) {
            const float k = kCap ? a.rules.c1 : a.scale_log2;
            if constexpr (kBias) {
              row_add = -slope * static_cast<float>(limit - key0);
              const float hi = fmaxf(slope * 31.f, 0.f);  // within a load's 32 columns
              mx0 = fmaf(mx0, k, hi);
              mx1 = fmaf(mx1, k, hi + slope * 32.f);
              mx2 = fmaf(mx2, k, hi + slope * 64.f);
              mx3 = fmaf(mx3, k, hi + slope * 96.f);
            } else {
              mx0 *= k;
              mx1 *= k;
              mx2 *= k;
              mx3 *= k;
            }
          }
        }
        if (masked || a.q_mode || ((kCap || kBias) && !near)) {
          // (a cap is odd: what it makes of a score changes sign with it)
          if constexpr (kCap)
            cap_scores(v, fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)), a.rules,
                       [&](auto f) { tmem_map128(srow, v, f); });
          if (a.q_mode) {
#pragma unroll
            for (int cc = 0; cc < kN; ++cc) v[cc] = a.q_mode == 1 ? -v[cc] : 0.f;
          }
          if constexpr (kCap || kBias) {
            if constexpr (kBias)
              row_add = bias_scores<kCap>(v, a.scale_log2, slope, limit - key0, ahead);
            mul = 1.f;
          }
          if (kRules != 0 && masked) {
            // column cc is seen if lo <= cc <= hi or cc < pre
            const int hi = limit - key0;
            const int lo = a.rules.window > 0 ? hi - a.rules.window + 1 : -key0;
            const int pre = prefix - key0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t seen = seen_bits(lo, hi, pre, w);
#pragma unroll
              for (int cc = 0; cc < 32; ++cc)
                v[32 * w + cc] = (seen >> cc) & 1u ? v[32 * w + cc] : -INFINITY;
            }
          }
          if (kRules == 0 && masked) {
            // word w: the visible ones of columns 32 w .. 32 w + 31
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int d0 = key0 + 32 * w - first_draft;  // drafted index of its first column
              uint32_t vis;
              if (d0 < 0) {
                vis = d0 <= -32 ? 0xffffffffu : (anc[0] << -d0) | ((1u << -d0) - 1u);
              } else {
                uint32_t lo = 0, hi = 0;
#pragma unroll
                for (int q = 0; q < kMaskWords; ++q) {
                  lo = (d0 >> 5) == q ? anc[q] : lo;
                  hi = (d0 >> 5) + 1 == q ? anc[q] : hi;
                }
                vis = __funnelshift_r(lo, hi, d0 & 31);
              }
#pragma unroll
              for (int cc = 0; cc < 32; ++cc)
                v[32 * w + cc] = (vis >> cc) & 1u ? v[32 * w + cc] : -INFINITY;
            }
          }
          mx0 = fmaxf(v[0], v[1]);
          mx1 = fmaxf(v[2], v[3]);
          mx2 = fmaxf(v[4], v[5]);
          mx3 = fmaxf(v[6], v[7]);
#pragma unroll
          for (int cc = 8; cc < kN; cc += 8) {
            mx0 = max3f(mx0, v[cc], v[cc + 1]);
            mx1 = max3f(mx1, v[cc + 2], v[cc + 3]);
            mx2 = max3f(mx2, v[cc + 4], v[cc + 5]);
            mx3 = max3f(mx3, v[cc + 6], v[cc + 7]);
          }
        }
        float mt = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
        if constexpr (!kCap && !kBias) mt *= a.scale_log2;
        if constexpr (kBias) mt += row_add;
        // Lazy rescale, warp-uniform, as in extend.cu: O moves to a new
        // reference only when a row's max grew by more than 2^8.
        const bool rescale = j > 0 && __any_sync(0xffffffffu, mt > m_used + kRescaleThreshold);
        float f = 1.f;
        if (j == 0) {
          m_used = mt;
        } else if (rescale) {
          const float m_new = fmaxf(m_used, mt);
          f = m_used == -INFINITY ? 0.f : fast_exp2(m_used - m_new);
          m_used = m_new;
        }
        const float nm = (m_used == -INFINITY ? 0.f : -m_used) + row_add;
        float sa0 = 0.f, sa1 = 0.f, sb0 = 0.f, sb1 = 0.f;
        // P: exp2 of arg(cc), in pairs; to bf16 (half a step, 2^-8 relative, per key)
        auto exponentials = [&](auto arg) {
#pragma unroll
          for (int cc = 0; cc < kN; cc += 32) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float y0, y1;
              arg(cc + 2 * e, y0, y1);
              y0 = fast_exp2(y0);
              y1 = fast_exp2(y1);
              if (e & 1)
                add2(sb0, sb1, y0, y1);
              else
                add2(sa0, sa1, y0, y1);
              w[e] = pack_bf16(y0, y1);
            }
            tmem_st16u(srow + cc / 2, w);
          }
        };
        if constexpr (kCap || kBias) {
          if (near)
            exponentials([&](int cc, float &y0, float &y1) {
              near_pair<kCap, kBias>(v[cc], v[cc + 1], cc, a.scale_log2, slope, nm, a.rules, y0,
                                     y1);
            });
          else
            exponentials([&](int cc, float &y0, float &y1) {
              fma2(y0, y1, v[cc], v[cc + 1], mul, nm);
            });
        } else {
          exponentials([&](int cc, float &y0, float &y1) {
            fma2(y0, y1, v[cc], v[cc + 1], a.scale_log2, nm);
          });
        }
        l = l * f + ((sa0 + sa1) + (sb0 + sb1));
        if (rescale) {
          // O_x is stable once P V(j - 1) is done: with two query tiles it
          // was issued before S(j); with one, its own barrier says so.
          if (kQT == 1 &&
              !(ok = mbar_wait_warp(bar(kBarPvDone), (pv_tiles + j - 1) & 1, abort)))
            break;
          tc_fence_after_sync();
#pragma unroll 1
          for (int cb = 0; cb < D / 32; ++cb) {
            float o[32];
            tmem_ld32(orow_t + cb * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 32; ++q) o[q] *= f;
            tmem_st32(orow_t + cb * 32, o);
          }
        }
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(bar(kBarPFull + buf));
      }
      if (!ok) break;
      next_segment<kQT, kRules>(a, blocks, walk, sg);  // the same one
      const int n_other = kQT == 1 ? 0 : tiles_of<kRules>(a, sg, tpb, 1 - x);
      const int tok = xq * tpt + tt;  // token within the block
      const bool valid = tt < tpt && tok < sg.b.tokens;
      pv_tiles += static_cast<uint32_t>(sg.n);
      if (n_x > 0) {
        if (!(ok = mbar_wait_warp(bar(kBarOFull + x), uses[x] & 1, abort))) break;
        ++uses[x];
      }
      float f0 = 1.f, f1 = 0.f;  // factors of O_0 (this group's) and O_1
      if (kQT == 2) {
        if (shared && x == 1) {
          // O_1 and its state are the first group's to join, and to hand back
          s_state[r] = make_float2(m_used, l);
          tc_fence_before_sync();
          mbar_arrive(bar(kBarState));
          if (n_other > 0) ++uses[0];
          ++states;
          continue;
        }
        if (shared) {
          if (!(ok = mbar_wait_warp(bar(kBarState), states & 1, abort) &&
                     mbar_wait_warp(bar(kBarOFull + 1), uses[1] & 1, abort)))
            break;
          ++states;
          const float2 st = s_state[r];
          const float m = fmaxf(m_used, st.x);
          const float ref = m == -INFINITY ? 0.f : m;
          f0 = fast_exp2(m_used - ref);
          f1 = fast_exp2(st.x - ref);
          l = l * f0 + st.y * f1;
          m_used = m;
        }
        if (n_other > 0) ++uses[1 - x];
      }
      if (n_x > 0) tc_fence_after_sync();
      // A query tile whose tokens see none of the segment's tiles (n_x = 0)
      // still owes its part of a shared block: o = 0, lse = -inf.
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const float lse = l == 0.f ? -INFINITY : (m_used + __log2f(l)) * kLn2;
      f0 *= inv;
      f1 *= inv;
      const int h = kvh * a.group + r % a.group;
      const int64_t orow = static_cast<int64_t>(valid ? sg.b.t_base + tok : 0) * a.hq + h;
      constexpr int kRows = kQT * kM;
      const int64_t part = static_cast<int64_t>(sg.slot) * a.hkv + kvh;
      float4 *po = reinterpret_cast<float4 *>(a.part_o) + part * (D / 4) * kRows + xq * kM + r;
      // O's columns, all at once where the registers hold them: one round trip
      constexpr int kO = kQT == 1 ? D : 32;
#pragma unroll 1
      for (int cb = 0; cb < D / kO; ++cb) {
        float o[kO];
        if (n_x > 0) {
#pragma unroll
          for (int q = 0; q < kO / 32; ++q)
            tmem_ld32(orow_t + cb * kO + q * 32, *reinterpret_cast<float(*)[32]>(&o[q * 32]));
          if (kQT == 2 && shared) {
            float o1[32];
            tmem_ld32(orow_t + kN + cb * 32, o1);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 32; ++q) o[q] = o[q] * f0 + o1[q] * f1;
          } else {
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < kO; ++q) o[q] *= f0;
          }
        } else {
#pragma unroll
          for (int q = 0; q < kO; ++q) o[q] = 0.f;
        }
        if (valid) {
          if (sg.whole) {
            uint4 *dst = reinterpret_cast<uint4 *>(a.o + orow * D + cb * kO);
#pragma unroll
            for (int q = 0; q < kO / 8; ++q)
              dst[q] = make_uint4(pack_bf16(o[8 * q], o[8 * q + 1]),
                                  pack_bf16(o[8 * q + 2], o[8 * q + 3]),
                                  pack_bf16(o[8 * q + 4], o[8 * q + 5]),
                                  pack_bf16(o[8 * q + 6], o[8 * q + 7]));
          } else {
#pragma unroll
            for (int q = 0; q < kO / 4; ++q)
              po[(cb * (kO / 4) + q) * kRows] =
                  make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          }
        }
        // tcgen05.ld wants the whole warp: without this barrier the compiler
        // may split the loop by `valid` and issue it from part of one
        __syncwarp();
      }
      if (valid) {
        if (!sg.whole)
          a.part_lse[part * kRows + xq * kM + r] = lse;
        else if (a.lse)
          a.lse[orow] = lse;
      }
      if (n_x > 0) {
        tc_fence_before_sync();
        mbar_arrive(bar(kBarOEmpty + x));
        if (shared) mbar_arrive(bar(kBarOEmpty + 1));
      }
    }
    if (!ok) {
      *abort = 1;
      flag_error(a.err, kErrTimeout);
    }
  }

  // Teardown: every role has left its loop; free TMEM once no MMA is in flight.
  if (warp == kMmaWarp && __any_sync(0xffffffffu, *abort != 0)) {
    if (elect_one()) {  // the lane that issued them
      umma_commit(bar(kBarTeardown));
      int never = 0;
      mbar_wait(bar(kBarTeardown), 0, &never);
    }
    __syncwarp();
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Merge of the blocks that more than one group computed: o = sum e^(lse_s -
// lse) o_s. One CTA per (block, kv head, 32 rows), eight warps with D / 8
// columns each; lane = row, so the states' [column group][row] layout is read
// in whole lines. States are taken kBatch at a time, all their loads together,
// with a running maximum: one round trip to L2 for the usual two.
constexpr int kMergeThreads = 256;

template <int D, int kQT>
__global__ void __launch_bounds__(kMergeThreads) direct_merge_kernel(const DirectArgs a) {
  constexpr int kRows = kQT * kM;
  constexpr int kCols = D / 4 / (kMergeThreads / 32);  // float4 columns per warp
  constexpr int kBatch = 2;
  const int b = blockIdx.x;
  grid_dependency_wait();
  const int4 e = a.table[b];  // first and last group, first token, tokens
  if (e.x < 0) return;
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int kvh = blockIdx.y;
  const int row = blockIdx.z * kMergeRows + lane;  // of the block's query tiles
  const int tt = (row % kM) / a.group;
  const int tok = (row / kM) * a.tokens_per_tile + tt;
  if (tt >= a.tokens_per_tile || tok >= e.w) return;
  // state s: slot 2 g + 1 of the block's first group, then 2 g of each further one
  const int n = e.y - e.x + 1;
  float m = -INFINITY, l = 0.f;
  float4 o[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < n; s0 += kBatch) {
    float lse[kBatch];
    float4 v[kBatch][kCols];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int s = s0 + u;
      const int64_t part = static_cast<int64_t>(2 * (e.x + s) + (s == 0 ? 1 : 0)) * a.hkv + kvh;
      const float4 *po = reinterpret_cast<const float4 *>(a.part_o) + part * (D / 4) * kRows +
                         static_cast<int64_t>(warp * kCols) * kRows + row;
      lse[u] = s < n ? a.part_lse[part * kRows + row] : -INFINITY;
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        v[u][c] = s < n ? po[c * kRows] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float mx = m;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) mx = fmaxf(mx, lse[u]);
    const float ref = mx == -INFINITY ? 0.f : mx;
    const float f = expf(m - ref);
    m = mx;
    l *= f;
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      o[c].x *= f;
      o[c].y *= f;
      o[c].z *= f;
      o[c].w *= f;
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const float w = expf(lse[u] - ref);
      l += w;
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        o[c].x += w * v[u][c].x;
        o[c].y += w * v[u][c].y;
        o[c].z += w * v[u][c].z;
        o[c].w += w * v[u][c].w;
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t orow =
      static_cast<int64_t>(e.z + tok) * a.hq + kvh * a.group + (row % kM) % a.group;
  uint2 *dst = reinterpret_cast<uint2 *>(a.o + orow * D) + warp * kCols;
#pragma unroll
  for (int c = 0; c < kCols; ++c)
    dst[c] = make_uint2(pack_bf16(o[c].x * inv, o[c].y * inv),
                        pack_bf16(o[c].z * inv, o[c].w * inv));
  if (warp == 0 && a.lse) a.lse[orow] = l == 0.f ? -INFINITY : m + logf(l);
}

// The kernel and, where a block can be shared by groups, the merge.
template <int D, int kQT, bool kTma, int kRules>
cudaError_t launch(const DirectArgs &a, const CUtensorMap &km, const CUtensorMap &vm,
                   const CUtensorMap &qm, cudaStream_t stream) {
  using S = DirectSmem<D, kQT>;
  if constexpr (kQT == 2) {
    // the register split waits forever if the launch has fewer than it hands out
    static const bool enough = [] {
      cudaFuncAttributes at{};
      return cudaFuncGetAttributes(&at, direct_kernel<D, kQT, kTma, kRules>) == cudaSuccess &&
             3 * at.numRegs >= 2 * kSoftmaxRegs + kOtherRegs;
    }();
    if (!enough) return cudaErrorInvalidConfiguration;
  }
  cudaError_t e = cudaFuncSetAttribute(direct_kernel<D, kQT, kTma, kRules>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, S::kTotal);
  if (e != cudaSuccess) return e;
  const dim3 grid(a.hkv, a.groups), block((4 * kQT + 1 + producer_warps(kQT, kTma)) * 32);
  e = launch_pdl(direct_kernel<D, kQT, kTma, kRules>, grid, block, S::kTotal, stream, km, vm, qm,
                 a);
  if (e != cudaSuccess || a.groups == 1 || a.whole) return e;
  const dim3 mgrid(a.max_blocks, a.hkv, kQT * kM / kMergeRows);
  return launch_pdl(direct_merge_kernel<D, kQT>, mgrid, dim3(kMergeThreads), 0, stream, a);
}

// In key tiles: what the search for a share, the partial states and the second
// kernel cost a call (about 6 us), and what a further block in a share costs it.
constexpr int share_cost(int tiles_per_block) { return tiles_per_block == 1 ? 8 : 6; }
constexpr int kFurtherBlock = 8;

// Groups of a call of at most `blocks` query blocks, each of at most
// block_tiles key tiles, and max_seq keys, and the workspace for partial states
// and the block table (0 if nothing can be shared; the same whether the call
// shares or not, so that it grows with the sizes).
//
// A group for each block, or equal shares? The longest block's tiles against a
// share's, about half of blocks * tiles / groups (lengths are ragged, the bound
// is the longest). Per call, 32/8 heads of 128, page size 1, a group for each
// block / shared: 1 request of 520 keys, 8 drafts 11.2 / 13.6 us, of 900 14.7 /
// 16.2, of 1400 17.3 / 15.4; 16 of up to 2000 25.1 / 30.2, of 2900 31.4 / 31.6;
// 64 drafts: 1 of 520 17.8 / 18.8, of 900 22.2 / 20.6; 16 of up to 2000 38.4 /
// 39.2, of 2900 47.7 / 37.5.
inline DirectPlan plan(int32_t blocks, int32_t query_tiles, int32_t tiles_per_block, int32_t hkv,
                       int32_t d, int32_t max_seq, int64_t block_tiles, int32_t sm_count) {
  DirectPlan p{};
  p.query_tiles = query_tiles;
  p.tiles_per_block = tiles_per_block;
  p.max_blocks = blocks;
  // one group per Hkv SMs, and no more than there are smallest shares
  const int64_t all = std::max<int64_t>(1, (sm_count > 0 ? sm_count : 1) / hkv);
  const int64_t tiles =
      static_cast<int64_t>(blocks) * ((static_cast<int64_t>(max_seq) + kN - 1) / kN);
  const int64_t groups =
      std::min<int64_t>(all, std::max<int64_t>(1, (tiles + kMinTiles - 1) / kMinTiles));
  p.groups = static_cast<int32_t>(groups);
  if (groups > 1) {
    const size_t rows = static_cast<size_t>(2 * groups) * hkv * query_tiles * kM;
    p.lse_offset = rows * d * sizeof(float);
    p.table_offset = (p.lse_offset + rows * sizeof(float) + 255) & ~size_t(255);
    p.workspace_bytes = p.table_offset + sizeof(int4) * static_cast<size_t>(blocks);
  }
  if (blocks <= all &&
      2 * all * (block_tiles - share_cost(tiles_per_block)) <=
          blocks * (block_tiles + kFurtherBlock)) {
    p.whole = 1;
    p.groups = blocks;
  }
  return p;
}

// The arguments that both uses share, and the tensor maps. false: a map could
// not be made. *tma: K/V by TMA boxes.
inline bool direct_args(DirectArgs *out, CUtensorMap *km, CUtensorMap *vm, CUtensorMap *qm,
                        bool *tma, const PoolGeom &g, int32_t layer, const void *q,
                        const int32_t *qo_indptr, void *o, float *lse, const int32_t *page_table,
                        int64_t table_stride, const int32_t *table_idx, const int32_t *seq_lens,
                        int32_t batch, int32_t total_q, int32_t hq, float scale,
                        const DirectPlan &plan, void *workspace, unsigned *err) {
  DirectArgs a{};
  a.k_plane = static_cast<const __nv_bfloat16 *>(g.base) + static_cast<int64_t>(layer) * g.plane;
  a.v_plane = a.k_plane + static_cast<int64_t>(g.num_layers) * g.plane;
  a.slots = g.slots;
  a.page_size = g.page_size;
  a.hkv = g.hkv;
  a.qo_indptr = qo_indptr;
  a.o = static_cast<__nv_bfloat16 *>(o);
  a.lse = lse;
  a.page_table = page_table;
  a.table_stride = table_stride;
  a.table_idx = table_idx;
  a.seq_lens = seq_lens;
  a.batch = batch;
  a.total_q = total_q;
  a.hq = hq;
  a.group = hq / g.hkv;
  a.tokens_per_tile = kM / a.group;
  a.tokens_per_block = plan.tiles_per_block * a.tokens_per_tile;
  a.max_blocks = plan.max_blocks;
  a.groups = plan.groups;
  a.whole = plan.whole;
  a.cost = tile_cost(g.d);
  a.q_mode = scale > 0.f ? 0 : (scale < 0.f ? 1 : 2);
  a.scale_log2 = scale > 0.f ? scale * kLog2e : (scale < 0.f ? -scale * kLog2e : kLog2e);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  a.part_o = reinterpret_cast<float *>(ws);
  a.part_lse = reinterpret_cast<float *>(ws + plan.lse_offset);
  a.table = reinterpret_cast<int4 *>(ws + plan.table_offset);
  a.err = err;
  // K/V boxes: the largest power of two that divides the page size, 8 to 128
  // rows (8: the swizzle's period; a tensor's rows are counted in 32 bits).
  int32_t box = 1;
  while (box < kN && g.page_size % (2 * box) == 0) box *= 2;
  *tma = box >= 8 && g.slots < (int64_t(1) << 31);
  a.box = box;
  const uint64_t cols = static_cast<uint64_t>(g.hkv) * g.d;
  *out = a;
  if (*tma && (!tensor_map_rows(km, a.k_plane, static_cast<uint64_t>(g.slots), cols, box) ||
               !tensor_map_rows(vm, a.v_plane, static_cast<uint64_t>(g.slots), cols, box)))
    return false;
  return tensor_map_q(qm, q, static_cast<uint64_t>(total_q), static_cast<uint64_t>(hq),
                      static_cast<uint64_t>(g.d), static_cast<uint32_t>(a.group),
                      static_cast<uint32_t>(a.tokens_per_tile));
}

}  // namespace direct
}  // namespace pkv
