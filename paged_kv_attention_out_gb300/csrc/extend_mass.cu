// extend_mass.cu - the attention weight that the keys of a row receive from a
// chunk's queries (all of them, or the last num_last), from the log-sum-exp that
// the attention call of the same queries returned.
//
// Mathematics, per request r, kv head h and key i, with p the cached prefix's length
// and t = p + j the position of chunk query j:
//   mass[row, h, i] = (accumulate and i < p ? mass[row, h, i] : 0)
//     + sum over the counted queries with t >= i and the group's q heads of
//       exp(s_ti - lse_t),   s the scores of the attention call
//
// S^T = K Q^T on tcgen05: keys are the rows (TMEM lanes), query rows the columns. A
// thread owns a key, so the sum over queries is a sum over the columns that it loads:
// nothing crosses threads, and no atomics. What a column needs, minus its lse, comes with
// the product: an extra k-step of 16 multiplies ones on the keys' side with -lse / scale
// on the queries' side, split into three bf16 terms (24 bits), so a score needs one
// multiplication and one exp2. Under a cap, and for scales without a usable reciprocal, it
// comes from shared memory instead, the same for all lanes.
//
// What bounds it: a 128 x 128 x 128 product takes 513 clocks alone (operands in shared
// memory, which its 64 KB keep as busy as the tensor pipe), the exponents of a unit
// 577-640 with 12 warps. Together a unit takes 733-762 clocks (D = 64: 697; under a cap
// 1217, since reads of lse beside the product stretch it to 856 and the sums to more), a
// call 10 us besides, until its first and after its last score. Measured, 32 : 8 heads of
// 128: 4 chunks of up to 2048 tokens after up to 6144, 140 us (0.61 of the bf16 rate on
// visible pairs; 157 with lse from shared memory).
//
// An item is a block of two 128-key tiles of one kv head, resident in shared memory,
// against which the request's query tiles (128 / group tokens x the group's heads, by TMA
// as 3-D boxes) are streamed; only those that see a key of the block. (Blocks of one tile
// take twice the Q traffic: 180 us.) The grid has a CTA an item, one runs per SM and takes
// over items of CTAs that have not started (clusterlaunchcontrol), so that items of any
// size even out and the roles run on across them (185 us with a CTA's items fixed). Calls
// with few items put a cluster on each: its CTAs take every size-th query tile and add up
// their sums through distributed shared memory, in order of rank, so the result does not
// depend on the order of execution.
//
// Roles: 12 warps that load K and then exponentiate and sum, one MMA warp, one warp that
// plans items and loads Q and lse. Units (a key tile against a query tile) go round
// three groups of four sum warps and four score buffers in TMEM, so that the MMAs of
// the next unit run while every group has one. Every wait is bounded (mbar_wait_*);
// after one ran out the sum warps still meet once an item, without work, so that no
// barrier waits for a warp that left.
#include <algorithm>
#include <cmath>

#include "launch.cuh"
#include "pkv_internal.h"
#include "row_units.cuh"
#include "score_rules.cuh"
#include "tc_common.cuh"
#include "tensor_map.h"

namespace pkv {
namespace {

constexpr int kM = 128;  // keys of a tile, and query rows of a tile
constexpr int kTiles = 2;
constexpr int kKeys = kTiles * kM;  // of an item
constexpr int kGroups = 3;  // of sum warps
constexpr int kSumWarps = 4 * kGroups;
constexpr int kSumThreads = kSumWarps * 32;
constexpr int kMmaWarp = kSumWarps;
constexpr int kQueryWarp = kSumWarps + 1;
constexpr int kMassThreads = (kSumWarps + 2) * 32;
constexpr int kCopyWarps = 8;  // of the sum warps, that load K
constexpr int kBufs = 4;       // score buffers
constexpr int kTmemCols = kBufs * kM;
constexpr int kStages = 4;     // query tiles in shared memory (their extra k-steps fill 128 bytes)
constexpr int kLseSlots = 8;   // query tiles whose lse is in shared memory
constexpr int kItemSlots = 8;  // items planned ahead
constexpr int kMaxMassCluster = 8;
constexpr int kTotalBarrier = 2;  // (1: the sum warps')

enum : int {
  kBarQFull = 0,                         // [kStages] Q landed (TMA bytes)
  kBarQEmpty = kBarQFull + kStages,      // [kStages] MMAs that read it done
  kBarLFull = kBarQEmpty + kStages,      // [kLseSlots] a query tile's lse written
  kBarLEmpty = kBarLFull + kLseSlots,    // [kLseSlots] read (4 warps for each of two units)
  kBarSFull = kBarLEmpty + kLseSlots,    // [kBufs] scores ready (MMAs), lse seen (MMA warp)
  kBarSEmpty = kBarSFull + kBufs,        // [kBufs] scores read (4 warps)
  kBarKFull = kBarSEmpty + kBufs,        // K in shared memory (kCopyWarps)
  kBarItemFull,                          // [kItemSlots] item described
  kBarItemEmpty = kBarItemFull + kItemSlots,  // [kItemSlots] read (sum warps + MMA warp)
  kBarTaken = kBarItemEmpty + kItemSlots,  // an answer about another CTA's item
  kBarTeardown,
  kBarCount,
};

template <int D>
struct MassSmem {
  static constexpr int kTileBytes = kM * D * 2;
  static constexpr int kK = 0;  // [kTiles]
  static constexpr int kQ = kTiles * kTileBytes;
  static constexpr int kLse = kQ + kStages * kTileBytes;  // [kLseSlots][128] fp32, or folded:
  static constexpr int kFold = kLse;  // a tile with the extra k-step of each Q stage,
  static constexpr int kOnes = kFold + kM * 128;  // and that of every key (32-byte rows of 1)
  static constexpr int kSum = kOnes + kM * 32;    // [2 items][kGroups][kKeys] fp32
  static constexpr int kBars = kSum + 2 * kGroups * kKeys * 4;
  static constexpr int kTotal = kBars + kBarCount * 8 + 1024;  // + alignment
  static_assert(kTotal <= 227 * 1024, "shared memory of a CTA");
};

__device__ __forceinline__ void mass_meet() {  // the cluster's threads
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ float mass_remote(uint32_t addr, int rank) {
  uint32_t there;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(there) : "memory");
  return v;
}

// mbar_wait_uniform for up to 32 barriers at once, one a lane (where `wait`).
__device__ __forceinline__ bool mbar_wait_lanes(uint32_t bar, uint32_t parity, bool wait,
                                                volatile int *abort) {
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    if (__all_sync(0xffffffffu, !wait || mbar_try(bar, parity))) return true;
    if ((i & 31) == 31) {
      const uint64_t t = global_timer_ns();
      if (t0 == 0) t0 = t;
      if (__any_sync(0xffffffffu, *abort != 0 || t - t0 > 2000000000ull)) return false;
    }
  }
}

__device__ __forceinline__ void named_barrier_arrive(int id, int threads) {
  __syncwarp();
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// A load that stays where it is written, ahead of its use.
__device__ __forceinline__ float load_early(const float *p) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

// A request's chunk, if its tables are sound (else without tokens).
struct Chunk {
  int n, c, beg, row;
};
__device__ __forceinline__ Chunk chunk_of(const MassArgs &a, int r, bool report) {
  Chunk k;
  k.n = a.seq_lens[r];
  k.beg = a.qo_indptr[r];
  const int end = a.qo_indptr[r + 1];
  k.row = a.table_idx ? a.table_idx[r] : r;
  k.c = 0;
  unsigned bad = 0;
  if (k.beg < 0 || end < k.beg || end > a.total_q) {
    bad |= kErrIndptr;
  } else if (end - k.beg > k.n) {
    bad |= k.n < 0 ? kErrSeqLen : kErrIndptr;
  }
  if (k.n < 0 || k.n > a.table_stride * a.page_size || k.n > a.mass_stride || k.n > kMaxRowKeys)
    bad |= kErrSeqLen;
  if (k.row < 0) bad |= kErrTableIdx;
  if (!bad) k.c = end - k.beg;
  if (bad && report) flag_error(a.err, bad);
  return k;
}

// How an exponent comes from a score and its query's lse.
enum : int {
  kPlain,   // score * scale - lse
  kCap,     // cap * tanh(score * scale / cap) - lse
  kFolded,  // the MMA has put -lse / scale on the score: times the scale
};

// 32 raw scores of this thread's key; under a cap also the largest absolute one.
template <int kForm>
__device__ __forceinline__ void load_scores(uint32_t taddr, float (&v)[32], float &top) {
  if constexpr (kForm == kCap)
    tmem_ld32_absmax(taddr, v, top);
  else
    tmem_ld32(taddr, v);
}

// exp2 of 32 scores in log2 units, less each query's lse (nlse: minus it), handed to
// sum(column, two, the next two) in fours. Under a cap the form of tanh goes by the
// largest score of the warp's 32 keys and 32 queries: the short polynomial within the
// exponential's argument, the longer one, or score by score.
template <int kForm, typename Sum>
__device__ __forceinline__ void exponents(const float (&v)[32], float top, const float4 *nlse,
                                          const MassArgs &a, Sum sum) {
  auto two = [](float x) { return make_float2(x, x); };
  auto each = [&](auto score) {  // score(v, v', nlse) -> exponents
#pragma unroll
    for (int cc = 0; cc < 32; cc += 4) {
      float4 nl = make_float4(0.f, 0.f, 0.f, 0.f);
      if constexpr (kForm != kFolded) nl = nlse[cc / 4];
      const float2 x = score(make_float2(v[cc], v[cc + 1]), make_float2(nl.x, nl.y));
      const float2 y = score(make_float2(v[cc + 2], v[cc + 3]), make_float2(nl.z, nl.w));
      sum(cc, make_float2(fast_exp2(x.x), fast_exp2(x.y)),
          make_float2(fast_exp2(y.x), fast_exp2(y.y)));
    }
  };
  if constexpr (kForm == kFolded) {
    each([&](float2 s, float2) { return __fmul2_rn(s, two(a.scale_log2)); });
  } else if constexpr (kForm == kPlain) {
    each([&](float2 s, float2 nl) { return __ffma2_rn(s, two(a.scale_log2), nl); });
  } else {
    if (__all_sync(0xffffffffu, top <= a.cap_near)) {
      each([&](float2 s, float2 nl) {
        const float2 u = __fmul2_rn(s, s);
        float2 p = __ffma2_rn(u, two(a.c5), two(a.c3));
        p = __ffma2_rn(u, p, two(a.c1));
        return __ffma2_rn(s, p, nl);
      });
    } else if (__all_sync(0xffffffffu, top <= a.cap_poly)) {
      each([&](float2 s, float2 nl) {
        const float2 x = __fmul2_rn(s, two(a.cap_in));
        const float2 u = __fmul2_rn(x, x);
        float2 p = __ffma2_rn(u, two(kTanh9), two(kTanh7));
        p = __ffma2_rn(u, p, two(kTanh5));
        p = __ffma2_rn(u, p, two(kTanh3));
        p = __ffma2_rn(__fmul2_rn(x, u), p, x);
        return __ffma2_rn(p, two(a.cap_log2), nl);
      });
    } else {
      each([&](float2 s, float2 nl) {
        return make_float2(fmaf(rule_tanh(s.x * a.cap_in), a.cap_log2, nl.x),
                           fmaf(rule_tanh(s.y * a.cap_in), a.cap_log2, nl.y));
      });
    }
  }
}

// The sum of exponentials of a unit for this thread's key: 128 columns of scores at srow,
// 32 at a time, the next ones on their way while these are computed. The score buffer is
// handed back (a lane of each warp arrives on `empty`) once all are read. whole: every
// column sees every key of the tile; else columns lo .. hi - 1 see this thread's.
template <int kForm>
__device__ __forceinline__ float unit_sum(uint32_t srow, const float4 *nlse, const MassArgs &a,
                                          bool whole, int lo, int hi, uint32_t empty) {
  const bool first_lane = (threadIdx.x & 31) == 0;
  float2 s0 = make_float2(0.f, 0.f), s1 = s0;
  if (whole) {  // (the same for the warp)
    float v[2][32], top[2];
    load_scores<kForm>(srow, v[0], top[0]);
#pragma unroll
    for (int q = 0; q < kM / 32; ++q) {
      tmem_ld_wait();
      if (q + 1 < kM / 32) {
        load_scores<kForm>(srow + (q + 1) * 32, v[(q + 1) & 1], top[(q + 1) & 1]);
      } else {
        tc_fence_before_sync();
        if (first_lane) mbar_arrive(empty);
        __syncwarp();
      }
      exponents<kForm>(v[q & 1], top[q & 1], nlse + q * 8, a, [&](int, float2 e, float2 f) {
        s0 = __fadd2_rn(s0, e);
        s1 = __fadd2_rn(s1, f);
      });
    }
  } else {
#pragma unroll 1
    for (int q = 0; q < kM / 32; ++q) {
      float v[32], top;
      load_scores<kForm>(srow + q * 32, v, top);
      tmem_ld_wait();
      const uint32_t seen = below_bits(hi - 32 * q) & ~below_bits(lo - 32 * q);
      exponents<kForm>(v, top, nlse + q * 8, a, [&](int cc, float2 e, float2 f) {
        e.x = (seen >> cc) & 1u ? e.x : 0.f;
        e.y = (seen >> (cc + 1)) & 1u ? e.y : 0.f;
        f.x = (seen >> (cc + 2)) & 1u ? f.x : 0.f;
        f.y = (seen >> (cc + 3)) & 1u ? f.y : 0.f;
        s0 = __fadd2_rn(s0, e);
        s1 = __fadd2_rn(s1, f);
      });
    }
    tc_fence_before_sync();
    if (first_lane) mbar_arrive(empty);
    __syncwarp();
  }
  return (s0.x + s0.y) + (s1.x + s1.y);
}

// umma_desc_sw128 for rows of 32 bytes (32-byte swizzle, groups of 8 rows 256 bytes apart).
__device__ __forceinline__ uint64_t umma_desc_sw32(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return umma_desc_sw128(saddr, lbo, sbo) ^ (static_cast<uint64_t>(2 ^ 6) << 61);
}

// Asks for a CTA of the grid that has not started; the answer, 16 bytes at shared address
// `to`, completes a phase of `bar`.
__device__ __forceinline__ void cancel_next(uint32_t to, uint32_t bar) {
  fence_async_shared();  // the previous answer has been read
  mbar_arrive_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], "
      "[%1];" ::"r"(to),
      "r"(bar)
      : "memory");
}
// That CTA, which will not start any more, or -1: there was none.
__device__ __forceinline__ int canceled_cta(uint32_t from) {
  int cta;
  asm volatile(
      "{\n .reg .b128 r;\n .reg .pred p;\n ld.shared.b128 r, [%1];\n mov.s32 %0, -1;\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n}\n"
      : "=r"(cta)
      : "r"(from)
      : "memory");
  return cta;
}

// One item as the planner publishes it: key block key0 .. of kv head h, and this CTA's
// query tiles: `mine` of them, tile i from chunk token j0 + i * step on. The first
// `one` of them see nothing of the second key tile, so its units are
//   u < one: query tile u, key tile 0
//   else v = u - one: query tile one + v / 2, key tile v % 2
struct MassItem {
  int row, n, beg, c;  // of the request
  int key0, h;
  int j0, mine, one;
};

template <int D, int kForm>
__global__ void __launch_bounds__(kMassThreads, 1)
    extend_mass_kernel(const __grid_constant__ CUtensorMap q_map, const MassArgs a, int size) {
  using S = MassSmem<D>;
  constexpr bool kFolds = kForm == kFolded;
  constexpr int kCh = D / 8;  // 16-byte chunks of a key
  extern __shared__ uint8_t smem_raw[];
  __shared__ MassItem s_item[kItemSlots];
  __shared__ __align__(16) uint4 s_taken;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_failed[2];  // a sum warp gave up in an item of this parity
  __shared__ int64_t s_total;
  const int tid = threadIdx.x;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int lane = tid & 31;
  const int rank = static_cast<int>(blockIdx.x) % size;
  const int64_t cluster = blockIdx.x / size, clusters = gridDim.x / size;
  const int tpt = a.tokens_per_tile;
  const int step = tpt * size;  // tokens between this CTA's query tiles
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_addr(smem);
  auto bar = [&](int i) { return sbase + S::kBars + 8u * static_cast<uint32_t>(i); };
  volatile int *abort = &s_abort;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(kBarQFull + i), kFolds ? 2 : 1);
      mbar_init(bar(kBarQEmpty + i), 1);
    }
    for (int i = 0; i < kLseSlots; ++i) {
      mbar_init(bar(kBarLFull + i), 1);
      mbar_init(bar(kBarLEmpty + i), 4 * kTiles);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(bar(kBarSFull + i), kFolds ? 1 : 2);
      mbar_init(bar(kBarSEmpty + i), 4);
    }
    mbar_init(bar(kBarKFull), kCopyWarps);
    for (int i = 0; i < kItemSlots; ++i) {
      mbar_init(bar(kBarItemFull + i), 1);
      mbar_init(bar(kBarItemEmpty + i), kSumWarps + 1);
    }
    mbar_init(bar(kBarTaken), 1);
    mbar_init(bar(kBarTeardown), 1);
    s_abort = s_failed[0] = s_failed[1] = 0;
    s_total = 0;
    mbar_init_fence();
  }
  {
    // Rows group * tpt .. 127 of a query tile are never loaded: zero them once.
    const int pad = kM - a.group * tpt;
    for (int i = tid; i < kStages * (D / 64) * pad * 8; i += kMassThreads) {
      const int chunk = i & 7, row = (i >> 3) % pad, region = (i >> 3) / pad;
      *reinterpret_cast<uint4 *>(smem + S::kQ + region * (kM * 128) + (kM - pad + row) * 128 +
                                 chunk * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    if constexpr (kFolds) {
      for (int i = tid; i < kM * 8; i += kMassThreads)
        *reinterpret_cast<uint4 *>(smem + S::kFold + i * 16) = make_uint4(0u, 0u, 0u, 0u);
      const uint32_t ones = 0x3f803f80u;  // two 1.0 in bf16
      for (int i = tid; i < kM * 2; i += kMassThreads)
        *reinterpret_cast<uint4 *>(smem + S::kOnes + i * 16) = make_uint4(ones, ones, ones, ones);
    }
    fence_async_shared();
  }
  if (warp == kMmaWarp) tmem_alloc(smem_addr(&s_tmem), kTmemCols);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s_tmem;
  grid_dependency_wait();
  grid_dependents_launch();

  // Items of the call: a request's key blocks times kv heads, kv heads innermost (the
  // heads of a key block are neighbours in memory), the blocks that most queries see
  // first.
  auto items_of = [&](const Chunk &k) -> int64_t {
    return k.c > 0 ? static_cast<int64_t>(a.hkv) * ((k.n + kKeys - 1) / kKeys) : 0;
  };
  {
    int64_t mine = 0;
    for (int r = tid; r < a.batch; r += kMassThreads)
      mine += items_of(chunk_of(a, r, true));
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, x);
    if (lane == 0 && mine > 0)
      atomicAdd(reinterpret_cast<unsigned long long *>(&s_total),
                static_cast<unsigned long long>(mine));
  }
  // A cluster's items are `cluster`, `cluster` + clusters, .. (one, where the grid was
  // sized right). A CTA on its own takes over further ones from CTAs that have not
  // started, until there are none; only its planner needs to know how many there are.
  int64_t total = INT64_MAX;
  int n_items = 0;
  auto count_items = [&] {
    __syncwarp();
    named_barrier_sync(kTotalBarrier, kMassThreads);
    total = s_total;
    n_items = cluster < total ? static_cast<int>((total - cluster + clusters - 1) / clusters) : 0;
  };
  if (warp != kQueryWarp) {
    if (size > 1)
      count_items();
    else
      named_barrier_arrive(kTotalBarrier, kMassThreads);
  }
  auto tile_tokens = [&](const MassItem &m, int j) { return min(tpt, m.c - j); };
  if (warp < kSumWarps) {
    // ------------------------------------------------------------ K, then sums
    const int group = warp >> 2;
    const int quarter = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const int key_row = quarter * 32 + lane;  // of a key tile
    // K: a copying warp has kRows keys of an item, one a lane looks up
    constexpr int kRows = kKeys / kCopyWarps;
    static_assert(kRows == 32, "a key a lane");
    const int64_t row_elems = static_cast<int64_t>(a.hkv) * D;
    auto look = [&](const MassItem &m) {
      const int key = m.key0 + warp * kRows + lane;
      if (key >= m.n) return -1;
      return __ldg(a.page_table + m.row * a.table_stride + a.page_of(key));
    };
    auto copy_keys = [&](const MassItem &m, int entry) {
      if (warp >= kCopyWarps) return;  // (a tile that the item lacks is zeros)
      const int key = m.key0 + warp * kRows + lane;
      int64_t slot = -1;
      if (key < m.n) {
        slot = static_cast<int64_t>(entry) * a.page_size + (key - a.page_of(key) * a.page_size);
        if (entry < 0 || slot >= a.slots) {
          slot = -1;
          flag_error(a.err, kErrPage);
        }
      }
      const int ch = lane % kCh;
      const __nv_bfloat16 *src = a.plane + m.h * D + ch * 8;
#pragma unroll
      for (int p = 0; p < kRows * kCh / 32; ++p) {
        const int i = p * (32 / kCh) + lane / kCh;
        const int64_t from = __shfl_sync(0xffffffffu, slot, i);
        const int k = warp * kRows + i;
        cp_async_16(sbase + S::kK + (k / kM) * S::kTileBytes + sw128_offset(kM, k % kM, ch * 8),
                    from >= 0 ? src + from * row_elems : a.plane, from >= 0 ? 16 : 0);
      }
      cp_async_wait_all();
      fence_async_shared();  // read next by tcgen05.mma
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarKFull));
    };
    auto wait_item = [&](int i) {
      return mbar_wait_warp(bar(kBarItemFull + i % kItemSlots), (i / kItemSlots) & 1, abort);
    };
    bool ok = true;
    // whether item it, which has been described, is one
    auto there = [&](int it) { return s_item[it % kItemSlots].n > 0; };
    if ((size == 1 || n_items > 0) && (ok = wait_item(0)) && there(0))
      copy_keys(s_item[0], look(s_item[0]));
    // over all items: query tiles and units before this one
    uint32_t tiles = 0, units = 0;
    for (int it = 0; size == 1 || it < n_items; ++it) {
      const int islot = it % kItemSlots;
      float had = 0.f;
      MassItem m{};
      if (ok) m = s_item[islot];
      if (ok && m.n > 0) {
        const int prefix = m.n - m.c;
        const int own = rank * (kKeys / size) + tid;  // key that this thread writes
        if (tid < kKeys / size && a.accumulate && m.key0 + own < prefix)
          had = __ldcg(a.mass + (static_cast<int64_t>(m.row) * a.hkv + m.h) * a.mass_stride +
                       m.key0 + own);
        float sum0 = 0.f, sum1 = 0.f;  // of this thread's key in both key tiles
        const int n_units = 2 * m.mine - m.one;
        // (from the first group on in every item, so that a sum does not depend on the items
        // that this CTA had before; the groups have just met, so none has to wait for it)
#pragma unroll 1
        for (int next = group; next < n_units; next += kGroups) {
          const int v = next - m.one;
          const int i = v < 0 ? next : m.one + (v >> 1);
          const int kt = v < 0 ? 0 : v & 1;
          const int j = m.j0 + i * step;
          const uint32_t unit = units + static_cast<uint32_t>(next);
          const int buf = static_cast<int>(unit % kBufs);
          const int ls = static_cast<int>((tiles + static_cast<uint32_t>(i)) % kLseSlots);
          if (!(ok = mbar_wait_warp(bar(kBarSFull + buf), (unit / kBufs) & 1, abort))) break;
          tc_fence_after_sync();
          const uint32_t srow = lanes + buf * kM;
          const float4 *nlse = reinterpret_cast<const float4 *>(smem + S::kLse + ls * kM * 4);
          const int tokens = tile_tokens(m, j);
          const int first = m.key0 + kt * kM;
          // columns lo .. hi - 1 see this thread's key; all do in most units
          const int lo = a.group * max(0, first + key_row - prefix - j), hi = a.group * tokens;
          const bool whole = tokens == tpt && first + kM - 1 <= prefix + j;
          const float given = unit_sum<kForm>(srow, nlse, a, whole, lo, hi, bar(kBarSEmpty + buf));
          if (kt == 0)
            sum0 += given;
          else
            sum1 += given;
          if constexpr (!kFolds) {
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bar(kBarLEmpty + ls));
              if (v < 0) mbar_arrive(bar(kBarLEmpty + ls));  // (for the unit that is not)
            }
          }
        }
        tiles += static_cast<uint32_t>(m.mine);
        units += static_cast<uint32_t>(n_units);
        float *sums = reinterpret_cast<float *>(smem + S::kSum) +
                      ((it & 1) * kGroups + group) * kKeys + key_row;
        sums[0] = sum0;
        sums[kM] = sum1;
      }
      // the page entry of this lane's key of the next item, on its way meanwhile
      int entry = -1;
      if (ok && (size == 1 || it + 1 < n_items) && m.n > 0 && (ok = wait_item(it + 1)) &&
          there(it + 1))
        entry = look(s_item[(it + 1) % kItemSlots]);
      if (!ok && lane == 0) {
        *abort = s_failed[it & 1] = 1;
        flag_error(a.err, kErrTimeout);
      }
      // The sums of all groups (and of the cluster) meet.
      if (size == 1)
        named_barrier_sync(1, kSumThreads);
      else
        mass_meet();
      // (what the sum warps said before they met: the same for all of them)
      ok = ok && s_failed[it & 1] == 0;
      if (size == 1 && (!ok || m.n == 0)) break;
      if (!ok) continue;
      // every MMA of this item is done: its keys make way for the next one's
      if ((size == 1 || it + 1 < n_items) && there(it + 1))
        copy_keys(s_item[(it + 1) % kItemSlots], entry);
      if (tid < kKeys / size) {
        const int own = rank * (kKeys / size) + tid;
        if (m.key0 + own < m.n) {
          float given = 0.f;
          for (int c = 0; c < size; ++c)
#pragma unroll
            for (int p = 0; p < kGroups; ++p) {
              const int at = ((it & 1) * kGroups + p) * kKeys + own;
              given += size == 1 ? reinterpret_cast<const float *>(smem + S::kSum)[at]
                                 : mass_remote(sbase + S::kSum + at * 4, c);
            }
          a.mass[(static_cast<int64_t>(m.row) * a.hkv + m.h) * a.mass_stride + m.key0 + own] =
              had + given;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarItemEmpty + islot));
    }
    cp_async_wait_all();  // (copies still in flight after a wait ran out)
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    const bool issuer = elect_one();
    constexpr uint32_t idesc = umma_idesc_bf16(kM, kM, 0, 0);
    const uint64_t dk0 = umma_desc_sw128(sbase + S::kK, 16, 1024);
    const uint64_t dq0 = umma_desc_sw128(sbase + S::kQ, 16, 1024);
    const uint64_t dfold = umma_desc_sw128(sbase + S::kFold, 16, 1024);
    const uint64_t dones = umma_desc_sw32(sbase + S::kOnes, 16, 256);
    auto kstep = [](int ks) -> uint64_t {
      return static_cast<uint64_t>(((ks >> 2) * (kM * 128) + (ks & 3) * 32) >> 4);
    };
    bool ok = true;
    uint32_t tiles = 0, units = 0;
    for (int it = 0; size == 1 || it < n_items; ++it) {
      const int islot = it % kItemSlots;
      if (ok && (ok = mbar_wait_uniform(bar(kBarItemFull + islot), (it / kItemSlots) & 1, abort))) {
        const MassItem m = s_item[islot];
        __syncwarp();
        if (issuer) mbar_arrive(bar(kBarItemEmpty + islot));
        if (m.n == 0) break;  // no more (a CTA on its own)
        ok = mbar_wait_uniform(bar(kBarKFull), it & 1, abort);
        for (int i = 0; ok && i < m.mine; ++i, ++tiles) {
          const int nk = i < m.one ? 1 : 2;
          const int st = static_cast<int>(tiles % kStages);
          const int ls = static_cast<int>(tiles % kLseSlots);
          const uint64_t dq = dq0 + static_cast<uint64_t>((st * S::kTileBytes) >> 4);
          // a lane for each of what has to be there: Q, lse, the units' buffers
          const uint32_t mine = units + static_cast<uint32_t>(lane - 2);  // (lanes 2 and 3)
          const int which = lane == 0   ? kBarQFull + st
                            : lane == 1 ? kBarLFull + ls
                                        : kBarSEmpty + static_cast<int>(mine % kBufs);
          const uint32_t phase = lane == 0   ? tiles / kStages
                                 : lane == 1 ? tiles / kLseSlots
                                             : mine / kBufs - 1;
          const bool wait = lane == 0 || (lane == 1 && !kFolds) ||
                            (lane >= 2 && lane < 2 + nk && mine >= kBufs);
          if (!(ok = mbar_wait_lanes(bar(which), phase & 1, wait, abort))) break;
          tc_fence_after_sync();
          if (issuer) {
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
              if (t >= nk) continue;
              const int buf = static_cast<int>((units + t) % kBufs);
              const uint64_t dk = dk0 + static_cast<uint64_t>((t * S::kTileBytes) >> 4);
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks)
                umma_bf16_ss(tmem + buf * kM, dk + kstep(ks), dq + kstep(ks), idesc,
                             ks > 0 ? 1u : 0u);
              if constexpr (kFolds)
                umma_bf16_ss(tmem + buf * kM, dones, dfold + kstep(st), idesc, 1u);
              umma_commit(bar(kBarSFull + buf));
              if constexpr (!kFolds)  // (releases the lse that this warp has seen)
                mbar_arrive(bar(kBarSFull + buf));
            }
            umma_commit(bar(kBarQEmpty + st));
          }
          __syncwarp();
          units += static_cast<uint32_t>(nk);
        }
      }
      if (!ok) {
        *abort = 1;
        flag_error(a.err, kErrTimeout);
        if (size == 1) break;
      }
      if (size > 1) mass_meet();
    }
  } else if (warp == kQueryWarp) {
    // ------------------------------------------------------------ items, Q and lse
    int tok[4], head[4];  // of this lane's four rows of a query tile
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      tok[e] = (4 * lane + e) / a.group;
      head[e] = (4 * lane + e) % a.group;
    }
    // The requests r0 + lane whose items are looked through, and the items before and
    // up to each.
    int r0 = 0;
    int64_t before = 0, up_to = 0;
    Chunk ck{};
    auto look_at = [&] {
      ck = r0 + lane < a.batch ? chunk_of(a, r0 + lane, false) : Chunk{};
      up_to = items_of(ck);
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, up_to, off);
        if (lane >= off) up_to += v;
      }
    };
    look_at();
    bool ok = true;
    // Publishes item number `item` of the call as this CTA's k-th; item >= total: no more.
    auto plan = [&](int k, int64_t item) -> bool {
      const int slot = k % kItemSlots;
      if (k >= kItemSlots &&
          !mbar_wait_uniform(bar(kBarItemEmpty + slot), (k / kItemSlots - 1) & 1, abort))
        return false;
      if (item >= total) {
        if (lane == 0) {
          s_item[slot].n = 0;
          mbar_arrive(bar(kBarItemFull + slot));
        }
        __syncwarp();
        return true;
      }
      if (item < before) {  // (items taken over need not come in order)
        before = 0;
        r0 = 0;
        look_at();
      }
      for (int64_t all; item >= before + (all = __shfl_sync(0xffffffffu, up_to, 31));) {
        before += all;
        r0 += 32;
        look_at();
      }
      const int l = __ffs(__ballot_sync(0xffffffffu, item < before + up_to)) - 1;
      const int64_t local = item - before - __shfl_sync(0xffffffffu, up_to - items_of(ck), l);
      if (lane == l) {
        MassItem m;
        m.row = ck.row;
        m.n = ck.n;
        m.beg = ck.beg;
        m.c = ck.c;
        const int kb = static_cast<int>(local / a.hkv);
        m.h = static_cast<int>(local - static_cast<int64_t>(kb) * a.hkv);
        m.key0 = kb * kKeys;
        // query tiles from the first that sees key0 on; this CTA's every size-th
        const int first = a.num_last > 0 ? max(0, ck.c - a.num_last) : 0;
        const int all_tiles = (ck.c - first + tpt - 1) / tpt;
        const int tile0 = max(0, m.key0 - (ck.n - ck.c) - first) / tpt + rank;
        m.j0 = first + tile0 * tpt;
        m.mine = max(0, (all_tiles - tile0 + size - 1) / size);
        // tiles whose last token is before the second key tile
        const int before_second = m.key0 + kM - (ck.n - ck.c);  // chunk tokens
        if (ck.c <= before_second)
          m.one = m.mine;
        else
          m.one = before_second < m.j0 + tpt
                      ? 0
                      : min(m.mine, (before_second - tpt - m.j0) / step + 1);
        s_item[slot] = m;
        mbar_arrive(bar(kBarItemFull + slot));
      }
      __syncwarp();
      return true;
    };
    const float unscale = -kLog2e / a.scale_log2;  // -1 / scale (folded)
    uint32_t tiles = 0, loads = 0;
    int64_t item = cluster;
    bool over = size > 1;  // nothing more to take over
    int answers = 0;
    // (the first item, if it is one of the requests looked at, before all are counted)
    const bool early = item < __shfl_sync(0xffffffffu, up_to, 31);
    if (early) ok = plan(0, item);
    count_items();
    if (!early && (size == 1 || n_items > 0)) ok = plan(0, item);
    for (int it = 0; size == 1 ? ok && item < total : it < n_items; ++it) {
      // the item after this one: the CTA's own, or one to be taken over
      int64_t after = item + clusters;
      const bool asks = after >= total && !over;
      if (asks) {
        if (lane == 0) cancel_next(smem_addr(&s_taken), bar(kBarTaken));
        __syncwarp();
      }
      if (ok) {
        const MassItem m = s_item[it % kItemSlots];
        // the lse of this lane's rows, read a tile ahead (+inf, no weight, for none)
        auto read_lse = [&](int j, float (&x)[4]) {
          const int tokens = tile_tokens(m, j);
          const float *p = a.lse + (static_cast<int64_t>(m.beg) + j) * a.hq + m.h * a.group;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[e] = tok[e] < tokens ? load_early(p + tok[e] * a.hq + head[e]) : INFINITY;
        };
        float next[4];
        if (m.mine > 0) read_lse(m.j0, next);
        for (int i = 0; i < m.mine; ++i, ++tiles) {
          const int j = m.j0 + i * step;
          const int st = static_cast<int>(tiles % kStages);
          const int ls = static_cast<int>(tiles % kLseSlots);
          float lse[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) lse[e] = next[e];
          if (i + 1 < m.mine) read_lse(j + step, next);
          if (tiles >= kStages && !(ok = mbar_wait_uniform(bar(kBarQEmpty + st),
                                                           (tiles / kStages - 1) & 1, abort)))
            break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(kBarQFull + st),
                                  (D / 64) * static_cast<uint32_t>(a.group * tpt) * 128u);
#pragma unroll
            for (int half = 0; half < D / 64; ++half)
              tma_load_3d(sbase + S::kQ + st * S::kTileBytes + half * (kM * 128), &q_map,
                          half * 64, m.h * a.group, m.beg + j, bar(kBarQFull + st));
          }
          loads = tiles + 1;
          if constexpr (kFolds) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // -lse / scale in three bf16 terms, 24 bits together. A row without weight (none,
              // or an empty one's -inf) gets the infinity that the scale turns negative.
              const float x = lse[e] == -INFINITY ? INFINITY * unscale : lse[e] * unscale;
              const __nv_bfloat16 x0 = __float2bfloat16_rn(x);
              const float left = __hisinf(x0) ? 0.f : x - __bfloat162float(x0);
              const __nv_bfloat16 x1 = __float2bfloat16_rn(left);
              const __nv_bfloat16 x2 = __float2bfloat16_rn(left - __bfloat162float(x1));
              const uint32_t at = sw128_offset(kM, 4 * lane + e, 16 * st);
              *reinterpret_cast<uint2 *>(smem + S::kFold + at) =
                  make_uint2(__bfloat16_as_ushort(x0) |
                                 static_cast<uint32_t>(__bfloat16_as_ushort(x1)) << 16,
                             __bfloat16_as_ushort(x2));
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarQFull + st));
            continue;
          }
          if (tiles >= kLseSlots && !(ok = mbar_wait_uniform(bar(kBarLEmpty + ls),
                                                             (tiles / kLseSlots - 1) & 1, abort)))
            break;
#pragma unroll
          for (int e = 0; e < 4; ++e)  // (an empty row's, -inf, gives no weight either)
            lse[e] = lse[e] == -INFINITY ? -INFINITY : -lse[e] * kLog2e;
          *reinterpret_cast<float4 *>(smem + S::kLse + ls * kM * 4 + lane * 16) =
              make_float4(lse[0], lse[1], lse[2], lse[3]);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarLFull + ls));
        }
      }
      if (asks) {
        int never = 0;  // (the answer comes whatever else went wrong)
        ok = mbar_wait_uniform(bar(kBarTaken), answers++ & 1, &never) && ok;
        const int taken = ok ? canceled_cta(smem_addr(&s_taken)) : -1;
        over = taken < 0 || taken >= total;  // (those left, if any, run on their own)
        after = over ? total : taken;
      }
      item = after;
      if (ok && (size == 1 || it + 1 < n_items)) ok = plan(it + 1, item);
      if (!ok) {
        *abort = 1;
        flag_error(a.err, kErrTimeout);
      }
      if (size > 1) mass_meet();
    }
    if (*abort && lane == 0) {
      // copies in flight land before the CTA can exit
      int never = 0;
      for (uint32_t u = loads > kStages ? loads - kStages : 0; u < loads; ++u)
        mbar_wait(bar(kBarQFull + static_cast<int>(u % kStages)), (u / kStages) & 1, &never);
    }
  }

  if (size > 1) mass_meet();  // no CTA ends while its sums are read
  if (warp == kMmaWarp && __any_sync(0xffffffffu, *abort != 0)) {
    if (elect_one()) {
      umma_commit(bar(kBarTeardown));  // tracks every MMA this lane issued
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

// ------------------------------------------------------------ few queries
// Where every request's counted queries fit kFewTiles query tiles, the call is bound by
// reading K, and the roles change places: a request's query tiles stay in shared memory
// and its keys stream past. CTA (range, kv head) takes one of `ranges` equal shares of
// all requests' key tiles, in order; the CTAs of a range's kv heads read neighbouring
// lines at about the same time. Four warps copy K tiles into a ring, three of them in
// flight (96 KB an SM at D = 128), the MMA warp multiplies each with the query tiles,
// and two groups of sum warps take a key tile each in turn: a thread has all weight of
// its key and adds it to what was there. Measured, 32 : 8 heads of 128, and the other form:
// the last 32 of 8 prompts of up to 32768 51 us (0.77 of the copy rate), 104; the last 64
// 69, 128; the last 64 of 4 of up to 2000 11.0, 11.0; 2 chunks of 24 after 176 7.5, 8.9.
// (One more tile in flight, where a call has one query tile only: 53.)
constexpr int kFewTiles = 2;
constexpr int kFewGroups = 2;
constexpr int kFewSumWarps = 4 * kFewGroups;
constexpr int kFewCopyWarp = kFewSumWarps;
constexpr int kFewCopyWarps = 4;  // 32 keys each of a tile
constexpr int kFewMmaWarp = kFewCopyWarp + kFewCopyWarps;
constexpr int kFewQueryWarp = kFewMmaWarp + 1;
constexpr int kFewThreads = (kFewQueryWarp + 1) * 32;
constexpr int kFewSlots = 4;  // K tiles in shared memory
constexpr int kFewAhead = 3;  // of them in flight
constexpr int kFewRuns = 4;   // runs planned ahead

enum : int {
  kFewKFull = 0,                           // [kFewSlots] K tile landed (copy warps)
  kFewKEmpty = kFewKFull + kFewSlots,      // [kFewSlots] MMAs that read it done
  kFewSFull = kFewKEmpty + kFewSlots,      // [kBufs] scores ready
  kFewSEmpty = kFewSFull + kBufs,          // [kBufs] scores read (4 warps)
  kFewQFull = kFewSEmpty + kBufs,          // a run's query tiles landed (TMA bytes)
  kFewQEmpty,                              // MMAs that read them done
  kFewRunFull,                             // [kFewRuns] run described
  kFewLFull = kFewRunFull + kFewRuns,      // [kFewRuns] its lse written
  kFewRunEmpty = kFewLFull + kFewRuns,     // [kFewRuns] read (all warps but the planner)
  kFewTeardown = kFewRunEmpty + kFewRuns,
  kFewCount,
};

template <int D>
struct FewSmem {
  static constexpr int kTileBytes = kM * D * 2;
  static constexpr int kK = 0;
  static constexpr int kQ = kFewSlots * kTileBytes;
  static constexpr int kLse = kQ + kFewTiles * kTileBytes;  // [kFewRuns][kFewTiles][128] fp32
  static constexpr int kBars = kLse + kFewRuns * kFewTiles * kM * 4;
  static constexpr int kTotal = kBars + kFewCount * 8 + 1024;  // + alignment
  static_assert(kTotal <= 227 * 1024, "shared memory of a CTA");
};

// Consecutive key tiles of one request: first .. first + count - 1, against `tiles`
// query tiles from chunk token j0 on. count 0: no more.
struct FewRun {
  int row, n, beg, c;
  int first, count;
  int j0, tiles;
};

template <int D, int kForm>
__global__ void __launch_bounds__(kFewThreads, 1)
    extend_mass_few_kernel(const __grid_constant__ CUtensorMap q_map, const MassArgs a) {
  using S = FewSmem<D>;
  constexpr int kCh = D / 8;
  extern __shared__ uint8_t smem_raw[];
  __shared__ FewRun s_run[kFewRuns];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ unsigned long long s_total;
  const int tid = threadIdx.x;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int lane = tid & 31;
  const int h = static_cast<int>(blockIdx.x) % a.hkv;
  const int64_t range = blockIdx.x / a.hkv, ranges = gridDim.x / a.hkv;
  const int tpt = a.tokens_per_tile;
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_addr(smem);
  auto bar = [&](int i) { return sbase + S::kBars + 8u * static_cast<uint32_t>(i); };
  volatile int *abort = &s_abort;

  if (tid == 0) {
    for (int i = 0; i < kFewSlots; ++i) {
      mbar_init(bar(kFewKFull + i), kFewCopyWarps);
      mbar_init(bar(kFewKEmpty + i), 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(bar(kFewSFull + i), 1);
      mbar_init(bar(kFewSEmpty + i), 4);
    }
    mbar_init(bar(kFewQFull), 1);
    mbar_init(bar(kFewQEmpty), 1);
    for (int i = 0; i < kFewRuns; ++i) {
      mbar_init(bar(kFewRunFull + i), 1);
      mbar_init(bar(kFewLFull + i), 1);
      mbar_init(bar(kFewRunEmpty + i), kFewQueryWarp);
    }
    mbar_init(bar(kFewTeardown), 1);
    s_abort = 0;
    s_total = 0;
    mbar_init_fence();
  }
  {
    // Rows group * tpt .. 127 of a query tile are never loaded: zero them once.
    const int pad = kM - a.group * tpt;
    for (int i = tid; i < kFewTiles * (D / 64) * pad * 8; i += kFewThreads) {
      const int chunk = i & 7, row = (i >> 3) % pad, region = (i >> 3) / pad;
      *reinterpret_cast<uint4 *>(smem + S::kQ + region * (kM * 128) + (kM - pad + row) * 128 +
                                 chunk * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_async_shared();
  }
  if (warp == kFewMmaWarp) tmem_alloc(smem_addr(&s_tmem), kTmemCols);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s_tmem;
  grid_dependency_wait();
  grid_dependents_launch();

  auto tiles_of = [&](const Chunk &k) { return k.c > 0 ? (k.n + kM - 1) / kM : 0; };
  {
    int64_t mine = 0;
    for (int r = tid; r < a.batch; r += kFewThreads)
      mine += tiles_of(chunk_of(a, r, blockIdx.x == 0));
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, x);
    if (lane == 0 && mine > 0) atomicAdd(&s_total, static_cast<unsigned long long>(mine));
  }
  __syncthreads();
  const int64_t total = static_cast<int64_t>(s_total);
  const int64_t begin = total * range / ranges, end = total * (range + 1) / ranges;

  // The next run, for a warp that reads (false: none, or a wait ran out).
  auto take_run = [&](int k, bool &ok) {
    ok = ok && mbar_wait_warp(bar(kFewRunFull + k % kFewRuns), (k / kFewRuns) & 1, abort);
    return ok && s_run[k % kFewRuns].count > 0;
  };
  auto leave_run = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kFewRunEmpty + k % kFewRuns));
  };

  bool ok = true;
  if (warp < kFewSumWarps) {
    // ------------------------------------------------------------ sums
    const int group = warp >> 2;
    const int key_row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    uint32_t tiles = 0;  // key tiles before this run
    uint32_t uses = 0;   // units of this group
    for (int k = 0; take_run(k, ok); ++k) {
      const FewRun m = s_run[k % kFewRuns];
      const int prefix = m.n - m.c;
      float *mass = a.mass + (static_cast<int64_t>(m.row) * a.hkv + h) * a.mass_stride;
      auto before = [&](int i) {  // what this thread's key of tile i of the run had
        const int key = (m.first + i) * kM + key_row;
        return a.accumulate && key < prefix && i < m.count ? __ldcg(mass + key) : 0.f;
      };
      int i = static_cast<int>((static_cast<uint32_t>(group) - tiles) % kFewGroups);
      float had = before(i);
      ok = mbar_wait_warp(bar(kFewLFull + k % kFewRuns), (k / kFewRuns) & 1, abort);
#pragma unroll 1
      for (; ok && i < m.count; i += kFewGroups) {
        const float next = before(i + kFewGroups);
        const int key = (m.first + i) * kM + key_row;
        float given = 0.f;
        for (int q = 0; q < m.tiles; ++q) {
          const uint32_t use = uses++;
          const int buf = 2 * group + static_cast<int>(use & 1);
          if (!(ok = mbar_wait_warp(bar(kFewSFull + buf), (use >> 1) & 1, abort))) break;
          tc_fence_after_sync();
          const int j = m.j0 + q * tpt;
          const int tokens = min(tpt, m.c - j);
          const int lo = a.group * max(0, key - prefix - j), hi = a.group * tokens;
          const bool whole = tokens == tpt && (m.first + i + 1) * kM - 1 <= prefix + j;
          given += unit_sum<kForm>(
              lanes + buf * kM,
              reinterpret_cast<const float4 *>(smem + S::kLse +
                                               ((k % kFewRuns) * kFewTiles + q) * kM * 4),
              a, whole, lo, hi, bar(kFewSEmpty + buf));
        }
        if (ok && key < m.n) mass[key] = had + given;
        had = next;
      }
      tiles += static_cast<uint32_t>(m.count);
      leave_run(k);
    }
  } else if (warp < kFewMmaWarp) {
    // ------------------------------------------------------------ K
    const int part = (warp - kFewCopyWarp) * 32;  // this warp's keys of a tile
    const int64_t row_elems = static_cast<int64_t>(a.hkv) * D;
    const int ch = lane % kCh;
    const __nv_bfloat16 *src = a.plane + h * D + ch * 8;
    uint32_t tiles = 0;   // tiles issued
    uint32_t landed = 0;  // tiles handed over
    auto hand_over = [&] {
      fence_async_shared();  // read next by tcgen05.mma
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kFewKFull + static_cast<int>(landed % kFewSlots)));
      ++landed;
    };
    for (int k = 0;; ++k) {
      // A run that is not there yet may wait for the tiles still held back (its planner
      // for the MMAs of the run before the last): all of them go out first.
      if (!__all_sync(0xffffffffu,
                      mbar_try(bar(kFewRunFull + k % kFewRuns), (k / kFewRuns) & 1))) {
        cp_async_wait_all();
        while (landed < tiles) hand_over();
      }
      if (!take_run(k, ok)) break;
      const FewRun m = s_run[k % kFewRuns];
      const int32_t *pages = a.page_table + m.row * a.table_stride;
      auto look = [&](int i) {
        const int key = (m.first + i) * kM + part + lane;
        return i < m.count && key < m.n ? __ldg(pages + a.page_of(key)) : -1;
      };
      int entry = look(0);
#pragma unroll 1
      for (int i = 0; i < m.count; ++i) {
        const int key = (m.first + i) * kM + part + lane;
        int64_t slot = -1;
        if (key < m.n) {
          slot = static_cast<int64_t>(entry) * a.page_size + (key - a.page_of(key) * a.page_size);
          if (entry < 0 || slot >= a.slots) {
            slot = -1;
            flag_error(a.err, kErrPage);
          }
        }
        entry = look(i + 1);
        const int s = static_cast<int>(tiles % kFewSlots);
        if (tiles >= kFewSlots &&
            !(ok = mbar_wait_warp(bar(kFewKEmpty + s), (tiles / kFewSlots - 1) & 1, abort)))
          break;
#pragma unroll
        for (int c = 0; c < kCh; ++c) {
          const int l = c * (32 / kCh) + lane / kCh;
          const int64_t from = __shfl_sync(0xffffffffu, slot, l);
          cp_async_16(sbase + S::kK + s * S::kTileBytes + sw128_offset(kM, part + l, ch * 8),
                      from >= 0 ? src + from * row_elems : a.plane, from >= 0 ? 16 : 0);
        }
        cp_async_commit();
        ++tiles;
        if (tiles - landed >= kFewAhead) {
          cp_async_wait<kFewAhead - 1>();
          hand_over();
        }
      }
      if (!ok) break;
      leave_run(k);
    }
    cp_async_wait_all();
    while (ok && landed < tiles) hand_over();
  } else if (warp == kFewMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    const bool issuer = elect_one();
    constexpr uint32_t idesc = umma_idesc_bf16(kM, kM, 0, 0);
    const uint64_t dk0 = umma_desc_sw128(sbase + S::kK, 16, 1024);
    const uint64_t dq0 = umma_desc_sw128(sbase + S::kQ, 16, 1024);
    auto kstep = [](int ks) -> uint64_t {
      return static_cast<uint64_t>(((ks >> 2) * (kM * 128) + (ks & 3) * 32) >> 4);
    };
    uint32_t tiles = 0;
    uint32_t uses0 = 0, uses1 = 0;  // units of each group
    for (int k = 0; take_run(k, ok); ++k) {
      const int count = s_run[k % kFewRuns].count, nq = s_run[k % kFewRuns].tiles;
      leave_run(k);
      ok = mbar_wait_uniform(bar(kFewQFull), k & 1, abort);
      for (int i = 0; ok && i < count; ++i, ++tiles) {
        const int s = static_cast<int>(tiles % kFewSlots);
        if (!(ok = mbar_wait_uniform(bar(kFewKFull + s), (tiles / kFewSlots) & 1, abort))) break;
        const uint64_t dk = dk0 + static_cast<uint64_t>((s * S::kTileBytes) >> 4);
        const int group = static_cast<int>(tiles % kFewGroups);
        for (int q = 0; q < nq; ++q) {
          const uint32_t use = group == 0 ? uses0++ : uses1++;
          const int buf = 2 * group + static_cast<int>(use & 1);
          if (use >= 2 &&
              !(ok = mbar_wait_uniform(bar(kFewSEmpty + buf), ((use >> 1) - 1) & 1, abort)))
            break;
          tc_fence_after_sync();
          if (issuer) {
            const uint64_t dq = dq0 + static_cast<uint64_t>((q * S::kTileBytes) >> 4);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
              umma_bf16_ss(tmem + buf * kM, dk + kstep(ks), dq + kstep(ks), idesc,
                           ks > 0 ? 1u : 0u);
            umma_commit(bar(kFewSFull + buf));
          }
          __syncwarp();
        }
        if (ok && issuer) umma_commit(bar(kFewKEmpty + s));
        __syncwarp();
      }
      if (ok && issuer) umma_commit(bar(kFewQEmpty));
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ runs, Q and lse
    int64_t before = 0;  // key tiles of the requests before r
    int k = 0;
    auto publish = [&](const FewRun &m) -> bool {
      const int slot = k % kFewRuns;
      if (k >= kFewRuns &&
          !mbar_wait_uniform(bar(kFewRunEmpty + slot), (k / kFewRuns - 1) & 1, abort))
        return false;
      if (lane == 0) s_run[slot] = m;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kFewRunFull + slot));  // (its keys set out at once)
      if (m.count > 0) {
        auto load_q = [&] {
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(kFewQFull), static_cast<uint32_t>(m.tiles) * (D / 64) *
                                                      static_cast<uint32_t>(a.group * tpt) * 128u);
            for (int q = 0; q < m.tiles; ++q)
#pragma unroll
              for (int half = 0; half < D / 64; ++half)
                tma_load_3d(sbase + S::kQ + q * S::kTileBytes + half * (kM * 128), &q_map,
                            half * 64, h * a.group, m.beg + m.j0 + q * tpt, bar(kFewQFull));
          }
          __syncwarp();
        };
        if (k == 0) load_q();
        for (int q = 0; q < kFewTiles; ++q) {
          float *to = reinterpret_cast<float *>(smem + S::kLse) + (slot * kFewTiles + q) * kM;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int rw = e * 32 + lane;  // row of the query tile
            const int tok = m.j0 + q * tpt + rw / a.group;
            float lse = INFINITY;  // no row, no weight (an empty one's, -inf, gives none either)
            if (rw < a.group * tpt && tok < m.c)
              lse = __ldg(a.lse + (static_cast<int64_t>(m.beg) + tok) * a.hq + h * a.group +
                          rw % a.group);
            to[rw] = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kFewLFull + slot));
        if (k > 0) {
          if (!mbar_wait_uniform(bar(kFewQEmpty), (k - 1) & 1, abort)) return false;
          load_q();
        }
      }
      ++k;
      return true;
    };
    for (int r0 = 0; ok && r0 < a.batch && before < end; r0 += 32) {
      const Chunk mine = r0 + lane < a.batch ? chunk_of(a, r0 + lane, false) : Chunk{};
      for (int l = 0; ok && l < 32 && r0 + l < a.batch && before < end; ++l) {
        Chunk ck;
        ck.n = __shfl_sync(0xffffffffu, mine.n, l);
        ck.c = __shfl_sync(0xffffffffu, mine.c, l);
        ck.beg = __shfl_sync(0xffffffffu, mine.beg, l);
        ck.row = __shfl_sync(0xffffffffu, mine.row, l);
        const int64_t n_tiles = tiles_of(ck);
        const int64_t lo = max(begin - before, int64_t(0)), hi = min(end - before, n_tiles);
        before += n_tiles;
        if (lo >= hi) continue;
        FewRun m;
        m.row = ck.row;
        m.n = ck.n;
        m.beg = ck.beg;
        m.c = ck.c;
        m.first = static_cast<int>(lo);
        m.count = static_cast<int>(hi - lo);
        m.j0 = a.num_last > 0 ? max(0, ck.c - a.num_last) : 0;
        m.tiles = (ck.c - m.j0 + tpt - 1) / tpt;
        ok = publish(m);
      }
    }
    if (ok) ok = publish(FewRun{});
    if (*abort && lane == 0 && k > 0) {
      int never = 0;  // copies in flight land before the CTA can exit
      mbar_wait(bar(kFewQFull), (k - 1) & 1, &never);
    }
  }
  if (!ok && lane == 0) {
    *abort = 1;
    flag_error(a.err, kErrTimeout);
  }

  __syncwarp();
  if (warp == kFewMmaWarp && __any_sync(0xffffffffu, *abort != 0)) {
    if (elect_one()) {
      umma_commit(bar(kFewTeardown));  // tracks every MMA this lane issued
      int never = 0;
      mbar_wait(bar(kFewTeardown), 0, &never);
    }
    __syncwarp();
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kFewMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, int kForm>
cudaError_t launch_few(const CUtensorMap &q_map, const MassArgs &a, int64_t grid,
                       cudaStream_t stream) {
  auto kernel = extend_mass_few_kernel<D, kForm>;
  constexpr int kSmem = FewSmem<D>::kTotal;
  cudaError_t e = allow_smem(kernel, kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kFewThreads), kSmem, stream,
                    q_map, a);
}

template <int D, int kForm>
cudaError_t launch(const CUtensorMap &q_map, const MassArgs &a, int64_t clusters, int size,
                   cudaStream_t stream) {
  auto kernel = extend_mass_kernel<D, kForm>;
  constexpr int kSmem = MassSmem<D>::kTotal;
  cudaError_t e = allow_smem(kernel, kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * size));
  cfg.blockDim = dim3(kMassThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(size);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, q_map, a, size);
}

template <int D>
cudaError_t launch_d(const CUtensorMap &q_map, const MassArgs &a, int64_t clusters, int size,
                     cudaStream_t stream) {
  if (a.cap_log2 > 0.f) return launch<D, kCap>(q_map, a, clusters, size, stream);
  // (a scale outside these bounds, zero first of all, has no place in 1 / scale)
  const float scale = std::abs(a.scale_log2);
  if (scale >= 0x1p-60f && scale <= 0x1p60f)
    return launch<D, kFolded>(q_map, a, clusters, size, stream);
  return launch<D, kPlain>(q_map, a, clusters, size, stream);
}

}  // namespace

cudaError_t launch_extend_mass(const PoolGeom &g, const MassArgs &a, const void *q,
                               int64_t total_keys, int32_t sm_count, cudaStream_t stream) {
  CUtensorMap q_map;
  if (!tensor_map_q(&q_map, q, static_cast<uint64_t>(a.total_q), static_cast<uint64_t>(a.hq),
                    static_cast<uint64_t>(g.d), static_cast<uint32_t>(a.group),
                    static_cast<uint32_t>(a.tokens_per_tile)))
    return cudaErrorInvalidValue;
  const int64_t sms = sm_count > 0 ? sm_count : 1;
  // query tiles of a request, about
  int64_t tokens = (static_cast<int64_t>(a.total_q) + a.batch - 1) / a.batch;
  if (a.num_last > 0) tokens = std::min<int64_t>(tokens, a.num_last);
  const int64_t query_tiles = (tokens + a.tokens_per_tile - 1) / a.tokens_per_tile;
  // (a bound on a request's counted query tiles)
  const int64_t most = a.num_last > 0 ? std::min(a.num_last, a.total_q) : a.total_q;
  if (most <= kFewTiles * a.tokens_per_tile) {
    const int64_t ranges = std::max<int64_t>(1, sms / g.hkv);
    const int64_t grid = ranges * g.hkv;
    if (a.cap_log2 > 0.f)
      return g.d == 128 ? launch_few<128, kCap>(q_map, a, grid, stream)
                        : launch_few<64, kCap>(q_map, a, grid, stream);
    return g.d == 128 ? launch_few<128, kPlain>(q_map, a, grid, stream)
                      : launch_few<64, kPlain>(q_map, a, grid, stream);
  }
  // CTAs of a cluster. A wave of the SMs takes about the time of kTurn units (start, K, the
  // meeting) and its items' units: those of the longest where one wave holds them all, else
  // of the average one (blocks of the chunk's own keys are seen by fewer queries). The
  // longest chunk of a batch is taken to be one and a half times the mean. Measured at 1,
  // 2, 4, 8 CTAs, D = 128: 6 chunks of up to 701 tokens, 28 : 4 heads 60, 49, 60, 107 us (2
  // taken); 1 of 2048, 32 : 8 heads 58, 34, 31, 58 (4); 1 of 512 after 3584 22, 30, 46, 86
  // (1); 1 of 1024 after 3840 35, 43 (1); 2 of up to 2048 99, 76, 104, 186 (2); 1 of 8192,
  // 16 : 2 heads 412, 212, 112, 157 (4).
  constexpr double kTurn = 20;
  const double keys = static_cast<double>(total_keys);
  const double blocks = g.hkv * (keys / kKeys + a.batch / 2.);
  const double longest = kTiles * static_cast<double>(query_tiles) * (a.batch > 1 ? 1.5 : 1.);
  const double own = std::min(1., static_cast<double>(tokens) * a.batch / std::max(keys, 1.));
  const double average = kTiles * static_cast<double>(query_tiles) * (1. - own / 2);
  auto cost = [&](int ctas) {
    // (the number of blocks is known to about a twentieth)
    const double waves = std::ceil(blocks * ctas / static_cast<double>(sms) - 0.05);
    return waves <= 1. ? kTurn + longest / ctas : waves * (kTurn + average / ctas);
  };
  int size = 1;
  for (int ctas = 2; ctas <= kMaxMassCluster && ctas <= query_tiles; ctas *= 2)
    if (cost(ctas) < cost(size)) size = ctas;
  int64_t items = g.hkv * ((total_keys + kKeys - 1) / kKeys + a.batch);  // or fewer
  // a CTA an item, within bounds (items past them go round)
  items = std::min<int64_t>(items, size > 1 ? int64_t(1) << 20 : 6 * sms);
  return g.d == 128 ? launch_d<128>(q_map, a, items, size, stream)
                    : launch_d<64>(q_map, a, items, size, stream);
}

}  // namespace pkv
