// decode_mass.cu - decode attention that adds each key's attention weight to what
// the key has received so far.
//
// Mathematics, per request b, kv head h and key i of its n keys, with the scores s
// and log-sum-exp of plain decode (under a soft cap, if any):
//   mass[row, h, i] = (i < n - 1 ? mass[row, h, i] : 0) + sum over the group's q
//   heads of exp(s_i - lse)
// A head with a score that is NaN or +inf has a sum of NaN: it is kept through the partial
// states and the merges (sums are compared with zero, not for being positive), so that lse, o
// and every weight of the kv head are NaN, not only what its own split adds.
//
// The weights need the row's sum, which is known only when every split is done.
// The decode kernel therefore leaves its scores (4 bytes a key and q head, where K
// and V are 4 D / group) in the workspace and a second kernel, which merges the
// splits anyway, turns them into weights: they are mostly still in L2. Going over K
// again instead would cost half of the call's bytes.
//
// Probabilities enter the product with V as two bf16 terms (2^-14.4 of each), so that o is as
// good as its own rounding. With one term it is off by up to 2^-8 of sum p |v| besides, which
// is more than o itself where values cancel, and 64 rows of up to 4096 keys take 87.7 us
// instead of 88.7.
//
// Bound by memory: K and V once, the weights read and written once, the scores
// written and read once. Measured: 64 rows of up to 4096 keys, 32 : 8 heads of 128, 89 us
// (0.79 of the copy rate; plain decode's two launches take 78 of them), 5 rows of up to
// 65537, 28 : 4 heads, 92 (0.70; 82).
#include <algorithm>

#include "decode_common.cuh"
#include "launch.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

template <int D, typename Args>
__global__ void __launch_bounds__(kDecodeThreads, 2) decode_scores_kernel(const Args a) {
  extern __shared__ __align__(128) uint8_t smem[];
  grid_dependency_wait();
  grid_dependents_launch();
  decode_body<D, kDecodeStages>(a, blockIdx.x, blockIdx.y, blockIdx.z, threadIdx.x, smem,
                                [] { __syncthreads(); });
}

// The same in one launch, for plans of a few splits whose clusters are all resident: the
// CTAs of a row's splits (of one kv head) are a cluster; after a barrier over it, which
// makes their states visible, each turns its own keys' scores into weights, and the
// heads' states are merged by the cluster's warps in turn. A launch less for the host:
// 3 rows of up to 600 keys 10.5 us a call from Python instead of 13.4, 8 of up to 1500, 32 :
// 8 heads of 128, 12.2 instead of 13.1; on the GPU alike. Where the clusters are not all
// resident it is slower (16 rows of up to 1000 18.9 us, 13.0 in two launches).
constexpr int kClusterSplits = 8;
constexpr int kClusterCtasPerSm = 2;

template <int D, typename Args>
__global__ void __launch_bounds__(kDecodeThreads, 2)
    decode_mass_cluster_kernel(const Args a, float *key_mass, int64_t mass_stride) {
  constexpr int kCols = D / 32;  // per lane
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_lse[8];
  grid_dependency_wait();
  grid_dependents_launch();
  const int h = static_cast<int>(blockIdx.x), split = static_cast<int>(blockIdx.y);
  const int b = static_cast<int>(blockIdx.z);
  decode_body<D, kDecodeStages>(a, h, split, b, threadIdx.x, smem, [] { __syncthreads(); });
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  const RowInfo ri = row_info(a, b, false);
  const int ns = ri.nsplit;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t pair0 = static_cast<int64_t>(b) * a.hq + h * a.group;
  for (int g = warp; g < a.group; g += kDecodeWarps) {
    const float *pl = a.part_lse + (pair0 + g) * a.pstride;
    const float x = lane < ns ? pl[lane] : -INFINITY;
    float m = x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float ref = m == -INFINITY ? 0.f : m;
    const float e = expf(x - ref);
    float l = e;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float lse = l != 0.f ? ref + logf(l) : -INFINITY;
    if (lane == 0) s_lse[g] = l != 0.f ? lse * kLog2e : INFINITY;
    if (g % static_cast<int>(gridDim.y) != split) continue;  // (a CTA of the cluster a head)
    const float *po = a.part_o + (pair0 + g) * a.pstride * D + lane * kCols;
    float v[kClusterSplits][kCols], o[kCols];
#pragma unroll
    for (int u = 0; u < kClusterSplits; ++u)
#pragma unroll
      for (int c = 0; c < kCols; ++c) v[u][c] = u < ns ? po[static_cast<int64_t>(u) * D + c] : 0.f;
#pragma unroll
    for (int c = 0; c < kCols; ++c) o[c] = 0.f;
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int u = 0; u < kClusterSplits; ++u) {
      const float w = __shfl_sync(0xffffffffu, e, u) * inv;
#pragma unroll
      for (int c = 0; c < kCols; ++c) o[c] += w * v[u][c];
    }
#pragma unroll
    for (int c = 0; c < kCols; c += 2)
      *reinterpret_cast<uint32_t *>(a.o + (pair0 + g) * D + lane * kCols + c) =
          pack_bf16(o[c], o[c + 1]);
    if (lane == 0 && a.lse) a.lse[pair0 + g] = lse;
  }
  __syncthreads();
  const int n = a.seq_lens[b];
  const int row = a.table_idx ? a.table_idx[b] : b;
  if (row < 0 || n <= 0) return;  // (flagged above, or nothing to add)
  if (n != ri.seq || n > mass_stride || n > a.most_keys) {
    if (split == 0 && h == 0 && threadIdx.x == 0) flag_error(a.err, kErrSeqLen);
    return;
  }
  const int begin = split * a.chunk, end = split >= ns - 1 ? n : begin + a.chunk;
  if (split >= ns) return;
  float *mass = key_mass + (static_cast<int64_t>(row) * a.hkv + h) * mass_stride;
  const float *sc = a.scores + (static_cast<int64_t>(b) * a.hkv + h) * a.score_keys * a.group;
  for (int i = begin + static_cast<int>(threadIdx.x); i < end; i += kDecodeThreads) {
    float sum = i < n - 1 ? __ldcg(mass + i) : 0.f;
    for (int g = 0; g < a.group; ++g)
      if (s_lse[g] != INFINITY)
        sum += decode_exp2(sc[static_cast<int64_t>(i) * a.group + g] - s_lse[g]);
    mass[i] = sum;
  }
}

// Warps of a CTA of the second kernel: one for each head of the group, at least (4 and 8
// for groups of 4: 64 rows of up to 4096 keys 87.7, 89.0 us, 16 of up to 8000 36.2, 38.0).
template <int G>
constexpr int kFinishWarps = G <= 4 ? 4 : 8;
constexpr int kFinishKeys = 1024;  // keys of a CTA that adds weights
constexpr int kFinishBatch = 8;    // states a warp has in flight
// A row's states are merged by a warp a head, beside its first weights, up to this many;
// more of them by a CTA a head. Always a warp, always a CTA: 5 rows of up to 65537 keys (121
// states) 99, 90 us; 64 of up to 4096 (5 states) 89, 93.
constexpr int kFewStates = 16;

struct FinishArgs {
  DecodeScoreArgs<0> d;
  float *mass;
  int64_t mass_stride;
  int32_t merge_ctas;  // CTAs of a (request, kv head) that merge: group, or 0 (few states)
};

// Scores of the group's heads for one key.
template <int G>
__device__ __forceinline__ void load_scores(const float *p, float (&s)[G]) {
  if constexpr (G % 4 == 0) {
#pragma unroll
    for (int g = 0; g < G; g += 4) {
      const float4 v = __ldcs(reinterpret_cast<const float4 *>(p + g));
      s[g] = v.x, s[g + 1] = v.y, s[g + 2] = v.z, s[g + 3] = v.w;
    }
  } else if constexpr (G % 2 == 0) {
#pragma unroll
    for (int g = 0; g < G; g += 2) {
      const float2 v = __ldcs(reinterpret_cast<const float2 *>(p + g));
      s[g] = v.x, s[g + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int g = 0; g < G; ++g) s[g] = __ldcs(p + g);
  }
}

// One warp's share of a head's states: every kStep-th from `first` on, with a running
// maximum; o, m and l are its state.
template <int D>
__device__ __forceinline__ void merge_states(const float *pl, const float *po, int first, int step,
                                             int ns, float (&o)[D / 32], float &m, float &l) {
  constexpr int kCols = D / 32;  // per lane
  m = -INFINITY, l = 0.f;
#pragma unroll
  for (int c = 0; c < kCols; ++c) o[c] = 0.f;
  for (int s0 = first; s0 < ns; s0 += step * kFinishBatch) {
    float lse[kFinishBatch], v[kFinishBatch][kCols];
#pragma unroll
    for (int u = 0; u < kFinishBatch; ++u) {
      const int s = s0 + u * step;
      lse[u] = s < ns ? pl[s] : -INFINITY;
#pragma unroll
      for (int c = 0; c < kCols; ++c) v[u][c] = s < ns ? po[static_cast<int64_t>(s) * D + c] : 0.f;
    }
    float mx = m;
#pragma unroll
    for (int u = 0; u < kFinishBatch; ++u) mx = fmaxf(mx, lse[u]);
    const float ref = mx == -INFINITY ? 0.f : mx;
    const float fac = expf(m - ref);
    m = mx;
    l *= fac;
#pragma unroll
    for (int c = 0; c < kCols; ++c) o[c] *= fac;
#pragma unroll
    for (int u = 0; u < kFinishBatch; ++u) {
      const float w = expf(lse[u] - ref);
      l += w;
#pragma unroll
      for (int c = 0; c < kCols; ++c) o[c] += w * v[u][c];
    }
  }
}

// CTA (x, kv head, request): for x < merge_ctas the states of q head x of the group
// merged, then the weights of kFinishKeys keys each. G: the group.
template <int D, int G>
__global__ void __launch_bounds__(32 * kFinishWarps<G>) decode_mass_kernel(const FinishArgs f) {
  constexpr int kCols = D / 32;  // per lane
  constexpr int kWarps = kFinishWarps<G>, kThreads = 32 * kWarps;
  __shared__ float s_o[kWarps][D];
  __shared__ float2 s_ml[kWarps];
  __shared__ float s_lse[G];
  const auto &a = f.d;
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5, lane = tid & 31;
  const int h = static_cast<int>(blockIdx.y), b = static_cast<int>(blockIdx.z);
  const int64_t pair0 = static_cast<int64_t>(b) * a.hq + h * G;  // of the group's heads
  if (static_cast<int>(blockIdx.x) >= f.merge_ctas) {
    const int chunk = static_cast<int>(blockIdx.x) - f.merge_ctas;
    const RowInfo ri = row_info(a, b, false);
    const int ns = ri.nsplit;
    const int n = a.seq_lens[b];
    const int row = a.table_idx ? a.table_idx[b] : b;
    const bool fits = row >= 0 && n >= 0 && n == ri.seq && n <= f.mass_stride && n <= a.most_keys;
    const int k0 = chunk * kFinishKeys;
    if (!fits && row >= 0 && n > 0 && chunk == 0 && h == 0 && tid == 0)
      flag_error(a.err, kErrSeqLen);
    const bool merges = f.merge_ctas == 0 && chunk == 0;
    const int keys = fits ? n : 0;
    if (k0 >= keys && !merges) return;
    float *mass = f.mass + (static_cast<int64_t>(row) * a.hkv + h) * f.mass_stride;
    constexpr int kPer = kFinishKeys / kThreads;
    float had[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = k0 + u * kThreads + tid;
      had[u] = i < keys - 1 ? __ldcg(mass + i) : 0.f;
    }
    grid_dependency_wait();  // states and scores come from the decode kernel
    // scores and states are asked for together
    const float *sc =
        a.scores + ((static_cast<int64_t>(b) * a.hkv + h) * a.score_keys + k0) * G;
    float s[kPer][G];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = u * kThreads + tid;
      if (k0 + i < keys) load_scores<G>(sc + i * G, s[u]);
    }
    // the log-sum-exp of the group's heads, log2 units: a warp each
    if (warp < G) {
      const float *pl = a.part_lse + (pair0 + warp) * a.pstride;
      float first = lane < ns ? pl[lane] : -INFINITY;
      float m = first;
      for (int t = lane + 32; t < ns; t += 32) m = fmaxf(m, pl[t]);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
      const float ref = m == -INFINITY ? 0.f : m;
      float l = expf(first - ref);
      for (int t = lane + 32; t < ns; t += 32) l += expf(pl[t] - ref);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
      if (lane == 0) s_lse[warp] = l != 0.f ? (ref + logf(l)) * kLog2e : INFINITY;
    }
    __syncthreads();
    float lse[G];  // +inf, no weight, for a row whose every score is -inf
#pragma unroll
    for (int g = 0; g < G; ++g) lse[g] = s_lse[g];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = k0 + u * kThreads + tid;
      if (i >= keys) continue;
      float sum = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (lse[g] != INFINITY) sum += decode_exp2(s[u][g] - lse[g]);
      mass[i] = had[u] + sum;
    }
    if (merges && warp < G) {
      float o[kCols], m, l;
      merge_states<D>(a.part_lse + (pair0 + warp) * a.pstride,
                      a.part_o + (pair0 + warp) * a.pstride * D + lane * kCols, 0, 1, ns, o, m, l);
      const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
      for (int c = 0; c < kCols; c += 2)
        *reinterpret_cast<uint32_t *>(a.o + (pair0 + warp) * D + lane * kCols + c) =
            pack_bf16(o[c] * inv, o[c + 1] * inv);
      if (lane == 0 && a.lse) a.lse[pair0 + warp] = l != 0.f ? m + logf(l) : -INFINITY;
    }
    return;
  }
  const int ns = row_info(a, b, false).nsplit;
  grid_dependency_wait();
  // each warp its share of the states, joined in shared memory
  const int64_t bh = pair0 + blockIdx.x;
  float o[kCols], m, l;
  merge_states<D>(a.part_lse + bh * a.pstride, a.part_o + bh * a.pstride * D + lane * kCols, warp,
                  kWarps, ns, o, m, l);
#pragma unroll
  for (int c = 0; c < kCols; ++c) s_o[warp][lane * kCols + c] = o[c];
  if (lane == 0) s_ml[warp] = make_float2(m, l);
  __syncthreads();
  if (tid >= D / 2) return;  // two columns a thread
  float M = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_ml[w].x);
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f, x = 0.f, y = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float fac = expf(s_ml[w].x - ref);
    L += fac * s_ml[w].y;
    x += fac * s_o[w][2 * tid];
    y += fac * s_o[w][2 * tid + 1];
  }
  const float inv = L > 0.f ? 1.f / L : 0.f;
  *reinterpret_cast<uint32_t *>(a.o + bh * D + 2 * tid) = pack_bf16(x * inv, y * inv);
  if (tid == 0 && a.lse) a.lse[bh] = L != 0.f ? ref + logf(L) : -INFINITY;
}

template <int D, int G>
cudaError_t launch_finish(const FinishArgs &f, dim3 grid, cudaStream_t stream) {
  return launch_pdl(decode_mass_kernel<D, G>, grid, dim3(32 * kFinishWarps<G>), 0, stream, f);
}

template <int D>
cudaError_t launch_finish_group(const FinishArgs &f, dim3 grid, cudaStream_t stream) {
  switch (f.d.group) {
    case 1: return launch_finish<D, 1>(f, grid, stream);
    case 2: return launch_finish<D, 2>(f, grid, stream);
    case 3: return launch_finish<D, 3>(f, grid, stream);
    case 4: return launch_finish<D, 4>(f, grid, stream);
    case 5: return launch_finish<D, 5>(f, grid, stream);
    case 6: return launch_finish<D, 6>(f, grid, stream);
    case 7: return launch_finish<D, 7>(f, grid, stream);
    default: return launch_finish<D, 8>(f, grid, stream);
  }
}

template <int D, typename Args>
cudaError_t launch_scores(const Args &a, dim3 grid, cudaStream_t stream) {
  cudaError_t e = allow_smem(decode_scores_kernel<D, Args>, DecodeSmem<D>::kTotal);
  if (e != cudaSuccess) return e;
  return launch_pdl(decode_scores_kernel<D, Args>, grid, dim3(kDecodeThreads),
                    DecodeSmem<D>::kTotal, stream, a);
}

template <int D, typename Args>
cudaError_t launch_cluster(const Args &a, float *mass, int64_t mass_stride, dim3 grid,
                           cudaStream_t stream) {
  auto kernel = decode_mass_cluster_kernel<D, Args>;
  cudaError_t e = allow_smem(kernel, DecodeSmem<D>::kTotal);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kDecodeThreads);
  cfg.dynamicSmemBytes = DecodeSmem<D>::kTotal;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = grid.y;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a, mass, mass_stride);
}

}  // namespace

DecodeMassLayout decode_mass_layout(int32_t batch, int32_t hq, int32_t hkv, int32_t d,
                                    int32_t max_keys, int32_t sm_count) {
  DecodeMassLayout l{};
  l.plan = plan_decode_rules(batch, hq, hkv, d, max_keys, sm_count);
  l.most_keys = max_keys;
  l.score_keys = (static_cast<int64_t>(max_keys) + 15) & ~int64_t(15);
  const size_t states =
      static_cast<size_t>(decode_rules_states(batch, hq, hkv, max_keys, sm_count));
  l.lse_offset = (states * d * sizeof(float) + 255) & ~size_t(255);
  l.score_offset = l.lse_offset + ((states * sizeof(float) + 255) & ~size_t(255));
  const size_t scores = static_cast<size_t>(batch) * hq * static_cast<size_t>(l.score_keys);
  l.total_bytes = l.score_offset + scores * sizeof(float);
  return l;
}

cudaError_t launch_decode_mass(const PoolGeom &g, int32_t layer, const void *q, void *o,
                               float *lse, float *mass, int64_t mass_stride,
                               const int32_t *page_table, int64_t table_stride,
                               const int32_t *table_idx, const int32_t *seq_lens, int32_t batch,
                               int32_t hq, float scale, const ScoreRules &rules,
                               const DecodeMassLayout &lay, void *workspace, unsigned *err,
                               cudaStream_t stream) {
  DecodeRuleArgs base{};
  base.pool = static_cast<const __nv_bfloat16 *>(g.base);
  base.plane = g.plane;
  base.slots = g.slots;
  base.num_layers = g.num_layers;
  base.layer = layer;
  base.page_size = g.page_size;
  base.hkv = g.hkv;
  base.q = static_cast<const __nv_bfloat16 *>(q);
  base.o = static_cast<__nv_bfloat16 *>(o);
  base.lse = lse;
  base.page_table = page_table;
  base.table_stride = table_stride;
  base.table_idx = table_idx;
  base.seq_lens = seq_lens;
  base.hq = hq;
  base.group = hq / g.hkv;
  base.scale_log2 = scale * kLog2e;
  base.heads_per_cta = lay.plan.heads_per_cta;
  base.warps_per_head = lay.plan.warps_per_head;
  base.chunk = lay.plan.chunk;
  base.splits = lay.plan.splits;
  base.pstride = lay.plan.splits;
  base.force_partial = 1;  // the second kernel merges every row
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  base.part_o = reinterpret_cast<float *>(ws);
  base.part_lse = reinterpret_cast<float *>(ws + lay.lse_offset);
  base.err = err;
  base.rules = rules;
  float *scores = reinterpret_cast<float *>(ws + lay.score_offset);
  const dim3 grid(lay.plan.head_groups, lay.plan.splits, batch);
  const bool cluster = lay.plan.splits <= kClusterSplits &&
                       static_cast<int64_t>(batch) * g.hkv * lay.plan.splits <=
                           kClusterCtasPerSm * static_cast<int64_t>(lay.plan.sm_count);
  auto main = [&](auto args) {
    args.scores = scores;
    args.score_keys = lay.score_keys;
    args.most_keys = lay.most_keys;
    if (cluster)
      return g.d == 128 ? launch_cluster<128>(args, mass, mass_stride, grid, stream)
                        : launch_cluster<64>(args, mass, mass_stride, grid, stream);
    return g.d == 128 ? launch_scores<128>(args, grid, stream)
                      : launch_scores<64>(args, grid, stream);
  };
  const cudaError_t e = rules.cap_log2 > 0.f ? main(DecodeScoreArgs<kRuleCap>(base))
                                             : main(DecodeScoreArgs<0>(base));
  if (e != cudaSuccess || cluster) return e;
  FinishArgs f{DecodeScoreArgs<0>(base), mass, mass_stride,
               lay.plan.splits > kFewStates ? base.group : 0};
  f.d.scores = scores;
  f.d.score_keys = lay.score_keys;
  f.d.most_keys = lay.most_keys;
  const dim3 fgrid(
      f.merge_ctas + static_cast<unsigned>((lay.score_keys + kFinishKeys - 1) / kFinishKeys),
      g.hkv, batch);
  return g.d == 128 ? launch_finish_group<128>(f, fgrid, stream)
                    : launch_finish_group<64>(f, fgrid, stream);
}

}  // namespace pkv
