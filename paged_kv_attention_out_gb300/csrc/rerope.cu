// rerope.cu - cached keys turned in place from the angles they were stored at to
// those of other positions (after an eviction, or where a cached run is used at
// another offset) or of other frequencies (a context that outgrew its training).
//
// Mathematics, per key i of a row, kv head and pair m of its rot_dim / 2 pairs:
//   angle = new_pos * new_freq[m] - old_pos * old_freq[m]
//   (a, b) -> factor * (a cos - b sin, b cos + a sin)
// in fp32, rounded once to bf16. Angles are exact before their sine: a frequency
// is kept as a 64-bit binary fraction of a turn, so position times frequency is an
// integer product modulo 2^64 and whole turns drop out by themselves. The fraction
// is off by 2^-52 of its value (1 / (2 pi) and the product, rounded in 64 bits) and by 2^-64, a
// position of 2^31 radians by 2^-23 of a turn; an fp32 product would be off by 2^-24 of
// the angle, 0.008 radians at 131072.
//
// Sines and cosines: polynomials, off by 2^-23.2 at most, so that a turned value is off by
// 2^-21.2 of its pair's radius before it is rounded. Where positions differ by kv head, angles
// are computed for every head and bound the call: there they come from the hardware,
// off by up to 2^-21.2 on [-pi, pi] (CUDA's stated bound), a turned value by 2^-19.3 of
// the radius, where half a step of bf16 is 2^-9 of the value or more. 8 rows of up to 16000
// keys, 8 heads of 128: 62.8 us, with the polynomials 68.1; one position a key, 8 rows of up
// to 32768: 84.4 us with either.
//
// Bound by memory: the rotated part of every key is read and written once, and
// nothing is read for the angles but the positions. rot_dim / 16 lanes hold a
// key's pairs, both chunks of 16 bytes of the same pairs, compute their eight
// angles once and use them for every kv head (once a head where positions differ
// by head). A lane writes nothing where none of its eight pairs turns under a factor of
// one; its first heads are read all the same, since they come while the angles are computed.
// Measured: 8 rows of up to 32768 keys, 8 heads of 128, 84 us (0.90 of the copy rate).
#include "bf16x8.cuh"
#include "pkv_common.cuh"
#include "pkv_internal.h"
#include "row_units.cuh"

namespace pkv {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;  // heads a thread has in flight

// The fraction of a turn, in units of 2^-64, that a frequency adds per position.
__device__ __forceinline__ uint64_t turn_fraction(float freq) {
  double t = static_cast<double>(freq) * 0.15915494309189535;  // 1 / (2 pi)
  t -= floor(t);
  // (below 1 as a double; the product is exact. Not finite: some fraction.)
  return static_cast<uint64_t>(t * 18446744073709551616.0);
}

// A load that stays where it is written.
__device__ __forceinline__ uint4 load_here(const uint4 *p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Of 2^-32 turns.
constexpr float kRadians = 1.4629180792671596e-9f;  // 2 pi / 2^32

// Sine and cosine of t / 2^32 turns, off by 2^-23.2 at most: polynomials (least maximum error,
// by reweighted least squares) in w quarter turns, |w| <= 1/2, round the nearest quarter.
__device__ __forceinline__ void sin_cos_turn(uint32_t t, float *sn, float *cs) {
  const uint32_t quarter = (t + 0x20000000u) >> 30;
  const float w = static_cast<float>(static_cast<int32_t>(t << 2)) * 0x1p-32f;
  const float z = w * w;
  float s = fmaf(z, -0.0046021771f, 0.079680227f);
  s = fmaf(z, s, -0.64596349f);
  s = w * fmaf(z, s, 1.5707964f);
  float c = fmaf(z, 0.00091181189f, -0.020863504f);
  c = fmaf(z, c, 0.25366962f);
  c = fmaf(z, c, -1.2337005f);
  c = fmaf(z, c, 1.f);
  const bool odd = quarter & 1;
  *sn = __uint_as_float(__float_as_uint(odd ? c : s) ^ (quarter & 2) << 30);
  *cs = __uint_as_float(__float_as_uint(odd ? s : c) ^ (quarter + 1 & 2) << 30);
}

struct Turns {
  float cs[8], sn[8];
  bool any;  // some angle is not zero
};

// kByHead: positions differ by kv head.
template <int D, bool kInterleaved, bool kByHead>
__global__ void __launch_bounds__(kRopeThreads, 3) rerope_kernel(const RopeArgs a) {
  __shared__ uint64_t s_old[D / 2], s_new[D / 2];
  const int tid = threadIdx.x;
  const int half = a.rot_dim / 2;
  grid_dependency_wait();  // keys, positions and frequencies may come from the previous kernel
  grid_dependents_launch();
  bool differ = false;
  for (int m = tid; m < half; m += kRopeThreads) {
    s_old[m] = a.old_freq ? turn_fraction(a.old_freq[m]) : 0;
    s_new[m] = a.new_freq ? turn_fraction(a.new_freq[m]) : 0;
    differ = s_old[m] != s_new[m];
  }
  // the same frequencies: only the distance moved counts
  const bool same = !__syncthreads_or(differ);
  const int hc = a.rot_dim / 16;                    // lanes per head row
  const int lanes = hc * a.head_parts;              // lanes per key
  const int per_cta = kRopeThreads / lanes;         // keys per unit
  const int heads = (a.hkv + a.head_parts - 1) / a.head_parts;  // of a lane
  const int64_t capacity = min(a.table_stride * a.page_size, static_cast<int64_t>(kMaxRowKeys));
  auto keys_of = [&](int r) -> int {  // of a request that is computed, else 0
    const int n = a.seq_lens[r];
    const bool fits = n >= 0 && n <= capacity && (!a.positioned || n <= a.position_stride);
    return fits && !(a.table_idx && a.table_idx[r] < 0) ? n : 0;
  };
  if (blockIdx.x == 0) {
    for (int r = tid; r < a.batch; r += kRopeThreads) {
      const int n = a.seq_lens[r];
      if (n < 0 || n > capacity || (a.positioned && n > a.position_stride))
        flag_error(a.err, kErrSeqLen);
      if (a.table_idx && a.table_idx[r] < 0) flag_error(a.err, kErrTableIdx);
    }
  }
  const int l = tid % lanes % hc;
  const int first = tid % lanes / hc * heads, last = min(a.hkv, first + heads);
  const int c0 = l, c1 = l + hc;  // 16-byte chunks of this lane
  for (int64_t unit = blockIdx.x;; unit += gridDim.x) {
    const RowUnit ru = find_row_unit<kRopeThreads>(
        unit, a.batch, [&](int r) { return (keys_of(r) + per_cta - 1) / per_cta; });
    if (ru.r < 0) break;
    const int r = ru.r;
    const int n = a.seq_lens[r];
    const int64_t i64 = ru.local * per_cta + tid / lanes;
    if (tid >= per_cta * lanes || i64 >= n) continue;
    const int i = static_cast<int>(i64);
    const int row = a.table_idx ? a.table_idx[r] : r;
    const int page = a.page_of(i);
    const int entry = a.page_table[row * a.table_stride + page];
    const int64_t slot = static_cast<int64_t>(entry) * a.page_size + (i - page * a.page_size);
    if (entry < 0 || slot >= a.slots) {
      if (l == 0) flag_error(a.err, kErrPage);
      continue;
    }
    uint4 *key = reinterpret_cast<uint4 *>(a.plane + slot * a.hkv * D);
    auto turns_of = [&](int64_t old_pos, int64_t new_pos) {
      Turns t;
      t.any = a.factor != 1.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int m = kInterleaved ? 4 * (e < 4 ? c0 : c1) + (e & 3) : 8 * l + e;
        const uint64_t turn = same ? static_cast<uint64_t>(new_pos - old_pos) * s_new[m]
                                   : static_cast<uint64_t>(new_pos) * s_new[m] -
                                         static_cast<uint64_t>(old_pos) * s_old[m];
        t.any = t.any || turn != 0;
        const uint32_t part = static_cast<uint32_t>(turn >> 32);
        float sn, cs;
        if constexpr (kByHead) {
          const float x = static_cast<float>(static_cast<int32_t>(part)) * kRadians;  // [-pi, pi)
          sn = __sinf(x);
          cs = __cosf(x);
        } else {
          sin_cos_turn(part, &sn, &cs);
        }
        t.sn[e] = sn * a.factor;
        t.cs[e] = cs * a.factor;
      }
      return t;
    };
    // a key's entry in the positions, of kv head 0
    const int64_t at = static_cast<int64_t>(r) * a.position_heads * a.position_stride + i;
    auto old_of = [&](int h) { return a.old_pos ? a.old_pos[at + h * a.position_stride] : i; };
    auto new_of = [&](int h) { return a.new_pos ? a.new_pos[at + h * a.position_stride] : i; };
    // the first heads' chunks come while the angles are computed
    uint4 ra[kRopeBatch], rb[kRopeBatch];
    int was[kByHead ? kRopeBatch : 1], is[kByHead ? kRopeBatch : 1];
    auto load = [&](int h0) {
#pragma unroll
      for (int u = 0; u < kRopeBatch; ++u) {
        if (h0 + u >= last) continue;
        ra[u] = load_here(key + (h0 + u) * (D / 8) + c0);
        rb[u] = load_here(key + (h0 + u) * (D / 8) + c1);
        if constexpr (kByHead) was[u] = old_of(h0 + u), is[u] = new_of(h0 + u);
      }
    };
    load(first);
    Turns t;
    if constexpr (!kByHead) {
      t = turns_of(old_of(0), new_of(0));
      if (!t.any) continue;
    }
    for (int h0 = first; h0 < last; h0 += kRopeBatch) {
      if (h0 > first) load(h0);
#pragma unroll
      for (int u = 0; u < kRopeBatch; ++u) {
        if (h0 + u >= last) continue;
        if constexpr (kByHead) t = turns_of(was[u], is[u]);
        if (!t.any) continue;
        Bf16x8 xa = unpack_bf16x8(ra[u]), xb = unpack_bf16x8(rb[u]);
        if (kInterleaved) {
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const float p0 = xa.v[2 * m], p1 = xa.v[2 * m + 1];
            xa.v[2 * m] = p0 * t.cs[m] - p1 * t.sn[m];
            xa.v[2 * m + 1] = p1 * t.cs[m] + p0 * t.sn[m];
            const float r0 = xb.v[2 * m], r1 = xb.v[2 * m + 1];
            xb.v[2 * m] = r0 * t.cs[4 + m] - r1 * t.sn[4 + m];
            xb.v[2 * m + 1] = r1 * t.cs[4 + m] + r0 * t.sn[4 + m];
          }
        } else {
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            const float p0 = xa.v[m], p1 = xb.v[m];
            xa.v[m] = p0 * t.cs[m] - p1 * t.sn[m];
            xb.v[m] = p1 * t.cs[m] + p0 * t.sn[m];
          }
        }
        key[(h0 + u) * (D / 8) + c0] = pack_bf16x8(xa);
        key[(h0 + u) * (D / 8) + c1] = pack_bf16x8(xb);
      }
    }
  }
}

template <int D, bool kInterleaved>
cudaError_t launch(const RopeArgs &args, int64_t total_keys, int32_t sm_count,
                   cudaStream_t stream) {
  RopeArgs a = args;
  const int64_t sms = sm_count > 0 ? sm_count : 1;
  // A key's heads to one lane set, which computes its angles once, or shared out while
  // there are fewer CTAs than SMs: 1 row of 509 keys of 4 kv heads of 64, 32 dims rotated,
  // 5.5 us instead of 7.5; 8 rows of up to 16000 keys of 8 kv heads, 16 dims (208 CTAs)
  // 20.8 us with one set, 22.0 with more.
  auto units = [&] {
    const int64_t per_cta = kRopeThreads / (a.rot_dim / 16 * a.head_parts);
    return (total_keys + per_cta - 1) / per_cta + a.batch;
  };
  a.head_parts = 1;
  while (2 * a.head_parts <= a.hkv && 2 * a.head_parts * (a.rot_dim / 16) <= kRopeThreads &&
         units() < sms)
    a.head_parts *= 2;
  const dim3 grid(static_cast<unsigned>(units() < 32 * sms ? units() : 32 * sms));
  const dim3 block(kRopeThreads);
  return a.position_heads != 1
             ? launch_pdl(rerope_kernel<D, kInterleaved, true>, grid, block, 0, stream, a)
             : launch_pdl(rerope_kernel<D, kInterleaved, false>, grid, block, 0, stream, a);
}

}  // namespace

cudaError_t launch_rerope(const PoolGeom &g, const RopeArgs &a, bool interleaved,
                          int64_t total_keys, int32_t sm_count, cudaStream_t stream) {
  if (g.d == 128)
    return interleaved ? launch<128, true>(a, total_keys, sm_count, stream)
                       : launch<128, false>(a, total_keys, sm_count, stream);
  return interleaved ? launch<64, true>(a, total_keys, sm_count, stream)
                     : launch<64, false>(a, total_keys, sm_count, stream);
}

}  // namespace pkv
