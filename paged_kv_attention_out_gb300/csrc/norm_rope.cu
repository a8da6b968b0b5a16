// norm_rope.cu - a step's q and k normed and rotated, k and v appended to the
// paged pool, all in one pass over the fused projection's output.
//
// Mathematics, per token t and head (x: the head's D values in fp32):
//   y = x * rsqrt(mean(x^2) + eps) * w          (q and k, if a weight is given)
//   (a, b) -> (a cos - b sin, b cos + a sin)    for each of the rot_dim / 2
//       pairs, angles of positions[t]; (a, b) = (y[m], y[m + rot_dim / 2]), or
//       (y[2m], y[2m + 1]) interleaved; dims rot_dim .. D - 1 pass unrotated
//   q_out[t] = q ; pool[0 | 1, layer, out_loc[t]] = k | v (v bits unchanged)
// Everything from the load to the one rounding to bf16 at the store is fp32.
//
// Bound by memory: each of q, k, v is read once and written once, plus one
// row of the cos / sin table per token. A head row is held by D / 16 lanes,
// two 16-byte chunks each, and a lane's two chunks are the halves of the same
// pairs (chunk l and chunk l + rot_dim / 16), so the rotation needs no
// exchange between lanes and only the norm's sum of squares crosses them (3
// shuffles at D = 128). One CTA of 128 threads takes one token: every thread
// keeps its 8 cosines and sines in registers for all the heads it serves and
// has up to kBatch heads' loads in flight (96 bytes per thread).
#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 3;  // head rows a thread has in flight

struct Chunk {
  float v[8];
};

__device__ __forceinline__ Chunk unpack(uint4 u) {
  Chunk c;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c.v[2 * i] = __uint_as_float(w[i] << 16);
    c.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return c;
}

__device__ __forceinline__ uint4 pack(const Chunk &c) {
  return make_uint4(pack_bf16(c.v[0], c.v[1]), pack_bf16(c.v[2], c.v[3]),
                    pack_bf16(c.v[4], c.v[5]), pack_bf16(c.v[6], c.v[7]));
}

__device__ __forceinline__ Chunk load_weight(const __nv_bfloat16 *w, int chunk) {
  return unpack(__ldg(reinterpret_cast<const uint4 *>(w) + chunk));
}

template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) norm_rope_store_kernel(const NormRopeArgs a) {
  constexpr int kLanes = D / 16;              // lanes per head row
  constexpr int kSlots = kThreads / kLanes;   // head rows a CTA serves at once
  const int l = threadIdx.x % kLanes;
  const int slot = threadIdx.x / kLanes;
  const int hc = a.rot_dim / 16;  // rotated chunk pairs
  // this lane's two chunks: the halves of the same pairs, or two neighbours
  // of the part that is not rotated
  const int c0 = l < hc ? l : 2 * l;
  const int c1 = l < hc ? l + hc : 2 * l + 1;
  const int heads = a.hq + 2 * a.hkv;  // q heads, then k heads, then v heads
  grid_dependency_wait();    // q, k, v may come from the previous kernel
  grid_dependents_launch();  // let the attention kernel that follows get scheduled
  const int64_t t = blockIdx.x;
  const int64_t dst_slot = a.out_loc[t];
  const bool stored = dst_slot >= 0 && dst_slot < a.slots;  // never write outside the pool
  if (!stored && threadIdx.x == 0) flag_error(a.err, kErrOutLoc);
  float cs[8], sn[8];
  if (hc > 0) {
    const int pos = a.positions[t];
    if (pos < 0 || pos >= a.num_positions) {  // uniform over the CTA: the token is skipped
      if (threadIdx.x == 0) flag_error(a.err, kErrPosition);
      return;
    }
    if (l < hc) {
      const float4 *row = reinterpret_cast<const float4 *>(
          a.cos_sin + static_cast<int64_t>(pos) * a.rot_dim);
      // pair m of the chunk halves: angle 8 l + m; interleaved: angles
      // 4 c + m / 2 of chunk c
      const int i0 = kInterleaved ? c0 : 2 * l;
      const int i1 = kInterleaved ? c1 : 2 * l + 1;
      const int half = a.rot_dim / 8;
      const float4 x0 = __ldg(row + i0), x1 = __ldg(row + i1);
      const float4 y0 = __ldg(row + half + i0), y1 = __ldg(row + half + i1);
      cs[0] = x0.x, cs[1] = x0.y, cs[2] = x0.z, cs[3] = x0.w;
      cs[4] = x1.x, cs[5] = x1.y, cs[6] = x1.z, cs[7] = x1.w;
      sn[0] = y0.x, sn[1] = y0.y, sn[2] = y0.z, sn[3] = y0.w;
      sn[4] = y1.x, sn[5] = y1.y, sn[6] = y1.z, sn[7] = y1.w;
    }
  }
  const int64_t row_elems = static_cast<int64_t>(a.hkv) * D;
  for (int h0 = slot; h0 - slot < heads; h0 += kSlots * kBatch) {
    uint4 ra[kBatch], rb[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = h0 + u * kSlots;
      ra[u] = rb[u] = make_uint4(0u, 0u, 0u, 0u);
      if (h < heads) {
        const __nv_bfloat16 *src =
            h < a.hq ? a.q + t * a.q_stride + h * D
                     : (h < a.hq + a.hkv ? a.k + t * a.kv_stride + (h - a.hq) * D
                                         : a.v + t * a.kv_stride + (h - a.hq - a.hkv) * D);
        ra[u] = __ldcs(reinterpret_cast<const uint4 *>(src) + c0);
        rb[u] = __ldcs(reinterpret_cast<const uint4 *>(src) + c1);
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = h0 + u * kSlots;
      const bool is_v = h >= a.hq + a.hkv;
      const __nv_bfloat16 *w = h < a.hq ? a.q_norm : (is_v ? nullptr : a.k_norm);
      Chunk xa = unpack(ra[u]), xb = unpack(rb[u]);
      if (a.q_norm || a.k_norm) {  // uniform: every lane takes part in the shuffles
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += xa.v[i] * xa.v[i] + xb.v[i] * xb.v[i];
#pragma unroll
        for (int x = kLanes / 2; x > 0; x >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, x);
        if (w) {
          const float r = rsqrtf(ss * (1.f / D) + a.eps);
          const Chunk wa = load_weight(w, c0), wb = load_weight(w, c1);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            xa.v[i] = xa.v[i] * r * wa.v[i];
            xb.v[i] = xb.v[i] * r * wb.v[i];
          }
        }
      }
      if (h >= heads) continue;
      if (l < hc && !is_v) {
        if (kInterleaved) {
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const float p0 = xa.v[2 * m], p1 = xa.v[2 * m + 1];
            xa.v[2 * m] = p0 * cs[m] - p1 * sn[m];
            xa.v[2 * m + 1] = p1 * cs[m] + p0 * sn[m];
            const float r0 = xb.v[2 * m], r1 = xb.v[2 * m + 1];
            xb.v[2 * m] = r0 * cs[4 + m] - r1 * sn[4 + m];
            xb.v[2 * m + 1] = r1 * cs[4 + m] + r0 * sn[4 + m];
          }
        } else {
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            const float p0 = xa.v[m], p1 = xb.v[m];
            xa.v[m] = p0 * cs[m] - p1 * sn[m];
            xb.v[m] = p1 * cs[m] + p0 * sn[m];
          }
        }
      }
      __nv_bfloat16 *dst;
      if (h < a.hq) {
        dst = a.q_out + (t * a.hq + h) * D;
      } else {
        if (!stored) continue;
        const int64_t plane = (is_v ? a.num_layers : 0) + a.layer;
        dst = a.pool + plane * a.plane + dst_slot * row_elems +
              (h - a.hq - (is_v ? a.hkv : 0)) * D;
      }
      // v (and q, k when nothing applies) go out with the bits they came in
      const bool same = is_v || (!w && l >= hc);
      reinterpret_cast<uint4 *>(dst)[c0] = same ? ra[u] : pack(xa);
      reinterpret_cast<uint4 *>(dst)[c1] = same ? rb[u] : pack(xb);
    }
  }
}

}  // namespace

cudaError_t launch_norm_rope_store(const PoolGeom &g, const NormRopeArgs &a, int64_t n,
                                   bool interleaved, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(n)), block(kThreads);
  if (g.d == 128)
    return interleaved ? launch_pdl(norm_rope_store_kernel<128, true>, grid, block, 0, stream, a)
                       : launch_pdl(norm_rope_store_kernel<128, false>, grid, block, 0, stream, a);
  return interleaved ? launch_pdl(norm_rope_store_kernel<64, true>, grid, block, 0, stream, a)
                     : launch_pdl(norm_rope_store_kernel<64, false>, grid, block, 0, stream, a);
}

}  // namespace pkv
