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
// shuffles at D = 128). A thread keeps its 8 cosines and sines, and one
// tensor's norm weights, in registers for all the heads it serves.
// Few tokens (at most four per SM): a CTA of 128 threads per token, for
// latency. Many: one warp per token. The narrower the CTA, the more tokens are
// in flight on an SM while each waits for its position, its table row and its
// heads in turn: 16384 tokens, 32/8 heads of 128, norm and full rotation take
// 83 us with 128 threads a token, 77 with 64, 69 with 32 (0.88 of the copy
// rate; 66 without the norm), two rows in flight per thread (three: 70, four:
// 73). A resident set of warps looping over the tokens was slower (76).
#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

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

// The cosines and sines of a lane's eight pairs.
struct Turn {
  float cs[8], sn[8];
};

template <int D, bool kInterleaved, int kThreads>
__global__ void __launch_bounds__(kThreads) norm_rope_store_kernel(const NormRopeArgs a) {
  constexpr int kLanes = D / 16;              // lanes per head row
  constexpr int kSlots = kThreads / kLanes;   // head rows a CTA serves at once
  constexpr int kBatch = 2;                   // rows a thread has in flight
  const int l = threadIdx.x % kLanes;
  const int slot = threadIdx.x / kLanes;
  const int hc = a.rot_dim / 16;  // rotated chunk pairs
  // this lane's two chunks: the halves of the same pairs, or two neighbours
  // of the part that is not rotated
  const bool turned = l < hc;
  const int c0 = turned ? l : 2 * l;
  const int c1 = turned ? l + hc : 2 * l + 1;
  grid_dependency_wait();    // q, k, v may come from the previous kernel
  grid_dependents_launch();  // let the attention kernel that follows get scheduled
  const int64_t t = blockIdx.x;
  const int64_t dst_slot = a.out_loc[t];
  const int pos = hc > 0 ? a.positions[t] : 0;

  // The heads of one tensor: rows src + h D -> dst + h D.
  auto rows = [&](const __nv_bfloat16 *src, __nv_bfloat16 *dst, int heads,
                  const __nv_bfloat16 *weight, bool plain, const Turn &turn) {
    uint4 wa_bits = make_uint4(0u, 0u, 0u, 0u), wb_bits = wa_bits;
    if (weight) {
      wa_bits = __ldg(reinterpret_cast<const uint4 *>(weight) + c0);
      wb_bits = __ldg(reinterpret_cast<const uint4 *>(weight) + c1);
    }
    for (int h0 = slot; h0 - slot < heads; h0 += kSlots * kBatch) {  // (uniform over the CTA)
      uint4 ra[kBatch], rb[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int h = h0 + u * kSlots;
        ra[u] = rb[u] = make_uint4(0u, 0u, 0u, 0u);
        if (h < heads) {
          ra[u] = __ldcs(reinterpret_cast<const uint4 *>(src + h * D) + c0);
          rb[u] = __ldcs(reinterpret_cast<const uint4 *>(src + h * D) + c1);
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int h = h0 + u * kSlots;
        if (!plain) {
          Chunk xa = unpack(ra[u]), xb = unpack(rb[u]);
          if (weight) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss += xa.v[i] * xa.v[i] + xb.v[i] * xb.v[i];
#pragma unroll
            for (int x = kLanes / 2; x > 0; x >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, x);
            const float r = rsqrtf(ss * (1.f / D) + a.eps);
            const Chunk wa = unpack(wa_bits), wb = unpack(wb_bits);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              xa.v[i] = xa.v[i] * r * wa.v[i];
              xb.v[i] = xb.v[i] * r * wb.v[i];
            }
          }
          if (turned) {
            if (kInterleaved) {
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                const float p0 = xa.v[2 * m], p1 = xa.v[2 * m + 1];
                xa.v[2 * m] = p0 * turn.cs[m] - p1 * turn.sn[m];
                xa.v[2 * m + 1] = p1 * turn.cs[m] + p0 * turn.sn[m];
                const float r0 = xb.v[2 * m], r1 = xb.v[2 * m + 1];
                xb.v[2 * m] = r0 * turn.cs[4 + m] - r1 * turn.sn[4 + m];
                xb.v[2 * m + 1] = r1 * turn.cs[4 + m] + r0 * turn.sn[4 + m];
              }
            } else {
#pragma unroll
              for (int m = 0; m < 8; ++m) {
                const float p0 = xa.v[m], p1 = xb.v[m];
                xa.v[m] = p0 * turn.cs[m] - p1 * turn.sn[m];
                xb.v[m] = p1 * turn.cs[m] + p0 * turn.sn[m];
              }
            }
          }
          if (weight || turned) {  // else the bits that came in go out
            ra[u] = pack(xa);
            rb[u] = pack(xb);
          }
        }
        if (h < heads) {
          reinterpret_cast<uint4 *>(dst + h * D)[c0] = ra[u];
          reinterpret_cast<uint4 *>(dst + h * D)[c1] = rb[u];
        }
      }
    }
  };

  Turn turn;
  const bool stored = dst_slot >= 0 && dst_slot < a.slots;  // never write outside the pool
  const bool placed = hc == 0 || (pos >= 0 && pos < a.num_positions);
  if (threadIdx.x == 0) {
    if (!stored) flag_error(a.err, kErrOutLoc);
    if (!placed) flag_error(a.err, kErrPosition);
  }
  if (!placed) return;  // the token is skipped
  if (turned) {
    const float4 *row =
        reinterpret_cast<const float4 *>(a.cos_sin + static_cast<int64_t>(pos) * a.rot_dim);
    // pair m of the chunk halves: angle 8 l + m; interleaved: angles 4 c + m / 2
    // of chunk c
    const int i0 = kInterleaved ? c0 : 2 * l;
    const int i1 = kInterleaved ? c1 : 2 * l + 1;
    const int half = a.rot_dim / 8;
    const float4 x0 = __ldg(row + i0), x1 = __ldg(row + i1);
    const float4 y0 = __ldg(row + half + i0), y1 = __ldg(row + half + i1);
    turn.cs[0] = x0.x, turn.cs[1] = x0.y, turn.cs[2] = x0.z, turn.cs[3] = x0.w;
    turn.cs[4] = x1.x, turn.cs[5] = x1.y, turn.cs[6] = x1.z, turn.cs[7] = x1.w;
    turn.sn[0] = y0.x, turn.sn[1] = y0.y, turn.sn[2] = y0.z, turn.sn[3] = y0.w;
    turn.sn[4] = y1.x, turn.sn[5] = y1.y, turn.sn[6] = y1.z, turn.sn[7] = y1.w;
  }
  if (stored) {
    const int64_t row_elems = static_cast<int64_t>(a.hkv) * D;
    __nv_bfloat16 *k_dst = a.pool + a.layer * a.plane + dst_slot * row_elems;
    rows(a.v + t * a.kv_stride, k_dst + a.num_layers * a.plane, a.hkv, nullptr, true, turn);
    rows(a.k + t * a.kv_stride, k_dst, a.hkv, a.k_norm, false, turn);
  }
  rows(a.q + t * a.q_stride, a.q_out + t * a.hq * D, a.hq, a.q_norm, false, turn);
}

template <int D, bool kInterleaved>
cudaError_t launch(const NormRopeArgs &a, int32_t sm_count, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.n));
  if (a.n <= 4 * static_cast<int64_t>(sm_count))
    return launch_pdl(norm_rope_store_kernel<D, kInterleaved, 128>, grid, dim3(128), 0, stream, a);
  return launch_pdl(norm_rope_store_kernel<D, kInterleaved, 32>, grid, dim3(32), 0,
                    stream, a);
}

}  // namespace

cudaError_t launch_norm_rope_store(const PoolGeom &g, const NormRopeArgs &a, bool interleaved,
                                   int32_t sm_count, cudaStream_t stream) {
  if (g.d == 128)
    return interleaved ? launch<128, true>(a, sm_count, stream)
                       : launch<128, false>(a, sm_count, stream);
  return interleaved ? launch<64, true>(a, sm_count, stream)
                     : launch<64, false>(a, sm_count, stream);
}

}  // namespace pkv
