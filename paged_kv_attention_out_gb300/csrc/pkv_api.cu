// pkv_api.cu - the C ABI declared in include/pkv.h: argument validation,
// per-device facts (compute capability, SM count), the decode split plan,
// and the kernel launches. No call here allocates, synchronises (except
// pkv_read_device_errors, documented as a debugging aid) or changes the
// current device.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <mutex>

#include "pkv.h"
#include "pkv_internal.h"
#include "score_rules.cuh"

namespace {

thread_local char g_last_error[256] = "";

// Device error word (PKV_DEVERR_* bits), one per device that loads the library.
__device__ unsigned int g_device_errors;

struct DevInfo {
  bool init = false;
  pkv_status status = PKV_OK;
  int sm_count = 0;
  unsigned *err = nullptr;
};

constexpr int kMaxDevices = 64;
DevInfo g_dev[kMaxDevices];
std::mutex g_mu;

pkv_status fail(pkv_status s, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
  va_end(ap);
  return s;
}

pkv_status cuda_fail(cudaError_t e, const char *what) {
  return fail(PKV_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Facts about the current device, computed once per device.
pkv_status device_info(DevInfo **out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(PKV_ERR_UNSUPPORTED, "device ordinal %d", dev);
  std::lock_guard<std::mutex> lock(g_mu);
  DevInfo &d = g_dev[dev];
  if (!d.init) {
    int major = 0, minor = 0, sms = 0;
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return cuda_fail(e, "cudaDeviceGetAttribute");
    if (major != 10 || minor != 3) {
      d.status = PKV_ERR_UNSUPPORTED;
    } else {
      void *p = nullptr;
      if ((e = cudaGetSymbolAddress(&p, g_device_errors)) != cudaSuccess)
        return cuda_fail(e, "cudaGetSymbolAddress(device error word)");
      d.err = static_cast<unsigned *>(p);
      d.status = PKV_OK;
    }
    d.sm_count = sms;
    d.init = true;
  }
  if (d.status != PKV_OK)
    return fail(d.status, "device %d is not compute capability 10.3 (sm_103a)", dev);
  *out = &d;
  return PKV_OK;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

pkv_status check_pool(const pkv_pool *pool, int32_t layer, pkv::PoolGeom *g) {
  if (!pool) return fail(PKV_ERR_INVALID_ARG, "pool is NULL");
  if (!pool->base) return fail(PKV_ERR_INVALID_ARG, "pool->base is NULL");
  if (!aligned(pool->base, 16)) return fail(PKV_ERR_INVALID_ARG, "pool->base not 16-byte aligned");
  if (pool->num_layers <= 0 || pool->num_pages <= 0 || pool->page_size <= 0 ||
      pool->num_kv_heads <= 0)
    return fail(PKV_ERR_INVALID_ARG, "pool sizes must be positive");
  if (pool->head_dim != 64 && pool->head_dim != 128)
    return fail(PKV_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", pool->head_dim);
  if (layer < 0 || layer >= pool->num_layers)
    return fail(PKV_ERR_INVALID_ARG, "layer %d outside [0, %d)", layer, pool->num_layers);
  const int64_t slots = pool->num_pages * static_cast<int64_t>(pool->page_size);
  if (slots / pool->page_size != pool->num_pages || slots > (int64_t(1) << 40))
    return fail(PKV_ERR_INVALID_ARG, "pool too large");
  g->base = pool->base;
  g->slots = slots;
  g->plane = slots * pool->num_kv_heads * pool->head_dim;
  g->num_layers = pool->num_layers;
  g->page_size = pool->page_size;
  g->hkv = pool->num_kv_heads;
  g->d = pool->head_dim;
  return PKV_OK;
}

int32_t effective_hint(int32_t hint) { return hint < 1 ? 1 : hint; }

}  // namespace

namespace pkv {
pkv_status fail_status(pkv_status s, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
  va_end(ap);
  return s;
}
}  // namespace pkv

extern "C" {

pkv_status pkv_init(void) {
  DevInfo *d = nullptr;
  return device_info(&d);
}

const char *pkv_status_string(pkv_status s) {
  switch (s) {
    case PKV_OK: return "PKV_OK";
    case PKV_ERR_INVALID_ARG: return "PKV_ERR_INVALID_ARG";
    case PKV_ERR_UNSUPPORTED: return "PKV_ERR_UNSUPPORTED";
    case PKV_ERR_WORKSPACE_TOO_SMALL: return "PKV_ERR_WORKSPACE_TOO_SMALL";
    case PKV_ERR_CUDA: return "PKV_ERR_CUDA";
  }
  return "PKV_UNKNOWN_STATUS";
}

const char *pkv_last_error(void) { return g_last_error; }

pkv_status pkv_kv_store(const pkv_pool *pool, int32_t layer, const void *k, const void *v,
                        int64_t kv_row_stride, const int32_t *out_loc, int64_t num_tokens,
                        cudaStream_t stream) {
  pkv::PoolGeom g;
  pkv_status s = check_pool(pool, layer, &g);
  if (s != PKV_OK) return s;
  if (num_tokens < 0) return fail(PKV_ERR_INVALID_ARG, "num_tokens < 0");
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !out_loc) return fail(PKV_ERR_INVALID_ARG, "k, v and out_loc must be non-NULL");
  if (!aligned(k, 16) || !aligned(v, 16))
    return fail(PKV_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
  if (!aligned(out_loc, 4)) return fail(PKV_ERR_INVALID_ARG, "out_loc must be 4-byte aligned");
  if (kv_row_stride < static_cast<int64_t>(g.hkv) * g.d || kv_row_stride % 8 != 0)
    return fail(PKV_ERR_INVALID_ARG, "kv_row_stride %lld must be >= Hkv*D and a multiple of 8",
                static_cast<long long>(kv_row_stride));
  DevInfo *d = nullptr;
  if ((s = device_info(&d)) != PKV_OK) return s;
  cudaError_t e = pkv::launch_kv_store(g, layer, k, v, kv_row_stride, out_loc, num_tokens,
                                       d->sm_count, d->err, stream);
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "kv_store launch");
}

// Byte range of n rows of `width` elements, `stride` elements apart.
struct Span {
  uintptr_t lo, hi;
};
static Span rows_span(const void *p, int64_t n, int64_t stride, int64_t width) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + 2 * static_cast<uintptr_t>((n - 1) * stride + width)};
}
static bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

pkv_status pkv_norm_rope_kv_store(const pkv_pool *pool, int32_t layer, const void *q,
                                  int64_t q_row_stride, void *q_out, int32_t num_q_heads,
                                  const void *k, const void *v, int64_t kv_row_stride,
                                  const void *q_norm, const void *k_norm, float eps,
                                  const float *cos_sin, int64_t num_positions, int32_t rot_dim,
                                  int32_t interleaved, const int32_t *positions,
                                  const int32_t *out_loc, int64_t num_tokens,
                                  cudaStream_t stream) {
  pkv::PoolGeom g;
  pkv_status s = check_pool(pool, layer, &g);
  if (s != PKV_OK) return s;
  if (num_tokens < 0) return fail(PKV_ERR_INVALID_ARG, "num_tokens < 0");
  if (num_q_heads < 0) return fail(PKV_ERR_INVALID_ARG, "num_q_heads < 0");
  if (rot_dim < 0 || rot_dim > g.d || rot_dim % 16 != 0)
    return fail(PKV_ERR_INVALID_ARG, "rot_dim %d must be a multiple of 16 in [0, %d]", rot_dim, g.d);
  if (!isfinite(eps) || eps < 0.f) return fail(PKV_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (num_tokens == 0) return PKV_OK;
  if (num_tokens > 0x7fffffff)
    return fail(PKV_ERR_UNSUPPORTED, "num_tokens %lld past 2^31 - 1",
                static_cast<long long>(num_tokens));
  if (!k || !v || !out_loc) return fail(PKV_ERR_INVALID_ARG, "k, v and out_loc must be non-NULL");
  if (num_q_heads > 0 && (!q || !q_out))
    return fail(PKV_ERR_INVALID_ARG, "q and q_out must be non-NULL with q heads");
  if (rot_dim > 0 && (!cos_sin || !positions || num_positions <= 0))
    return fail(PKV_ERR_INVALID_ARG, "a rotation needs positions and a non-empty cos_sin table");
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q_norm, 16) || !aligned(k_norm, 16) ||
      (num_q_heads > 0 && (!aligned(q, 16) || !aligned(q_out, 16))) ||
      (rot_dim > 0 && !aligned(cos_sin, 16)))
    return fail(PKV_ERR_INVALID_ARG, "q, q_out, k, v, norms and cos_sin must be 16-byte aligned");
  if (!aligned(out_loc, 4) || (rot_dim > 0 && !aligned(positions, 4)))
    return fail(PKV_ERR_INVALID_ARG, "int32 tables must be 4-byte aligned");
  const int64_t kv_row = static_cast<int64_t>(g.hkv) * g.d;
  const int64_t q_row = static_cast<int64_t>(num_q_heads) * g.d;
  if (kv_row_stride < kv_row || kv_row_stride % 8 != 0)
    return fail(PKV_ERR_INVALID_ARG, "kv_row_stride %lld must be >= Hkv*D and a multiple of 8",
                static_cast<long long>(kv_row_stride));
  const Span sp{reinterpret_cast<uintptr_t>(g.base),
                reinterpret_cast<uintptr_t>(g.base) +
                    4 * static_cast<uintptr_t>(g.num_layers) * static_cast<uintptr_t>(g.plane)};
  const Span sk = rows_span(k, num_tokens, kv_row_stride, kv_row);
  const Span sv = rows_span(v, num_tokens, kv_row_stride, kv_row);
  if (overlap(sk, sp) || overlap(sv, sp))
    return fail(PKV_ERR_INVALID_ARG, "k and v may not overlap the pool");
  if (num_q_heads > 0) {
    if (q_row_stride < q_row || q_row_stride % 8 != 0)
      return fail(PKV_ERR_INVALID_ARG, "q_row_stride %lld must be >= Hq*D and a multiple of 8",
                  static_cast<long long>(q_row_stride));
    const Span sq = rows_span(q, num_tokens, q_row_stride, q_row);
    const Span so = rows_span(q_out, num_tokens, q_row, q_row);
    if (overlap(sq, sp) || overlap(so, sp))
      return fail(PKV_ERR_INVALID_ARG, "q and q_out may not overlap the pool");
    if (overlap(so, sk) || overlap(so, sv) ||
        (overlap(so, sq) && !(q_out == q && q_row_stride == q_row)))
      return fail(PKV_ERR_INVALID_ARG, "q_out may not overlap q, k or v (or be a contiguous q itself)");
  }
  DevInfo *d = nullptr;
  if ((s = device_info(&d)) != PKV_OK) return s;
  pkv::NormRopeArgs a{};
  a.pool = static_cast<__nv_bfloat16 *>(const_cast<void *>(g.base));
  a.plane = g.plane;
  a.slots = g.slots;
  a.num_layers = g.num_layers;
  a.layer = layer;
  a.hkv = g.hkv;
  a.hq = num_q_heads;
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.q_stride = q_row_stride;
  a.q_out = static_cast<__nv_bfloat16 *>(q_out);
  a.k = static_cast<const __nv_bfloat16 *>(k);
  a.v = static_cast<const __nv_bfloat16 *>(v);
  a.kv_stride = kv_row_stride;
  a.q_norm = num_q_heads > 0 ? static_cast<const __nv_bfloat16 *>(q_norm) : nullptr;
  a.k_norm = static_cast<const __nv_bfloat16 *>(k_norm);
  a.eps = eps;
  a.cos_sin = cos_sin;
  a.num_positions = num_positions;
  a.rot_dim = rot_dim;
  a.positions = positions;
  a.out_loc = out_loc;
  a.n = num_tokens;
  a.err = d->err;
  cudaError_t e = pkv::launch_norm_rope_store(g, a, interleaved != 0, d->sm_count, stream);
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "norm_rope_kv_store launch");
}

size_t pkv_decode_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                 int32_t head_dim, int32_t max_seq_len_hint) {
  if (batch <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      num_q_heads % num_kv_heads != 0)
    return 0;
  DevInfo *d = nullptr;
  if (device_info(&d) != PKV_OK) return 0;
  return pkv::plan_decode(batch, num_q_heads, num_kv_heads, head_dim,
                          effective_hint(max_seq_len_hint), d->sm_count)
      .workspace_bytes;
}

size_t pkv_decode_mod_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                     int32_t head_dim, int32_t max_keys_hint) {
  if (batch <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      num_q_heads % num_kv_heads != 0)
    return 0;
  DevInfo *d = nullptr;
  if (device_info(&d) != PKV_OK) return 0;
  // (a call whose rules change nothing runs as plain decode, with its plan)
  return pkv::decode_rules_workspace(batch, num_q_heads, num_kv_heads, head_dim,
                                     effective_hint(max_keys_hint), d->sm_count);
}

// The score rules of a call as the kernels take them; *used = false if they
// change nothing.
static pkv_status score_rules(const pkv_score_mod *mod, float scale, pkv::ScoreRules *out,
                              bool *used) {
  *used = false;
  if (!mod) return PKV_OK;
  if (!isfinite(mod->soft_cap) || mod->soft_cap < 0.f)
    return fail(PKV_ERR_INVALID_ARG, "soft_cap must be finite and >= 0");
  if (mod->window < 0) return fail(PKV_ERR_INVALID_ARG, "window must be >= 0");
  if (!aligned(mod->alibi_slopes, 4) || !aligned(mod->prefix_lens, 4))
    return fail(PKV_ERR_INVALID_ARG, "alibi_slopes and prefix_lens must be 4-byte aligned");
  *out = pkv::ScoreRules{};
  if (mod->soft_cap > 0.f) {
    out->cap_in = scale / mod->soft_cap;
    out->cap_log2 = mod->soft_cap * pkv::kLog2e;
    // the polynomial's coefficients hold powers of cap_in up to the fourth
    const double c = static_cast<double>(scale) / mod->soft_cap;
    if (!(fabs(c) <= 1e6) || !isfinite(out->cap_log2) || out->cap_log2 < 1e-30f)
      return fail(PKV_ERR_INVALID_ARG, "soft_cap %g out of range for scale %g",
                  static_cast<double>(mod->soft_cap), static_cast<double>(scale));
    const double c1 = static_cast<double>(out->cap_log2) * c;
    out->c1 = static_cast<float>(c1);
    out->c3 = static_cast<float>(c1 * c * c * pkv::kTanhNear3);
    out->c5 = static_cast<float>(c1 * c * c * c * c * pkv::kTanhNear5);
    // no score is near where the coefficients leave fp32 (scales of 1e14 and more)
    out->near =
        !isfinite(out->c1) || !isfinite(out->c3) || !isfinite(out->c5)
            ? -1.f
            : static_cast<float>(fmin(c == 0.0 ? 3e38 : pkv::kTanhNear / fabs(c),
                                      c1 == 0.0 ? 3e38 : pkv::kNearLog2 / fabs(c1)));
  }
  out->alibi_slopes = mod->alibi_slopes;
  // a window longer than any row is none (and the kernels' distances stay in 32 bits)
  out->window = mod->window >= 0x7fffff00 ? 0 : mod->window;
  out->prefix_lens = mod->prefix_lens;
  *used = mod->soft_cap > 0.f || mod->alibi_slopes || out->window > 0 || mod->prefix_lens;
  return PKV_OK;
}

// Decode, optionally with the step's new key / value rows stored first
// (k_new != NULL: the fused store of pkv_paged_decode_attn_store).
static pkv_status decode_call(const pkv_pool *pool, int32_t layer, const void *q,
                              const void *k_new, const void *v_new, int64_t kv_row_stride,
                              void *o, float *lse, const int32_t *page_table,
                              int64_t table_stride, const int32_t *table_idx,
                              const int32_t *seq_lens, int32_t batch, int32_t num_q_heads,
                              float scale, int32_t max_seq_len_hint, void *workspace,
                              size_t workspace_bytes, cudaStream_t stream,
                              const pkv_score_mod *mod = nullptr) {
  pkv::PoolGeom g;
  pkv_status s = check_pool(pool, layer, &g);
  if (s != PKV_OK) return s;
  if (batch < 0) return fail(PKV_ERR_INVALID_ARG, "batch < 0");
  if (num_q_heads <= 0 || num_q_heads % g.hkv != 0)
    return fail(PKV_ERR_INVALID_ARG, "num_q_heads %d is not a positive multiple of Hkv %d",
                num_q_heads, g.hkv);
  const int group = num_q_heads / g.hkv;
  if (group > 8) return fail(PKV_ERR_UNSUPPORTED, "decode supports Hq/Hkv <= 8, got %d", group);
  if (g.hkv < 4 ? (4 % g.hkv != 0) : (g.hkv % 4 != 0))
    return fail(PKV_ERR_UNSUPPORTED, "decode supports Hkv in {1, 2} or a multiple of 4, got %d",
                g.hkv);
  if (batch > 65535) return fail(PKV_ERR_UNSUPPORTED, "decode batch %d > 65535", batch);
  if (table_stride <= 0) return fail(PKV_ERR_INVALID_ARG, "table_stride must be positive");
  if (!isfinite(scale)) return fail(PKV_ERR_INVALID_ARG, "scale is not finite");
  pkv::ScoreRules rules;
  bool ruled = false;
  if ((s = score_rules(mod, scale, &rules, &ruled)) != PKV_OK) return s;
  if (batch == 0) return PKV_OK;
  if (!q || !o || !page_table || !seq_lens)
    return fail(PKV_ERR_INVALID_ARG, "q, o, page_table and seq_lens must be non-NULL");
  if (!aligned(q, 16) || !aligned(o, 16))
    return fail(PKV_ERR_INVALID_ARG, "q and o must be 16-byte aligned");
  if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4) ||
      !aligned(table_idx, 4))
    return fail(PKV_ERR_INVALID_ARG, "int32/fp32 tables must be 4-byte aligned");
  DevInfo *d = nullptr;
  if ((s = device_info(&d)) != PKV_OK) return s;
  const pkv::DecodePlan plan =
      ruled ? pkv::plan_decode_rules(batch, num_q_heads, g.hkv, g.d,
                                     effective_hint(max_seq_len_hint), d->sm_count)
            : pkv::plan_decode(batch, num_q_heads, g.hkv, g.d, effective_hint(max_seq_len_hint),
                               d->sm_count);
  if (plan.workspace_bytes > 0) {
    if (!workspace)
      return fail(PKV_ERR_WORKSPACE_TOO_SMALL, "workspace is NULL, %zu bytes needed",
                  plan.workspace_bytes);
    if (workspace_bytes < plan.workspace_bytes)
      return fail(PKV_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, %zu needed", workspace_bytes,
                  plan.workspace_bytes);
    if (!aligned(workspace, 256))
      return fail(PKV_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  }
  cudaError_t e = pkv::launch_decode(g, layer, q, o, lse, page_table, table_stride, table_idx,
                                     seq_lens, batch, num_q_heads, scale, plan, workspace, d->err,
                                     stream, k_new, v_new, kv_row_stride,
                                     ruled ? &rules : nullptr);
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "decode launch");
}

pkv_status pkv_paged_decode_attn(const pkv_pool *pool, int32_t layer, const void *q, void *o,
                                 float *lse, const int32_t *page_table, int64_t table_stride,
                                 const int32_t *table_idx, const int32_t *seq_lens,
                                 int32_t batch, int32_t num_q_heads, float scale,
                                 int32_t max_seq_len_hint, void *workspace,
                                 size_t workspace_bytes, cudaStream_t stream) {
  return decode_call(pool, layer, q, nullptr, nullptr, 0, o, lse, page_table, table_stride,
                     table_idx, seq_lens, batch, num_q_heads, scale, max_seq_len_hint, workspace,
                     workspace_bytes, stream);
}

pkv_status pkv_paged_decode_attn_mod(const pkv_pool *pool, int32_t layer, const void *q, void *o,
                                     float *lse, const int32_t *page_table, int64_t table_stride,
                                     const int32_t *table_idx, const int32_t *seq_lens,
                                     int32_t batch, int32_t num_q_heads, float scale,
                                     const pkv_score_mod *mod, int32_t max_keys_hint,
                                     void *workspace, size_t workspace_bytes,
                                     cudaStream_t stream) {
  return decode_call(pool, layer, q, nullptr, nullptr, 0, o, lse, page_table, table_stride,
                     table_idx, seq_lens, batch, num_q_heads, scale, max_keys_hint, workspace,
                     workspace_bytes, stream, mod);
}

pkv_status pkv_paged_decode_attn_store(const pkv_pool *pool, int32_t layer, const void *q,
                                       const void *k_new, const void *v_new,
                                       int64_t kv_row_stride, void *o, float *lse,
                                       const int32_t *page_table, int64_t table_stride,
                                       const int32_t *table_idx, const int32_t *seq_lens,
                                       int32_t batch, int32_t num_q_heads, float scale,
                                       int32_t max_seq_len_hint, void *workspace,
                                       size_t workspace_bytes, cudaStream_t stream) {
  if (batch > 0) {
    if (!k_new || !v_new) return fail(PKV_ERR_INVALID_ARG, "k_new and v_new must be non-NULL");
    if (!aligned(k_new, 16) || !aligned(v_new, 16))
      return fail(PKV_ERR_INVALID_ARG, "k_new and v_new must be 16-byte aligned");
    if (pool && (kv_row_stride < static_cast<int64_t>(pool->num_kv_heads) * pool->head_dim ||
                 kv_row_stride % 8 != 0))
      return fail(PKV_ERR_INVALID_ARG, "kv_row_stride %lld must be >= Hkv*D and a multiple of 8",
                  static_cast<long long>(kv_row_stride));
  }
  return decode_call(pool, layer, q, batch > 0 ? k_new : nullptr, v_new, kv_row_stride, o, lse,
                     page_table, table_stride, table_idx, seq_lens, batch, num_q_heads, scale,
                     max_seq_len_hint, workspace, workspace_bytes, stream);
}

static size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

size_t pkv_cascade_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                  int32_t head_dim, int32_t num_groups,
                                  int32_t max_prefix_len_hint, int32_t max_suffix_len_hint) {
  if (batch <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_groups <= 0 ||
      num_q_heads % num_kv_heads != 0 || max_prefix_len_hint < 1)
    return 0;
  DevInfo *d = nullptr;
  if (device_info(&d) != PKV_OK) return 0;
  const pkv::DecodePlan plan = pkv::plan_cascade_suffix(
      batch, num_q_heads, num_kv_heads, head_dim, effective_hint(max_suffix_len_hint), d->sm_count);
  const int32_t ks = pkv::cascade_prefix_splits(batch, num_q_heads, num_kv_heads, num_groups,
                                                max_prefix_len_hint, max_suffix_len_hint,
                                                d->sm_count);
  return align256(pkv::cascade_partial_bytes(batch, num_q_heads, head_dim, plan.splits + ks));
}

pkv_status pkv_paged_cascade_decode_attn(
    const pkv_pool *pool, int32_t layer, const void *q, void *o, float *lse,
    const int32_t *prefix_page_table, int64_t prefix_table_stride, const int32_t *prefix_lens,
    const int32_t *member_indptr, const int32_t *members, int32_t num_groups,
    const int32_t *page_table, int64_t table_stride, const int32_t *table_idx,
    const int32_t *seq_lens, int32_t batch, int32_t num_q_heads, float scale,
    int32_t max_prefix_len_hint, int32_t max_suffix_len_hint, void *workspace,
    size_t workspace_bytes, cudaStream_t stream) {
  pkv::PoolGeom g;
  pkv_status s = check_pool(pool, layer, &g);
  if (s != PKV_OK) return s;
  if (batch < 0 || num_groups < 0) return fail(PKV_ERR_INVALID_ARG, "batch and num_groups must be >= 0");
  if (num_q_heads <= 0 || num_q_heads % g.hkv != 0)
    return fail(PKV_ERR_INVALID_ARG, "num_q_heads %d is not a positive multiple of Hkv %d",
                num_q_heads, g.hkv);
  const int group = num_q_heads / g.hkv;
  if (group > 8) return fail(PKV_ERR_UNSUPPORTED, "cascade decode supports Hq/Hkv <= 8, got %d", group);
  if (g.hkv < 4 ? (4 % g.hkv != 0) : (g.hkv % 4 != 0))
    return fail(PKV_ERR_UNSUPPORTED, "decode supports Hkv in {1, 2} or a multiple of 4, got %d",
                g.hkv);
  if (batch > 65535 || num_groups >= 65535)
    return fail(PKV_ERR_UNSUPPORTED, "cascade decode: batch %d or groups %d too large", batch,
                num_groups);
  if (table_stride <= 0 || prefix_table_stride <= 0)
    return fail(PKV_ERR_INVALID_ARG, "table strides must be positive");
  if (!isfinite(scale)) return fail(PKV_ERR_INVALID_ARG, "scale is not finite");
  if (batch == 0) return PKV_OK;
  if (num_groups == 0)
    return fail(PKV_ERR_INVALID_ARG, "cascade decode needs every request in a group (num_groups 0)");
  if (!q || !o || !page_table || !seq_lens || !prefix_page_table || !prefix_lens ||
      !member_indptr || !members)
    return fail(PKV_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned(q, 16) || !aligned(o, 16))
    return fail(PKV_ERR_INVALID_ARG, "q and o must be 16-byte aligned");
  if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4) ||
      !aligned(table_idx, 4) || !aligned(prefix_page_table, 4) || !aligned(prefix_lens, 4) ||
      !aligned(member_indptr, 4) || !aligned(members, 4))
    return fail(PKV_ERR_INVALID_ARG, "int32/fp32 tables must be 4-byte aligned");
  const int64_t prefix_row_capacity = prefix_table_stride * g.page_size;
  int64_t pcap = max_prefix_len_hint >= 1 ? max_prefix_len_hint : prefix_row_capacity;
  if (pcap > prefix_row_capacity) pcap = prefix_row_capacity;
  if (pcap > (int64_t(1) << 30)) pcap = int64_t(1) << 30;
  if (static_cast<int64_t>(pkv::cascade_prefix_blocks(batch, num_q_heads, g.hkv, num_groups)) >
      65535)
    return fail(PKV_ERR_UNSUPPORTED, "cascade: too many member blocks in one call");
  DevInfo *d = nullptr;
  if ((s = device_info(&d)) != PKV_OK) return s;
  const pkv::DecodePlan plan = pkv::plan_cascade_suffix(
      batch, num_q_heads, g.hkv, g.d, effective_hint(max_suffix_len_hint), d->sm_count);
  const int32_t ks = pkv::cascade_prefix_splits(batch, num_q_heads, g.hkv, num_groups,
                                                static_cast<int32_t>(pcap), max_suffix_len_hint,
                                                d->sm_count);
  const int32_t slots = plan.splits + ks;
  const size_t need = align256(pkv::cascade_partial_bytes(batch, num_q_heads, g.d, slots));
  if (!workspace)
    return fail(PKV_ERR_WORKSPACE_TOO_SMALL, "workspace is NULL, %zu bytes needed", need);
  if (workspace_bytes < need)
    return fail(PKV_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, %zu needed", workspace_bytes,
                need);
  if (!aligned(workspace, 256)) return fail(PKV_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  float *part_o = nullptr, *part_lse = nullptr;
  pkv::cascade_partial_ptrs(workspace, batch, num_q_heads, g.d, slots, &part_o, &part_lse);
  // All on `stream`, in this order:
  // 1. the shared-prefix states of every member (slots splits .. splits +
  //    ks - 1): each group's prefix once per kv head and key range, K/V read
  //    from the pool by the tensor-core prefix kernel;
  cudaError_t e = pkv::launch_cascade_prefix(
      g, layer, q, prefix_page_table, prefix_table_stride, prefix_lens, member_indptr, members,
      num_groups, batch, num_q_heads, scale, part_o, part_lse, slots, plan.splits, ks, d->err,
      stream);
  if (e != cudaSuccess) return cuda_fail(e, "cascade prefix launch");
  // 2. the suffix partial states (slots 0 .. splits - 1): split-KV decode,
  //    started as soon as every prefix CTA is running (it reads nothing the
  //    prefix kernel writes; its last request's split-0 CTAs wait for that
  //    kernel at their exit, so this grid completes after it);
  float *po = nullptr, *pl = nullptr;
  e = pkv::launch_cascade_suffix(g, layer, q, o, lse, page_table, table_stride, table_idx,
                                 seq_lens, batch, num_q_heads, scale, plan, ks, workspace, d->err,
                                 stream, &po, &pl);
  if (e != cudaSuccess) return cuda_fail(e, "cascade suffix launch");
  // 3. the merge of every request's suffix splits and prefix states.
  e = pkv::launch_cascade_merge(g, layer, q, o, lse, page_table, table_stride, table_idx,
                                seq_lens, batch, num_q_heads, scale, plan, ks, part_o, part_lse,
                                d->err, stream);
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "cascade merge launch");
}

size_t pkv_extend_workspace_size(int32_t batch, int32_t num_kv_heads, int32_t head_dim,
                                 int32_t max_seq_len_hint, int64_t max_total_keys_hint) {
  if (batch <= 0 || num_kv_heads <= 0 || head_dim <= 0 || max_seq_len_hint < 1) return 0;
  return pkv::extend_layout(batch, num_kv_heads, head_dim, max_seq_len_hint, max_total_keys_hint)
      .total_bytes;
}

size_t pkv_extend_mod_workspace_size(int32_t batch, int32_t total_q, int32_t num_q_heads,
                                     int32_t num_kv_heads, int32_t head_dim,
                                     int32_t max_seq_len_hint, int64_t max_total_keys_hint) {
  const size_t gathered = pkv_extend_workspace_size(batch, num_kv_heads, head_dim,
                                                    max_seq_len_hint, max_total_keys_hint);
  if (gathered == 0 || total_q <= 0 || num_q_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
      num_q_heads / num_kv_heads > 16)
    return 0;
  DevInfo *d = nullptr;
  if (device_info(&d) != PKV_OK) return 0;
  // either form may be the faster one for a smaller call
  const size_t direct = pkv::extend_direct_workspace(
      batch, total_q, num_q_heads, num_kv_heads, head_dim, max_seq_len_hint, d->sm_count);
  return direct > gathered ? direct : gathered;
}

static pkv_status check_workspace(const void *workspace, size_t workspace_bytes, size_t need) {
  if (need == 0) return PKV_OK;
  if (!workspace)
    return fail(PKV_ERR_WORKSPACE_TOO_SMALL, "workspace is NULL, %zu bytes needed", need);
  if (workspace_bytes < need)
    return fail(PKV_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, %zu needed", workspace_bytes,
                need);
  if (!aligned(workspace, 256))
    return fail(PKV_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return PKV_OK;
}

// Extend with (k_new != NULL) or without the fused store of the chunk's K/V.
static pkv_status extend_call(const pkv_pool *pool, int32_t layer, const void *q,
                              const void *k_new, const void *v_new, int64_t kv_row_stride,
                              const int32_t *qo_indptr, void *o, float *lse,
                              const int32_t *page_table, int64_t table_stride,
                              const int32_t *table_idx, const int32_t *seq_lens, int32_t batch,
                              int32_t total_q, int32_t num_q_heads, float scale,
                              int32_t max_seq_len_hint, int64_t max_total_keys_hint,
                              void *workspace, size_t workspace_bytes, cudaStream_t stream,
                              const pkv_score_mod *mod = nullptr) {
  pkv::PoolGeom g;
  pkv_status s = check_pool(pool, layer, &g);
  if (s != PKV_OK) return s;
  if (batch < 0 || total_q < 0) return fail(PKV_ERR_INVALID_ARG, "batch and total_q must be >= 0");
  if (num_q_heads <= 0 || num_q_heads % g.hkv != 0)
    return fail(PKV_ERR_INVALID_ARG, "num_q_heads %d is not a positive multiple of Hkv %d",
                num_q_heads, g.hkv);
  const int group = num_q_heads / g.hkv;
  if (group > 16) return fail(PKV_ERR_UNSUPPORTED, "extend supports Hq/Hkv <= 16, got %d", group);
  if (batch >= 65535) return fail(PKV_ERR_UNSUPPORTED, "extend supports batch < 65535");
  if (g.hkv > 65535) return fail(PKV_ERR_UNSUPPORTED, "too many kv heads");
  if (table_stride <= 0) return fail(PKV_ERR_INVALID_ARG, "table_stride must be positive");
  if (!isfinite(scale)) return fail(PKV_ERR_INVALID_ARG, "scale is not finite");
  // the scale's sign is folded into Q, a zero scale zeroes it: the cap's
  // factor is positive like the kernel's own
  pkv::ScoreRules rules;
  bool ruled = false;
  if ((s = score_rules(mod, scale == 0.f ? 1.f : fabsf(scale), &rules, &ruled)) != PKV_OK)
    return s;
  if (batch == 0 || total_q == 0) return PKV_OK;
  if (!q || !o || !qo_indptr || !page_table || !seq_lens)
    return fail(PKV_ERR_INVALID_ARG, "q, o, qo_indptr, page_table and seq_lens must be non-NULL");
  if (!aligned(q, 16) || !aligned(o, 16))
    return fail(PKV_ERR_INVALID_ARG, "q and o must be 16-byte aligned");
  if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4) ||
      !aligned(table_idx, 4) || !aligned(qo_indptr, 4))
    return fail(PKV_ERR_INVALID_ARG, "int32/fp32 tables must be 4-byte aligned");
  const int64_t row_capacity = table_stride * g.page_size;
  int64_t cap = max_seq_len_hint >= 1 ? max_seq_len_hint : row_capacity;
  if (cap > row_capacity) cap = row_capacity;
  if (cap > (int64_t(1) << 30)) return fail(PKV_ERR_UNSUPPORTED, "sequence capacity too large");
  if (max_total_keys_hint > (int64_t(1) << 40))
    return fail(PKV_ERR_UNSUPPORTED, "max_total_keys_hint too large");
  if (ruled) {
    // few query blocks: straight from the pool, the work shared out by key tiles
    DevInfo *d = nullptr;
    if ((s = device_info(&d)) != PKV_OK) return s;
    pkv::DirectPlan plan;
    if (pkv::extend_direct_plan(batch, total_q, num_q_heads, g.hkv, g.d,
                                static_cast<int32_t>(cap), max_total_keys_hint,
                                rules.prefix_lens ? 0 : rules.window, d->sm_count, &plan)) {
      if (!plan.whole &&
          (s = check_workspace(workspace, workspace_bytes, plan.workspace_bytes)) != PKV_OK)
        return s;
      const cudaError_t e = pkv::launch_extend_direct(
          g, layer, q, qo_indptr, o, lse, page_table, table_stride, table_idx, seq_lens, batch,
          total_q, num_q_heads, scale, rules, plan, workspace, d->err, stream);
      return e == cudaSuccess ? PKV_OK : cuda_fail(e, "extend launch");
    }
  }
  const pkv::ExtendLayout lay = pkv::extend_layout(batch, g.hkv, g.d, cap, max_total_keys_hint);
  if (2 * g.hkv * lay.cap_rows >= (int64_t(1) << 31) || lay.max_blocks >= (int64_t(1) << 28))
    return fail(PKV_ERR_UNSUPPORTED, "extend: kv heads x key bound too large (%lld rows)",
                static_cast<long long>(2 * g.hkv * lay.cap_rows));
  const size_t need = lay.total_bytes;
  if (!workspace)
    return fail(PKV_ERR_WORKSPACE_TOO_SMALL, "workspace is NULL, %zu bytes needed", need);
  if (workspace_bytes < need)
    return fail(PKV_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, %zu needed", workspace_bytes,
                need);
  if (!aligned(workspace, 256)) return fail(PKV_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  const int64_t tpc = 2 * (128 / group);  // chunk tokens per CTA (two 128-row query tiles)
  if ((static_cast<int64_t>(total_q) + tpc - 1) / tpc + batch > 65535)
    return fail(PKV_ERR_UNSUPPORTED, "extend: too many query tiles in one call");
  DevInfo *d = nullptr;
  if ((s = device_info(&d)) != PKV_OK) return s;
  pkv::ExtendMode mode;
  mode.k_new = k_new;
  mode.v_new = v_new;
  mode.kv_row_stride = kv_row_stride;
  mode.rules = ruled ? &rules : nullptr;
  cudaError_t e = pkv::launch_extend(g, layer, q, qo_indptr, o, lse, page_table, table_stride,
                                     table_idx, seq_lens, batch, total_q, num_q_heads, scale, lay,
                                     workspace, d->sm_count, d->err, stream, mode);
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "extend launch");
}

pkv_status pkv_paged_extend_attn(const pkv_pool *pool, int32_t layer, const void *q,
                                 const int32_t *qo_indptr, void *o, float *lse,
                                 const int32_t *page_table, int64_t table_stride,
                                 const int32_t *table_idx, const int32_t *seq_lens,
                                 int32_t batch, int32_t total_q, int32_t num_q_heads,
                                 float scale, int32_t max_seq_len_hint,
                                 int64_t max_total_keys_hint, void *workspace,
                                 size_t workspace_bytes, cudaStream_t stream) {
  return extend_call(pool, layer, q, nullptr, nullptr, 0, qo_indptr, o, lse, page_table,
                     table_stride, table_idx, seq_lens, batch, total_q, num_q_heads, scale,
                     max_seq_len_hint, max_total_keys_hint, workspace, workspace_bytes, stream);
}

pkv_status pkv_paged_extend_attn_mod(const pkv_pool *pool, int32_t layer, const void *q,
                                     const int32_t *qo_indptr, void *o, float *lse,
                                     const int32_t *page_table, int64_t table_stride,
                                     const int32_t *table_idx, const int32_t *seq_lens,
                                     int32_t batch, int32_t total_q, int32_t num_q_heads,
                                     float scale, const pkv_score_mod *mod,
                                     int32_t max_seq_len_hint, int64_t max_total_keys_hint,
                                     void *workspace, size_t workspace_bytes,
                                     cudaStream_t stream) {
  return extend_call(pool, layer, q, nullptr, nullptr, 0, qo_indptr, o, lse, page_table,
                     table_stride, table_idx, seq_lens, batch, total_q, num_q_heads, scale,
                     max_seq_len_hint, max_total_keys_hint, workspace, workspace_bytes, stream,
                     mod);
}

pkv_status pkv_paged_extend_attn_store(const pkv_pool *pool, int32_t layer, const void *q,
                                       const void *k_new, const void *v_new,
                                       int64_t kv_row_stride, const int32_t *qo_indptr, void *o,
                                       float *lse, const int32_t *page_table,
                                       int64_t table_stride, const int32_t *table_idx,
                                       const int32_t *seq_lens, int32_t batch, int32_t total_q,
                                       int32_t num_q_heads, float scale,
                                       int32_t max_seq_len_hint, int64_t max_total_keys_hint,
                                       void *workspace, size_t workspace_bytes,
                                       cudaStream_t stream) {
  if (batch > 0 && total_q > 0) {
    if (!k_new || !v_new) return fail(PKV_ERR_INVALID_ARG, "k_new and v_new must be non-NULL");
    if (!aligned(k_new, 16) || !aligned(v_new, 16))
      return fail(PKV_ERR_INVALID_ARG, "k_new and v_new must be 16-byte aligned");
    if (pool && (kv_row_stride < static_cast<int64_t>(pool->num_kv_heads) * pool->head_dim ||
                 kv_row_stride % 8 != 0))
      return fail(PKV_ERR_INVALID_ARG, "kv_row_stride %lld must be >= Hkv*D and a multiple of 8",
                  static_cast<long long>(kv_row_stride));
  }
  return extend_call(pool, layer, q, batch > 0 && total_q > 0 ? k_new : nullptr, v_new,
                     kv_row_stride, qo_indptr, o, lse, page_table, table_stride, table_idx,
                     seq_lens, batch, total_q, num_q_heads, scale, max_seq_len_hint,
                     max_total_keys_hint, workspace, workspace_bytes, stream);
}

size_t pkv_tree_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                               int32_t head_dim, int32_t max_tree_tokens,
                               int32_t max_seq_len_hint) {
  if (batch <= 0 || batch > 65535 || num_kv_heads <= 0 || num_q_heads <= 0 ||
      num_q_heads % num_kv_heads != 0 || num_q_heads / num_kv_heads > 16 ||
      (head_dim != 64 && head_dim != 128) || max_tree_tokens < 1 ||
      max_tree_tokens > PKV_MAX_TREE_TOKENS || max_seq_len_hint < 1)
    return 0;
  DevInfo *d = nullptr;
  if (device_info(&d) != PKV_OK) return 0;
  return pkv::tree_plan(batch, num_q_heads, num_kv_heads, head_dim, max_tree_tokens,
                        max_seq_len_hint, d->sm_count)
      .workspace_bytes;
}

pkv_status pkv_paged_tree_attn(const pkv_pool *pool, int32_t layer, const void *q,
                               const int32_t *qo_indptr, const int32_t *parents, void *o,
                               float *lse, const int32_t *page_table, int64_t table_stride,
                               const int32_t *table_idx, const int32_t *seq_lens, int32_t batch,
                               int32_t total_q, int32_t num_q_heads, float scale,
                               int32_t max_tree_tokens, int32_t max_seq_len_hint, void *workspace,
                               size_t workspace_bytes, cudaStream_t stream) {
  pkv::PoolGeom g;
  pkv_status s = check_pool(pool, layer, &g);
  if (s != PKV_OK) return s;
  if (batch < 0 || total_q < 0) return fail(PKV_ERR_INVALID_ARG, "batch and total_q must be >= 0");
  if (num_q_heads <= 0 || num_q_heads % g.hkv != 0)
    return fail(PKV_ERR_INVALID_ARG, "num_q_heads %d is not a positive multiple of Hkv %d",
                num_q_heads, g.hkv);
  if (num_q_heads / g.hkv > 16)
    return fail(PKV_ERR_UNSUPPORTED, "tree attention supports Hq/Hkv <= 16, got %d",
                num_q_heads / g.hkv);
  if (max_tree_tokens < 1) return fail(PKV_ERR_INVALID_ARG, "max_tree_tokens must be >= 1");
  if (max_tree_tokens > PKV_MAX_TREE_TOKENS)
    return fail(PKV_ERR_UNSUPPORTED, "max_tree_tokens %d > %d", max_tree_tokens,
                PKV_MAX_TREE_TOKENS);
  if (batch > 65535) return fail(PKV_ERR_UNSUPPORTED, "tree attention batch %d > 65535", batch);
  if (g.hkv > 65535) return fail(PKV_ERR_UNSUPPORTED, "too many kv heads");
  if (table_stride <= 0) return fail(PKV_ERR_INVALID_ARG, "table_stride must be positive");
  if (!isfinite(scale)) return fail(PKV_ERR_INVALID_ARG, "scale is not finite");
  if (batch == 0 || total_q == 0) return PKV_OK;
  if (!q || !o || !qo_indptr || !parents || !page_table || !seq_lens)
    return fail(PKV_ERR_INVALID_ARG,
                "q, o, qo_indptr, parents, page_table and seq_lens must be non-NULL");
  if (!aligned(q, 16) || !aligned(o, 16))
    return fail(PKV_ERR_INVALID_ARG, "q and o must be 16-byte aligned");
  if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4) ||
      !aligned(table_idx, 4) || !aligned(qo_indptr, 4) || !aligned(parents, 4))
    return fail(PKV_ERR_INVALID_ARG, "int32/fp32 tables must be 4-byte aligned");
  const int64_t row_capacity = table_stride * g.page_size;
  if (row_capacity > 0x7fffff00)
    return fail(PKV_ERR_UNSUPPORTED, "page-table rows of %lld keys (at most 2^31 - 256)",
                static_cast<long long>(row_capacity));
  int64_t cap = max_seq_len_hint >= 1 ? max_seq_len_hint : row_capacity;
  if (cap > row_capacity) cap = row_capacity;
  DevInfo *d = nullptr;
  if ((s = device_info(&d)) != PKV_OK) return s;
  const pkv::DirectPlan plan =
      pkv::tree_plan(batch, num_q_heads, g.hkv, g.d, max_tree_tokens, static_cast<int32_t>(cap),
                     d->sm_count);
  if (!plan.whole &&
      (s = check_workspace(workspace, workspace_bytes, plan.workspace_bytes)) != PKV_OK)
    return s;
  cudaError_t e = pkv::launch_tree(g, layer, q, qo_indptr, parents, o, lse, page_table,
                                   table_stride, table_idx, seq_lens, batch, total_q, num_q_heads,
                                   scale, max_tree_tokens, plan, workspace, d->err, stream);
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "tree launch");
}

pkv_status pkv_merge_lse(const float *o_a, const float *lse_a, const float *o_b,
                         const float *lse_b, void *o_out, int32_t o_out_is_bf16,
                         float *lse_out, int64_t rows, int32_t heads, int32_t head_dim,
                         cudaStream_t stream) {
  if (rows < 0 || heads <= 0 || head_dim <= 0 || head_dim % 4 != 0)
    return fail(PKV_ERR_INVALID_ARG, "rows >= 0, heads > 0 and head_dim a positive multiple of 4");
  if (rows == 0) return PKV_OK;
  if (!o_a || !lse_a || !o_b || !lse_b || !o_out)
    return fail(PKV_ERR_INVALID_ARG, "o_a, lse_a, o_b, lse_b and o_out must be non-NULL");
  if (!aligned(o_a, 16) || !aligned(o_b, 16) || !aligned(o_out, 16))
    return fail(PKV_ERR_INVALID_ARG, "o pointers must be 16-byte aligned");
  if (!aligned(lse_a, 4) || !aligned(lse_b, 4) || !aligned(lse_out, 4))
    return fail(PKV_ERR_INVALID_ARG, "lse pointers must be 4-byte aligned");
  DevInfo *d = nullptr;
  pkv_status s = device_info(&d);
  if (s != PKV_OK) return s;
  cudaError_t e = pkv::launch_merge(o_a, lse_a, o_b, lse_b, o_out, o_out_is_bf16 != 0, lse_out,
                                    rows, heads, head_dim, d->sm_count, stream);
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "merge launch");
}

pkv_status pkv_read_device_errors(uint32_t *flags) {
  if (!flags) return fail(PKV_ERR_INVALID_ARG, "flags is NULL");
  DevInfo *d = nullptr;
  pkv_status s = device_info(&d);
  if (s != PKV_OK) return s;
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceSynchronize");
  unsigned v = 0;
  if ((e = cudaMemcpyFromSymbol(&v, g_device_errors, sizeof v)) != cudaSuccess)
    return cuda_fail(e, "read device error word");
  const unsigned zero = 0;
  if ((e = cudaMemcpyToSymbol(g_device_errors, &zero, sizeof zero)) != cudaSuccess)
    return cuda_fail(e, "clear device error word");
  *flags = v;
  return PKV_OK;
}

}  // extern "C"
