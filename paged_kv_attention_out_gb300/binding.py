"""Thin ctypes binding of the pkv C ABI (include/pkv.h), same names.

Argument marshalling only: every function takes torch tensors that already
live on the current CUDA device, checks their dtypes and shapes, and passes
raw pointers, sizes and the current stream to the C entry point of the same
name. All arithmetic runs in the library's CUDA kernels. If the library is
not built, importing this module's functions raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

_c_int32 = ctypes.c_int32
_c_int64 = ctypes.c_int64
_p = ctypes.c_void_p


class PkvPool(ctypes.Structure):
    _fields_ = [("base", _p), ("num_layers", _c_int32), ("num_pages", _c_int64),
                ("page_size", _c_int32), ("num_kv_heads", _c_int32), ("head_dim", _c_int32)]


class PkvScoreMod(ctypes.Structure):
    _fields_ = [("soft_cap", ctypes.c_float), ("alibi_slopes", _p), ("window", _c_int32),
                ("prefix_lens", _p)]


PKV_OK = 0
STATUS_NAMES = {0: "PKV_OK", 1: "PKV_ERR_INVALID_ARG", 2: "PKV_ERR_UNSUPPORTED",
                3: "PKV_ERR_WORKSPACE_TOO_SMALL", 4: "PKV_ERR_CUDA"}


class PkvError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


_lib = None


def library_path() -> str:
    return _build.LIB


def load() -> ctypes.CDLL:
    """Load libpkv.so (built by __graft_entry__.build()); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"pkv CUDA library not built ({path}); run "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(path)
    pool_p = ctypes.POINTER(PkvPool)
    L.pkv_init.restype = ctypes.c_int
    L.pkv_status_string.restype = ctypes.c_char_p
    L.pkv_status_string.argtypes = [ctypes.c_int]
    L.pkv_last_error.restype = ctypes.c_char_p
    L.pkv_kv_store.restype = ctypes.c_int
    L.pkv_kv_store.argtypes = [pool_p, _c_int32, _p, _p, _c_int64, _p, _c_int64, _p]
    L.pkv_norm_rope_kv_store.restype = ctypes.c_int
    L.pkv_norm_rope_kv_store.argtypes = [pool_p, _c_int32, _p, _c_int64, _p, _c_int32, _p, _p,
                                         _c_int64, _p, _p, ctypes.c_float, _p, _c_int64,
                                         _c_int32, _c_int32, _p, _p, _c_int64, _p]
    L.pkv_decode_workspace_size.restype = ctypes.c_size_t
    L.pkv_decode_workspace_size.argtypes = [_c_int32] * 5
    L.pkv_paged_decode_attn.restype = ctypes.c_int
    L.pkv_paged_decode_attn.argtypes = [pool_p, _c_int32, _p, _p, _p, _p, _c_int64, _p, _p,
                                        _c_int32, _c_int32, ctypes.c_float, _c_int32, _p,
                                        ctypes.c_size_t, _p]
    L.pkv_paged_decode_attn_store.restype = ctypes.c_int
    L.pkv_paged_decode_attn_store.argtypes = [pool_p, _c_int32, _p, _p, _p, _c_int64, _p, _p, _p,
                                              _c_int64, _p, _p, _c_int32, _c_int32,
                                              ctypes.c_float, _c_int32, _p, ctypes.c_size_t, _p]
    L.pkv_paged_decode_attn_noalloc.restype = ctypes.c_int
    L.pkv_paged_decode_attn_noalloc.argtypes = [pool_p, _c_int32, _p, _p, _p, _p, _c_int64, _p,
                                                _p, _c_int32, _c_int32, ctypes.c_float,
                                                _c_int32, _p]
    mod_p = ctypes.POINTER(PkvScoreMod)
    L.pkv_decode_mod_workspace_size.restype = ctypes.c_size_t
    L.pkv_decode_mod_workspace_size.argtypes = [_c_int32] * 5
    L.pkv_paged_decode_attn_mod.restype = ctypes.c_int
    L.pkv_paged_decode_attn_mod.argtypes = [pool_p, _c_int32, _p, _p, _p, _p, _c_int64, _p, _p,
                                            _c_int32, _c_int32, ctypes.c_float, mod_p, _c_int32,
                                            _p, ctypes.c_size_t, _p]
    L.pkv_extend_mod_workspace_size.restype = ctypes.c_size_t
    L.pkv_extend_mod_workspace_size.argtypes = [_c_int32] * 6 + [_c_int64]
    L.pkv_paged_extend_attn_mod.restype = ctypes.c_int
    L.pkv_paged_extend_attn_mod.argtypes = [pool_p, _c_int32, _p, _p, _p, _p, _p, _c_int64, _p,
                                            _p, _c_int32, _c_int32, _c_int32, ctypes.c_float,
                                            mod_p, _c_int32, _c_int64, _p, ctypes.c_size_t, _p]
    L.pkv_extend_workspace_size.restype = ctypes.c_size_t
    L.pkv_extend_workspace_size.argtypes = [_c_int32] * 4 + [_c_int64]
    L.pkv_paged_extend_attn.restype = ctypes.c_int
    L.pkv_paged_extend_attn.argtypes = [pool_p, _c_int32, _p, _p, _p, _p, _p, _c_int64, _p, _p,
                                        _c_int32, _c_int32, _c_int32, ctypes.c_float,
                                        _c_int32, _c_int64, _p, ctypes.c_size_t, _p]
    L.pkv_paged_extend_attn_store.restype = ctypes.c_int
    L.pkv_paged_extend_attn_store.argtypes = [pool_p, _c_int32, _p, _p, _p, _c_int64, _p, _p, _p,
                                              _p, _c_int64, _p, _p, _c_int32, _c_int32,
                                              _c_int32, ctypes.c_float, _c_int32, _c_int64, _p,
                                              ctypes.c_size_t, _p]
    L.pkv_tree_workspace_size.restype = ctypes.c_size_t
    L.pkv_tree_workspace_size.argtypes = [_c_int32] * 6
    L.pkv_paged_tree_attn.restype = ctypes.c_int
    L.pkv_paged_tree_attn.argtypes = [pool_p, _c_int32, _p, _p, _p, _p, _p, _p, _c_int64, _p, _p,
                                      _c_int32, _c_int32, _c_int32, ctypes.c_float, _c_int32,
                                      _c_int32, _p, ctypes.c_size_t, _p]
    L.pkv_decode_mass_workspace_size.restype = ctypes.c_size_t
    L.pkv_decode_mass_workspace_size.argtypes = [_c_int32] * 5
    L.pkv_paged_decode_attn_mass.restype = ctypes.c_int
    L.pkv_paged_decode_attn_mass.argtypes = [pool_p, _c_int32, _p, _p, _p, _p, _c_int64, _p,
                                             _c_int64, _p, _p, _c_int32, _c_int32, ctypes.c_float,
                                             ctypes.c_float, _c_int32, _p, ctypes.c_size_t, _p]
    L.pkv_paged_extend_mass.restype = ctypes.c_int
    L.pkv_paged_extend_mass.argtypes = [pool_p, _c_int32, _p, _p, _p, _p, _c_int64, _p, _c_int64,
                                        _p, _p, _c_int32, _c_int32, _c_int32, ctypes.c_float,
                                        ctypes.c_float, _c_int32, _c_int32, _c_int32, _c_int64, _p]
    L.pkv_kv_evict.restype = ctypes.c_int
    L.pkv_kv_evict.argtypes = [pool_p, _c_int32, _p, _c_int64, _p, _c_int64, _p, _p, _c_int32,
                               _c_int32, _c_int32, _c_int32, _p, _c_int32, _p]
    L.pkv_kv_rerope.restype = ctypes.c_int
    L.pkv_kv_rerope.argtypes = [pool_p, _c_int32, _p, _c_int64, _p, _p, _c_int32, _p, _p, _c_int32,
                                _c_int64, _p, _p, _c_int32, _c_int32, ctypes.c_float, _c_int32,
                                _c_int64, _p]
    L.pkv_cascade_workspace_size.restype = ctypes.c_size_t
    L.pkv_cascade_workspace_size.argtypes = [_c_int32] * 7
    L.pkv_paged_cascade_decode_attn.restype = ctypes.c_int
    L.pkv_paged_cascade_decode_attn.argtypes = [pool_p, _c_int32, _p, _p, _p, _p, _c_int64, _p, _p,
                                                _p, _c_int32, _p, _c_int64, _p, _p, _c_int32,
                                                _c_int32, ctypes.c_float, _c_int32, _c_int32, _p,
                                                ctypes.c_size_t, _p]
    L.pkv_merge_lse.restype = ctypes.c_int
    L.pkv_merge_lse.argtypes = [_p, _p, _p, _p, _p, _c_int32, _p, _c_int64, _c_int32,
                                _c_int32, _p]
    L.pkv_read_device_errors.restype = ctypes.c_int
    L.pkv_read_device_errors.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    _lib = L
    return L


def _check(status: int) -> None:
    if status != PKV_OK:
        msg = load().pkv_last_error().decode(errors="replace")
        raise PkvError(status, msg)


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:  # the handle alone: building a Stream object costs 3 us a call
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _want(t: torch.Tensor, dtype, name: str, ndim: int | None = None):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def _contig(t: torch.Tensor, name: str):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# The calls below are launch-bound at decode sizes, so each tensor is checked by
# one short expression; what is wrong is found out only when something is.
_bf16, _f32, _i32 = torch.bfloat16, torch.float32, torch.int32
# torch.cuda.current_device without its lazy set-up (None in a torch without CUDA)
_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _handle(stream, dev: int) -> int:
    return _raw_stream(dev) if stream is None else stream.cuda_stream


def _refuse(t, dtype, ndim: int, dev: int, name: str):
    _want(t, dtype, name, ndim)
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    _contig(t, name)


def _arg(t, dtype, ndim: int, dev: int, name: str) -> int:
    """Address of a contiguous tensor of this type on the current device `dev`."""
    if t.dtype is not dtype or t.get_device() != dev or t.dim() != ndim \
            or not t.is_contiguous():
        _refuse(t, dtype, ndim, dev, name)
    return t.data_ptr()


def _rows_arg(t, shape, dev: int, name: str) -> tuple[int, int]:
    """(address, elements between rows) of a bf16 [N, heads, D] tensor with contiguous rows."""
    if t.dtype is not _bf16 or t.get_device() != dev or t.shape != shape:
        _want(t, _bf16, name, 3)
        if t.shape != shape:
            raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
        _refuse(t, _bf16, 3, dev, name)
    n, h, d = shape
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != d and h != 1):
        raise ValueError(f"{name} must have its heads and dims contiguous")
    return t.data_ptr(), s0 if n != 1 else h * d


def _pool_arg(pool, dev: int) -> PkvPool:
    base = _arg(pool, _bf16, 6, dev, "pool")
    two, L, NP, P, H, D = pool.shape
    if two != 2:
        raise ValueError("pool dim 0 must be 2 (K, V)")
    return PkvPool(base, L, NP, P, H, D)


def _queries(q, o, lse, ps: PkvPool, dev: int):
    """Addresses of q, o [T, Hq, D] bf16 and lse [T, Hq] fp32 (or None), then T and Hq."""
    qp = _arg(q, _bf16, 3, dev, "q")
    op = _arg(o, _bf16, 3, dev, "o")
    shape = q.shape
    if o.shape != shape:
        raise ValueError("o must match q")
    t, hq, d = shape
    if d != ps.head_dim:
        raise ValueError("q must have the pool's head_dim")
    if lse is None:
        return qp, op, None, t, hq
    lp = _arg(lse, _f32, 2, dev, "lse")
    if lse.shape != (t, hq):
        raise ValueError("lse must be [T, Hq]")
    return qp, op, lp, t, hq


def _tables(page_table, seq_lens, table_idx, batch: int, dev: int):
    """Addresses of page_table [rows, stride], seq_lens [B], table_idx [B] (or None), and the
    table's stride."""
    pp = _arg(page_table, _i32, 2, dev, "page_table")
    rows, stride = page_table.shape
    sp = _ints(seq_lens, batch, dev, "seq_lens")
    if table_idx is None:
        if rows < batch:
            raise ValueError("page_table must have a row per request")
        return pp, sp, None, stride
    return pp, sp, _ints(table_idx, batch, dev, "table_idx"), stride


def _ints(t, n: int, dev: int, name: str) -> int:
    """Address of an int32 tensor of n entries."""
    p = _arg(t, _i32, 1, dev, name)
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} entries")
    return p


def _workspace(workspace, dev: int):
    """(address, bytes) of a workspace tensor or None."""
    if workspace is None:
        return None, 0
    if workspace.get_device() != dev:
        raise ValueError(f"workspace is on {workspace.device}, the current device is cuda:{dev}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.nbytes


def pool_struct(pool: torch.Tensor) -> PkvPool:
    """Descriptor of a (2, layers, pages, page_size, kv_heads, head_dim) bf16 pool."""
    _want(pool, torch.bfloat16, "pool", 6)
    _contig(pool, "pool")
    if pool.shape[0] != 2:
        raise ValueError("pool dim 0 must be 2 (K, V)")
    _, L, NP, P, H, D = pool.shape
    return PkvPool(pool.data_ptr(), L, NP, P, H, D)


def pkv_init() -> None:
    _check(load().pkv_init())


def pkv_kv_store(pool, layer: int, k, v, out_loc, stream=None) -> None:
    """pool[0|1, layer, out_loc[i]] = k[i] | v[i]; k, v [N, Hkv, D] bf16 (row stride free)."""
    ps = pool_struct(pool)
    _want(k, torch.bfloat16, "k", 3)
    _want(v, torch.bfloat16, "v", 3)
    _want(out_loc, torch.int32, "out_loc", 1)
    _contig(out_loc, "out_loc")
    n = out_loc.shape[0]
    if k.shape != v.shape or k.shape[0] != n:
        raise ValueError("k, v must be [N, Hkv, D] with N = len(out_loc)")
    if k.stride(0) != v.stride(0) or k.stride(1) != k.shape[2] or k.stride(2) != 1 \
            or v.stride(1) != v.shape[2] or v.stride(2) != 1:
        raise ValueError("k and v rows must share a row stride with heads/dims contiguous")
    _check(load().pkv_kv_store(ctypes.byref(ps), int(layer), _ptr(k), _ptr(v), k.stride(0),
                               _ptr(out_loc), n, _stream(stream)))


def pkv_norm_rope_kv_store(pool, layer: int, q, k, v, q_out, positions, out_loc, cos_sin=None,
                           q_norm=None, k_norm=None, eps: float = 1e-6,
                           interleaved: bool = False, stream=None) -> None:
    """Norm and rotate q [N, Hq, D] into q_out (contiguous; q itself if q is) and k [N, Hkv, D],
    append k and v to the pool at out_loc [N]; rows may be strided (slices of a fused projection).
    cos_sin [positions, rot_dim] fp32, cosines first, or None (no rotation: positions may be None);
    q_norm, k_norm [D] bf16 weights or None. q and q_out None: append only."""
    dev = _device()
    ps = _pool_arg(pool, dev)
    n, d = k.shape[0], ps.head_dim
    kv_shape = (n, ps.num_kv_heads, d)
    kp, ks = _rows_arg(k, kv_shape, dev, "k")
    vp, vs = _rows_arg(v, kv_shape, dev, "v")
    if vs != ks:
        raise ValueError("k and v rows must share a row stride")
    qp = op = tp = pp = qn = kn = None
    hq = qs = rot = rows = 0
    if q is not None:
        hq = q.shape[1]
        qp, qs = _rows_arg(q, (n, hq, d), dev, "q")
        op = _arg(q_out, _bf16, 3, dev, "q_out")
        if q_out.shape != q.shape:
            raise ValueError("q_out must match q")
    if cos_sin is not None:
        tp = _arg(cos_sin, _f32, 2, dev, "cos_sin")
        rows, rot = cos_sin.shape
        pp = _ints(positions, n, dev, "positions")
    if q_norm is not None:
        qn = _arg(q_norm, _bf16, 1, dev, "q_norm")
        if q_norm.numel() != d:
            raise ValueError("q_norm must have head_dim entries")
    if k_norm is not None:
        kn = _arg(k_norm, _bf16, 1, dev, "k_norm")
        if k_norm.numel() != d:
            raise ValueError("k_norm must have head_dim entries")
    _check(load().pkv_norm_rope_kv_store(
        ctypes.byref(ps), int(layer), qp, qs, op, hq, kp, vp, ks, qn, kn, float(eps), tp, rows, rot,
        bool(interleaved), pp, _ints(out_loc, n, dev, "out_loc"), n, _handle(stream, dev)))


def pkv_decode_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                              max_seq_len_hint: int) -> int:
    return int(load().pkv_decode_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                max_seq_len_hint))


def pkv_paged_decode_attn(pool, layer: int, q, o, lse, page_table, seq_lens, scale: float,
                          max_seq_len_hint: int, workspace=None, table_idx=None,
                          stream=None) -> None:
    """Decode attention; q, o [B, Hq, D] bf16; lse [B, Hq] fp32 or None."""
    ps = pool_struct(pool)
    _want(q, torch.bfloat16, "q", 3)
    _want(o, torch.bfloat16, "o", 3)
    _contig(q, "q")
    _contig(o, "o")
    _want(page_table, torch.int32, "page_table", 2)
    _contig(page_table, "page_table")
    _want(seq_lens, torch.int32, "seq_lens", 1)
    B, Hq, D = q.shape
    if o.shape != q.shape or seq_lens.shape[0] != B:
        raise ValueError("o must match q and seq_lens must have batch entries")
    if lse is not None:
        _want(lse, torch.float32, "lse", 2)
        _contig(lse, "lse")
    if table_idx is not None:
        _want(table_idx, torch.int32, "table_idx", 1)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().pkv_paged_decode_attn(
        ctypes.byref(ps), int(layer), _ptr(q), _ptr(o), _ptr(lse), _ptr(page_table),
        page_table.shape[1], _ptr(table_idx), _ptr(seq_lens), B, Hq, float(scale),
        int(max_seq_len_hint), _ptr(workspace), ws_bytes, _stream(stream)))


def pkv_decode_mod_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                  max_keys_hint: int) -> int:
    return int(load().pkv_decode_mod_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                    max_keys_hint))


def _score_mod(soft_cap, alibi_slopes, window, prefix_lens, batch: int, hq: int,
               dev: int) -> PkvScoreMod:
    sp = pp = None
    if alibi_slopes is not None:
        sp = _arg(alibi_slopes, _f32, 1, dev, "alibi_slopes")
        if alibi_slopes.shape[0] != hq:
            raise ValueError("alibi_slopes must have one entry per q head")
    if prefix_lens is not None:
        pp = _ints(prefix_lens, batch, dev, "prefix_lens")
    if not -0x80000000 <= window <= 0x7fffffff:  # (ctypes would wrap it)
        raise ValueError("window must fit 32 bits")
    return PkvScoreMod(float(soft_cap), sp, int(window), pp)


def pkv_paged_decode_attn_mod(pool, layer: int, q, o, lse, page_table, seq_lens, scale: float,
                              max_keys_hint: int, workspace=None, soft_cap: float = 0.0,
                              alibi_slopes=None, window: int = 0, prefix_lens=None,
                              table_idx=None, stream=None) -> None:
    """Decode attention under score rules: a soft cap, alibi_slopes [Hq] fp32, a window, and
    prefix_lens [B] int32 first keys that stay visible. max_keys_hint: a bound on the keys a
    request sees (min(seq_len, window + prefix) with a window)."""
    dev = _device()
    ps = _pool_arg(pool, dev)
    qp, op, lp, B, Hq = _queries(q, o, lse, ps, dev)
    pp, sp, tp, stride = _tables(page_table, seq_lens, table_idx, B, dev)
    mod = _score_mod(soft_cap, alibi_slopes, window, prefix_lens, B, Hq, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    _check(load().pkv_paged_decode_attn_mod(
        ctypes.byref(ps), int(layer), qp, op, lp, pp, stride, tp, sp, B, Hq, float(scale), ctypes.byref(mod),
        int(max_keys_hint), ws, ws_bytes, _handle(stream, dev)))


def pkv_paged_decode_attn_store(pool, layer: int, q, k_new, v_new, o, lse, page_table, seq_lens,
                                scale: float, max_seq_len_hint: int, workspace=None,
                                table_idx=None, stream=None) -> None:
    """Decode step with store_kv fused: k_new, v_new [B, Hkv, D] bf16 go to key
    seq_lens[b] - 1 of each row, then decode as pkv_paged_decode_attn."""
    ps = pool_struct(pool)
    _want(q, torch.bfloat16, "q", 3)
    _want(o, torch.bfloat16, "o", 3)
    _contig(q, "q")
    _contig(o, "o")
    for t, name in ((k_new, "k_new"), (v_new, "v_new")):
        _want(t, torch.bfloat16, name, 3)
    if k_new.stride(0) != v_new.stride(0) or k_new.stride(1) != k_new.shape[2] \
            or k_new.stride(2) != 1 or v_new.stride(1) != v_new.shape[2] or v_new.stride(2) != 1:
        raise ValueError("k_new and v_new rows must share a row stride with heads/dims contiguous")
    _want(page_table, torch.int32, "page_table", 2)
    _contig(page_table, "page_table")
    _want(seq_lens, torch.int32, "seq_lens", 1)
    B, Hq, D = q.shape
    if o.shape != q.shape or seq_lens.shape[0] != B or k_new.shape[0] != B:
        raise ValueError("o must match q; seq_lens and k_new must have batch entries")
    if lse is not None:
        _want(lse, torch.float32, "lse", 2)
        _contig(lse, "lse")
    if table_idx is not None:
        _want(table_idx, torch.int32, "table_idx", 1)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().pkv_paged_decode_attn_store(
        ctypes.byref(ps), int(layer), _ptr(q), _ptr(k_new), _ptr(v_new), k_new.stride(0), _ptr(o),
        _ptr(lse), _ptr(page_table), page_table.shape[1], _ptr(table_idx), _ptr(seq_lens), B, Hq,
        float(scale), int(max_seq_len_hint), _ptr(workspace), ws_bytes, _stream(stream)))


def pkv_paged_decode_attn_noalloc(pool, layer: int, q, o, lse, page_table, seq_lens,
                                  scale: float, max_seq_len_hint: int, table_idx=None,
                                  stream=None) -> None:
    """Decode attention with no workspace, for callers that cannot allocate.

    The split-KV scratch is a fixed library-owned device array (32 MiB), so
    nothing is allocated; calls whose kernels overlap on the GPU race on it.
    """
    ps = pool_struct(pool)
    _want(q, torch.bfloat16, "q", 3)
    _want(o, torch.bfloat16, "o", 3)
    _contig(q, "q")
    _contig(o, "o")
    _want(page_table, torch.int32, "page_table", 2)
    _contig(page_table, "page_table")
    _want(seq_lens, torch.int32, "seq_lens", 1)
    B, Hq, D = q.shape
    if o.shape != q.shape or seq_lens.shape[0] != B:
        raise ValueError("o must match q and seq_lens must have batch entries")
    if lse is not None:
        _want(lse, torch.float32, "lse", 2)
        _contig(lse, "lse")
    if table_idx is not None:
        _want(table_idx, torch.int32, "table_idx", 1)
    _check(load().pkv_paged_decode_attn_noalloc(
        ctypes.byref(ps), int(layer), _ptr(q), _ptr(o), _ptr(lse), _ptr(page_table),
        page_table.shape[1], _ptr(table_idx), _ptr(seq_lens), B, Hq, float(scale),
        int(max_seq_len_hint), _stream(stream)))


def pkv_extend_workspace_size(batch: int, num_kv_heads: int, head_dim: int,
                              max_seq_len_hint: int, max_total_keys_hint: int = 0) -> int:
    """max_total_keys_hint: a bound on the sum of the call's seq_lens (0: none,
    batch x max_seq_len_hint is used)."""
    return int(load().pkv_extend_workspace_size(batch, num_kv_heads, head_dim,
                                                max_seq_len_hint, int(max_total_keys_hint)))


def pkv_paged_extend_attn(pool, layer: int, q, qo_indptr, o, lse, page_table, seq_lens,
                          scale: float, max_seq_len_hint: int, workspace, table_idx=None,
                          stream=None, max_total_keys_hint: int = 0) -> None:
    """Extend attention; q, o [T, Hq, D] bf16; qo_indptr [B+1]; lse [T, Hq] fp32 or None;
    workspace: device tensor of at least pkv_extend_workspace_size(...) bytes for the same
    hints."""
    ps = pool_struct(pool)
    _want(q, torch.bfloat16, "q", 3)
    _want(o, torch.bfloat16, "o", 3)
    _contig(q, "q")
    _contig(o, "o")
    _want(qo_indptr, torch.int32, "qo_indptr", 1)
    _want(page_table, torch.int32, "page_table", 2)
    _contig(page_table, "page_table")
    _want(seq_lens, torch.int32, "seq_lens", 1)
    T, Hq, D = q.shape
    B = seq_lens.shape[0]
    if o.shape != q.shape or qo_indptr.shape[0] != B + 1:
        raise ValueError("o must match q and qo_indptr must have batch+1 entries")
    if lse is not None:
        _want(lse, torch.float32, "lse", 2)
        _contig(lse, "lse")
    if table_idx is not None:
        _want(table_idx, torch.int32, "table_idx", 1)
    if workspace is not None:
        _contig(workspace, "workspace")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().pkv_paged_extend_attn(
        ctypes.byref(ps), int(layer), _ptr(q), _ptr(qo_indptr), _ptr(o), _ptr(lse),
        _ptr(page_table), page_table.shape[1], _ptr(table_idx), _ptr(seq_lens), B, T, Hq,
        float(scale), int(max_seq_len_hint), int(max_total_keys_hint), _ptr(workspace), ws_bytes,
        _stream(stream)))


def pkv_extend_mod_workspace_size(batch: int, total_q: int, num_q_heads: int, num_kv_heads: int,
                                  head_dim: int, max_seq_len_hint: int,
                                  max_total_keys_hint: int = 0) -> int:
    return int(load().pkv_extend_mod_workspace_size(batch, total_q, num_q_heads, num_kv_heads,
                                                    head_dim, max_seq_len_hint,
                                                    int(max_total_keys_hint)))


def pkv_paged_extend_attn_mod(pool, layer: int, q, qo_indptr, o, lse, page_table, seq_lens,
                              scale: float, max_seq_len_hint: int, workspace,
                              soft_cap: float = 0.0, alibi_slopes=None, window: int = 0,
                              prefix_lens=None, table_idx=None, stream=None,
                              max_total_keys_hint: int = 0) -> None:
    """Extend attention under score rules (as pkv_paged_decode_attn_mod's), chunk query j of
    request r at position seq_lens[r] - c_r + j; prefix_lens also lets the queries inside the
    prefix see the keys behind them."""
    dev = _device()
    ps = _pool_arg(pool, dev)
    qp, op, lp, T, Hq = _queries(q, o, lse, ps, dev)
    B = seq_lens.numel()
    pp, sp, tp, stride = _tables(page_table, seq_lens, table_idx, B, dev)
    mod = _score_mod(soft_cap, alibi_slopes, window, prefix_lens, B, Hq, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    _check(load().pkv_paged_extend_attn_mod(
        ctypes.byref(ps), int(layer), qp, _ints(qo_indptr, B + 1, dev, "qo_indptr"), op, lp, pp, stride,
        tp, sp, B, T, Hq, float(scale), ctypes.byref(mod), int(max_seq_len_hint), int(max_total_keys_hint), ws,
        ws_bytes, _handle(stream, dev)))


def pkv_paged_extend_attn_store(pool, layer: int, q, k_new, v_new, qo_indptr, o, lse,
                                page_table, seq_lens, scale: float, max_seq_len_hint: int,
                                workspace, table_idx=None, stream=None,
                                max_total_keys_hint: int = 0) -> None:
    """Extend step with store_kv fused: k_new, v_new [T, Hkv, D] bf16 (row t = query
    token t) go to the chunk's key positions of each row, then extend as
    pkv_paged_extend_attn."""
    ps = pool_struct(pool)
    _want(q, torch.bfloat16, "q", 3)
    _want(o, torch.bfloat16, "o", 3)
    _contig(q, "q")
    _contig(o, "o")
    for t, name in ((k_new, "k_new"), (v_new, "v_new")):
        _want(t, torch.bfloat16, name, 3)
    if k_new.stride(0) != v_new.stride(0) or k_new.stride(1) != k_new.shape[2] \
            or k_new.stride(2) != 1 or v_new.stride(1) != v_new.shape[2] or v_new.stride(2) != 1:
        raise ValueError("k_new and v_new rows must share a row stride with heads/dims contiguous")
    _want(qo_indptr, torch.int32, "qo_indptr", 1)
    _want(page_table, torch.int32, "page_table", 2)
    _contig(page_table, "page_table")
    _want(seq_lens, torch.int32, "seq_lens", 1)
    T, Hq, D = q.shape
    B = seq_lens.shape[0]
    if o.shape != q.shape or qo_indptr.shape[0] != B + 1:
        raise ValueError("o must match q and qo_indptr must have batch+1 entries")
    if k_new.shape[0] != T or v_new.shape[0] != T:
        raise ValueError("k_new and v_new must have total_q rows")
    if lse is not None:
        _want(lse, torch.float32, "lse", 2)
        _contig(lse, "lse")
    if table_idx is not None:
        _want(table_idx, torch.int32, "table_idx", 1)
    if workspace is not None:
        _contig(workspace, "workspace")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().pkv_paged_extend_attn_store(
        ctypes.byref(ps), int(layer), _ptr(q), _ptr(k_new), _ptr(v_new), k_new.stride(0),
        _ptr(qo_indptr), _ptr(o), _ptr(lse), _ptr(page_table), page_table.shape[1],
        _ptr(table_idx), _ptr(seq_lens), B, T, Hq, float(scale), int(max_seq_len_hint),
        int(max_total_keys_hint), _ptr(workspace), ws_bytes, _stream(stream)))


def pkv_tree_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                            max_tree_tokens: int, max_seq_len_hint: int) -> int:
    return int(load().pkv_tree_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                              max_tree_tokens, max_seq_len_hint))


def pkv_paged_tree_attn(pool, layer: int, q, qo_indptr, parents, o, lse, page_table, seq_lens,
                        scale: float, max_tree_tokens: int, max_seq_len_hint: int,
                        workspace=None, table_idx=None, stream=None) -> None:
    """Attention of drafted tokens: q, o [T, Hq, D] bf16, qo_indptr [B+1] and parents [T] int32
    (index within the request, -1 for a root); lse [T, Hq] fp32 or None; seq_lens count the
    drafted tokens, whose keys are in the pool."""
    dev = _device()
    ps = _pool_arg(pool, dev)
    qp, op, lp, T, Hq = _queries(q, o, lse, ps, dev)
    B = seq_lens.numel()
    pp, sp, tp, stride = _tables(page_table, seq_lens, table_idx, B, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    _check(load().pkv_paged_tree_attn(
        ctypes.byref(ps), int(layer), qp, _ints(qo_indptr, B + 1, dev, "qo_indptr"),
        _ints(parents, T, dev, "parents"), op, lp, pp, stride, tp, sp, B, T, Hq, float(scale),
        int(max_tree_tokens), int(max_seq_len_hint), ws, ws_bytes, _handle(stream, dev)))


def _mass_arg(key_mass, page_table, table_idx, batch: int, hkv: int, dev: int):
    """(address, stride) of key_mass [rows, Hkv, stride] fp32, a row per page_table row."""
    p = _arg(key_mass, _f32, 3, dev, "key_mass")
    rows, h, stride = key_mass.shape
    if h != hkv:
        raise ValueError("key_mass must have the pool's kv heads")
    if rows < (batch if table_idx is None else page_table.shape[0]):
        raise ValueError("key_mass must have a row per request, or per page_table row with "
                         "table_idx")
    return p, stride


def _int32(x, name: str) -> int:
    x = int(x)
    if not -0x80000000 <= x <= 0x7fffffff:  # (ctypes would wrap it)
        raise ValueError(f"{name} must fit 32 bits")
    return x


def pkv_decode_mass_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                   max_seq_len_hint: int) -> int:
    return int(load().pkv_decode_mass_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                     max_seq_len_hint))


def pkv_paged_decode_attn_mass(pool, layer: int, q, o, lse, key_mass, page_table, seq_lens,
                               scale: float, max_seq_len_hint: int, workspace,
                               soft_cap: float = 0.0, table_idx=None, stream=None) -> None:
    """Decode attention that adds each key's weight to key_mass [rows, Hkv, stride] fp32 (the
    newest key's entry starts here); workspace: pkv_decode_mass_workspace_size(...) bytes."""
    dev = _device()
    ps = _pool_arg(pool, dev)
    qp, op, lp, B, Hq = _queries(q, o, lse, ps, dev)
    pp, sp, tp, stride = _tables(page_table, seq_lens, table_idx, B, dev)
    mp, ms = _mass_arg(key_mass, page_table, table_idx, B, ps.num_kv_heads, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    _check(load().pkv_paged_decode_attn_mass(
        ctypes.byref(ps), int(layer), qp, op, lp, mp, ms, pp, stride, tp, sp, B, Hq, float(scale),
        float(soft_cap), _int32(max_seq_len_hint, "max_seq_len_hint"), ws, ws_bytes,
        _handle(stream, dev)))


def pkv_paged_extend_mass(pool, layer: int, q, qo_indptr, lse, key_mass, page_table, seq_lens,
                          scale: float, max_seq_len_hint: int = 0, soft_cap: float = 0.0,
                          num_last: int = 0, accumulate: bool = True, table_idx=None, stream=None,
                          max_total_keys_hint: int = 0) -> None:
    """The weights that a chunk's queries (all, or the last num_last) give to the keys of their
    rows, from the lse [T, Hq] of its extend call, into key_mass [rows, Hkv, stride] fp32: added
    to what the prefix's keys had if accumulate; the chunk's own keys start here."""
    dev = _device()
    ps = _pool_arg(pool, dev)
    qp = _arg(q, _bf16, 3, dev, "q")
    T, Hq, d = q.shape
    if d != ps.head_dim:
        raise ValueError("q must have the pool's head_dim")
    lp = _arg(lse, _f32, 2, dev, "lse")
    if lse.shape != (T, Hq):
        raise ValueError("lse must be [T, Hq]")
    B = seq_lens.numel()
    pp, sp, tp, stride = _tables(page_table, seq_lens, table_idx, B, dev)
    mp, ms = _mass_arg(key_mass, page_table, table_idx, B, ps.num_kv_heads, dev)
    _check(load().pkv_paged_extend_mass(
        ctypes.byref(ps), int(layer), qp, _ints(qo_indptr, B + 1, dev, "qo_indptr"), lp, mp, ms, pp,
        stride, tp, sp, B, T, Hq, float(scale), float(soft_cap), _int32(num_last, "num_last"),
        bool(accumulate), _int32(max_seq_len_hint, "max_seq_len_hint"), int(max_total_keys_hint),
        _handle(stream, dev)))


def pkv_kv_evict(pool, layer: int, key_mass, kept, page_table, seq_lens, budget: int,
                 num_first: int = 0, num_recent: int = 0, max_seq_len_hint: int = 0,
                 table_idx=None, stream=None) -> None:
    """Rows of more than `budget` keys cut to it, per kv head: the first num_first, the last
    num_recent and the heaviest by key_mass between stay, in order, moved together with their
    values and weights. kept [B, Hkv, budget] int32: the old index of each place, -1 where a row
    has fewer keys. seq_lens is not changed."""
    dev = _device()
    ps = _pool_arg(pool, dev)
    B = seq_lens.numel()
    budget = _int32(budget, "budget")
    pp, sp, tp, stride = _tables(page_table, seq_lens, table_idx, B, dev)
    mp, ms = _mass_arg(key_mass, page_table, table_idx, B, ps.num_kv_heads, dev)
    kp = _arg(kept, _i32, 3, dev, "kept")
    if kept.shape != (B, ps.num_kv_heads, budget):
        raise ValueError("kept must be [batch, Hkv, budget]")
    _check(load().pkv_kv_evict(
        ctypes.byref(ps), int(layer), mp, ms, pp, stride, tp, sp, B, budget,
        _int32(num_first, "num_first"), _int32(num_recent, "num_recent"), kp,
        _int32(max_seq_len_hint, "max_seq_len_hint"), _handle(stream, dev)))


def pkv_kv_rerope(pool, layer: int, page_table, seq_lens, old_freq, new_freq, old_positions=None,
                  new_positions=None, interleaved: bool = False, factor: float = 1.0,
                  max_seq_len_hint: int = 0, max_total_keys_hint: int = 0, table_idx=None,
                  stream=None) -> None:
    """Cached keys turned in place from old_positions * old_freq to new_positions * new_freq
    (times factor). old_freq, new_freq [rot_dim / 2] fp32, radians per position, one of them may be
    None (not rotated); positions [B, 1 or Hkv, stride] int32 by key index, or None: the index."""
    dev = _device()
    ps = _pool_arg(pool, dev)
    B = seq_lens.numel()
    pp, sp, tp, stride = _tables(page_table, seq_lens, table_idx, B, dev)
    fp = [None, None]
    pairs = None
    for x, (f, name) in enumerate(((old_freq, "old_freq"), (new_freq, "new_freq"))):
        if f is not None:
            fp[x] = _arg(f, _f32, 1, dev, name)
            if pairs is not None and f.numel() != pairs:
                raise ValueError("old_freq and new_freq must have the same length")
            pairs = f.numel()
    if pairs is None:
        raise ValueError("old_freq and new_freq may not both be None")
    at = [None, None]
    heads = width = 0
    for x, (t, name) in enumerate(((old_positions, "old_positions"),
                                   (new_positions, "new_positions"))):
        if t is not None:
            at[x] = _arg(t, _i32, 3, dev, name)
            if t.shape[0] != B or (width and t.shape[1:] != (heads, width)):
                raise ValueError(f"{name} must be [batch, 1 or Hkv, stride], both the same")
            _, heads, width = t.shape
    _check(load().pkv_kv_rerope(
        ctypes.byref(ps), int(layer), pp, stride, tp, sp, B, at[0], at[1], heads, width, fp[0],
        fp[1], 2 * pairs, bool(interleaved), float(factor),
        _int32(max_seq_len_hint, "max_seq_len_hint"), int(max_total_keys_hint),
        _handle(stream, dev)))


def pkv_cascade_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                               num_groups: int, max_prefix_len_hint: int,
                               max_suffix_len_hint: int) -> int:
    return int(load().pkv_cascade_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                 num_groups, max_prefix_len_hint,
                                                 max_suffix_len_hint))


def pkv_paged_cascade_decode_attn(pool, layer: int, q, o, lse, prefix_page_table, prefix_lens,
                                  member_indptr, members, page_table, seq_lens, scale: float,
                                  max_prefix_len_hint: int, max_suffix_len_hint: int, workspace,
                                  table_idx=None, stream=None) -> None:
    """Cascade decode: q, o [B, Hq, D] bf16; lse [B, Hq] fp32 or None; prefix_page_table
    [G, stride_p] and prefix_lens [G]; member_indptr [G+1] and members [B] partition the
    requests into groups; page_table rows and seq_lens [B] hold each request's suffix."""
    ps = pool_struct(pool)
    for t, name in ((q, "q"), (o, "o")):
        _want(t, torch.bfloat16, name, 3)
        _contig(t, name)
    for t, name, nd in ((prefix_page_table, "prefix_page_table", 2), (prefix_lens, "prefix_lens", 1),
                        (member_indptr, "member_indptr", 1), (members, "members", 1),
                        (page_table, "page_table", 2), (seq_lens, "seq_lens", 1)):
        _want(t, torch.int32, name, nd)
        _contig(t, name)
    B, Hq, D = q.shape
    G = prefix_lens.shape[0]
    if o.shape != q.shape or seq_lens.shape[0] != B or member_indptr.shape[0] != G + 1 \
            or prefix_page_table.shape[0] < G:
        raise ValueError("inconsistent cascade shapes")
    if lse is not None:
        _want(lse, torch.float32, "lse", 2)
        _contig(lse, "lse")
    if table_idx is not None:
        _want(table_idx, torch.int32, "table_idx", 1)
    if workspace is not None:
        _contig(workspace, "workspace")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().pkv_paged_cascade_decode_attn(
        ctypes.byref(ps), int(layer), _ptr(q), _ptr(o), _ptr(lse), _ptr(prefix_page_table),
        prefix_page_table.shape[1], _ptr(prefix_lens), _ptr(member_indptr), _ptr(members), G,
        _ptr(page_table), page_table.shape[1], _ptr(table_idx), _ptr(seq_lens), B, Hq,
        float(scale), int(max_prefix_len_hint), int(max_suffix_len_hint), _ptr(workspace),
        ws_bytes, _stream(stream)))


def pkv_merge_lse(o_a, lse_a, o_b, lse_b, o_out, lse_out=None, stream=None) -> None:
    """Merge two states: o_* [rows, H, D] fp32, lse_* [rows, H] fp32; o_out bf16 or fp32."""
    for t, name in ((o_a, "o_a"), (o_b, "o_b")):
        _want(t, torch.float32, name, 3)
        _contig(t, name)
    for t, name in ((lse_a, "lse_a"), (lse_b, "lse_b")):
        _want(t, torch.float32, name, 2)
        _contig(t, name)
    if o_out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("o_out must be fp32 or bf16")
    _contig(o_out, "o_out")
    rows, H, D = o_a.shape
    if o_b.shape != o_a.shape or o_out.shape != o_a.shape or lse_a.shape != (rows, H) \
            or lse_b.shape != (rows, H):
        raise ValueError("shape mismatch")
    if lse_out is not None:
        _want(lse_out, torch.float32, "lse_out", 2)
    _check(load().pkv_merge_lse(_ptr(o_a), _ptr(lse_a), _ptr(o_b), _ptr(lse_b), _ptr(o_out),
                                1 if o_out.dtype == torch.bfloat16 else 0, _ptr(lse_out), rows,
                                H, D, _stream(stream)))


def pkv_read_device_errors() -> int:
    """Read and clear the device error word (synchronises the device)."""
    v = ctypes.c_uint32(0)
    _check(load().pkv_read_device_errors(ctypes.byref(v)))
    return int(v.value)
