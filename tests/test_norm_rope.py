"""A step's q and k normed and rotated and its k and v appended to the pool in one launch
(pkv_norm_rope_kv_store), against the formula in 64 bits.

Tolerance: everything is fp32 until one rounding to bf16, so a value y of the exact result may be
off by half a bf16 step, 2^-8 |y|, plus fp32 errors. A rotated value is a sum of two products of
magnitude at most R = sqrt(a^2 + b^2) of its pair: the norm's factor (a mean of D squares by a
tree of at most 19 additions, rsqrtf within 2 ulp, three products) and the rotation are at most
40 roundings of 2^-24 relative to R, below 2^-18 R."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from helpers import ensure_built

HALF_BF16 = 2.0 ** -8
FP32_PART = 2.0 ** -18


def rope_table(positions, rot, device="cuda"):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().to(device)


def reference(x, w, eps, table, pos, interleaved):
    """(value, pair radius) in 64 bits of x [N, H, D] normed by w and rotated."""
    x = x.double().cpu()
    if w is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double().cpu()
    r = x.abs()
    if table is None:
        return x, r
    rot = table.shape[1]
    t = table.double().cpu()[pos.long().cpu()][:, None]
    c, s = t[..., :rot // 2], t[..., rot // 2:]
    y = x.clone()
    if interleaved:
        ia, ib = slice(0, rot, 2), slice(1, rot, 2)
    else:
        ia, ib = slice(0, rot // 2), slice(rot // 2, rot)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    r[..., ia] = r[..., ib] = (a * a + b * b).sqrt()
    return y, r


def check(got, want, radius, what):
    err = (got.double().cpu() - want).abs()
    tol = HALF_BF16 * want.abs() + FP32_PART * radius
    assert torch.isfinite(got.float()).all(), what
    assert (err <= tol).all(), f"{what}: {float((err - tol).max()):.3e} past the tolerance"


def setup(n, hq, hkv, d, page, rot, norm, seed=0, fused=True, table_rows=500):
    ensure_built()
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = -(-(n + 5) // page) + 2
    pool = torch.randn(2, 3, pages, page, hkv, d, generator=g, device="cuda").bfloat16()
    if fused:
        qkv = torch.randn(n, (hq + 2 * hkv) * d, generator=g, device="cuda").bfloat16()
        q, k, v = (x.view(n, -1, d) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    else:
        q, k, v = (torch.randn(n, h, d, generator=g, device="cuda").bfloat16()
                   for h in (hq, hkv, hkv))
    w = [(1 + torch.randn(d, generator=g, device="cuda") / 4).bfloat16() if norm else None
         for _ in (0, 1)]
    table = rope_table(table_rows, rot) if rot else None
    pos = torch.randint(0, table_rows, (n,), generator=g, device="cuda", dtype=torch.int32)
    loc = torch.randperm(pages * page, generator=g, device="cuda")[:n].int()
    return pool, q, k, v, w, table, pos, loc


def run_and_check(pool, q, k, v, w, table, pos, loc, eps=1e-6, interleaved=False, in_place=False):
    import paged_kv_attention_out_gb300 as pkv
    before = pool.clone()
    q0 = q.clone()
    q_out = q if in_place else torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    pkv.pkv_read_device_errors()
    pkv.pkv_norm_rope_kv_store(pool, 1, q, k, v, q_out, pos, loc, table, q_norm=w[0], k_norm=w[1],
                               eps=eps, interleaved=interleaved)
    assert pkv.pkv_read_device_errors() == 0
    check(q_out, *reference(q0, w[0], eps, table, pos, interleaved), "q")
    rows = pool[0, 1].flatten(0, 1)[loc.long()]
    check(rows, *reference(k, w[1], eps, table, pos, interleaved), "k")
    want = before.clone()
    want[0, 1].flatten(0, 1)[loc.long()] = rows
    want[1, 1].flatten(0, 1)[loc.long()] = v
    assert torch.equal(pool.view(torch.int16), want.view(torch.int16)), "v bits or other rows"


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (128, 16), (128, 48), (128, 0),
                                   (64, 64), (64, 32), (64, 16)])
def test_every_rotation_matches_the_formula(d, rot, norm, interleaved):
    run_and_check(*setup(37, 8, 2, d, 16, rot, norm, seed=rot), interleaved=interleaved)


@pytest.mark.gpu
@pytest.mark.parametrize("n,hq,hkv,d,page", [(1, 1, 1, 64, 1), (1, 32, 8, 128, 16),
                                             (2, 28, 4, 128, 7), (333, 40, 8, 128, 64),
                                             (5, 71, 1, 64, 1), (3, 128, 16, 128, 16),
                                             (1000, 12, 4, 64, 1)])
@pytest.mark.parametrize("fused", [False, True])
def test_head_layouts_and_lengths(n, hq, hkv, d, page, fused):
    run_and_check(*setup(n, hq, hkv, d, page, d, True, seed=n, fused=fused))


@pytest.mark.gpu
def test_in_place_rows_with_norm_of_one_side_only():
    pool, q, k, v, w, table, pos, loc = setup(50, 8, 4, 128, 16, 128, True, fused=False)
    run_and_check(pool, q, k, v, [w[0], None], table, pos, loc, in_place=True)
    run_and_check(pool, q, k, v, [None, w[1]], table, pos, loc, eps=0.0)


@pytest.mark.gpu
def test_without_norm_or_rotation_it_is_kv_store():
    import paged_kv_attention_out_gb300 as pkv
    pool, q, k, v, _, _, _, loc = setup(90, 8, 4, 64, 16, 0, False)
    k.view(torch.int16)[3, 0, 5] = 0x7fc1  # a NaN's payload survives
    other = pool.clone()
    q_out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    pkv.pkv_norm_rope_kv_store(pool, 2, q, k, v, q_out, None, loc)
    pkv.pkv_kv_store(other, 2, k, v, loc)
    assert torch.equal(pool.view(torch.int16), other.view(torch.int16))
    assert torch.equal(q_out, q)
    pool.copy_(other.flip(2))
    pkv.pkv_kv_store(other.copy_(pool), 2, k, v, loc)
    pkv.pkv_norm_rope_kv_store(pool, 2, None, k, v, None, None, loc)  # append only
    assert torch.equal(pool.view(torch.int16), other.view(torch.int16))


@pytest.mark.gpu
def test_large_and_tiny_values():
    pool, q, k, v, w, table, pos, loc = setup(8, 4, 2, 128, 1, 128, True)
    q[0] *= 1e15
    q[1] *= 1e-15
    q[2] = 0
    k[0] *= 1e15
    run_and_check(pool, q, k, v, w, table, pos, loc)


@pytest.mark.gpu
def test_bad_positions_and_slots_are_flagged_and_skipped():
    import paged_kv_attention_out_gb300 as pkv
    pool, q, k, v, w, table, pos, loc = setup(6, 4, 2, 64, 1, 64, True, table_rows=10)
    pos[1], pos[2] = 10, -1
    loc_bad = loc.clone()
    loc_bad[3], loc_bad[4] = -1, pool.shape[2] * pool.shape[3]
    q_out = torch.zeros(q.shape, dtype=q.dtype, device="cuda")
    before = pool.clone()
    pkv.pkv_read_device_errors()
    pkv.pkv_norm_rope_kv_store(pool, 0, q, k, v, q_out, pos, loc_bad, table)
    assert pkv.pkv_read_device_errors() == 0x41
    good = [0, 3, 4, 5]
    want, radius = reference(q[good], None, 0, table, pos[good], False)
    check(q_out[good], want, radius, "q")
    assert not q_out[[1, 2]].any()
    touched = (pool != before)[:, 0].flatten(1, 2).any(-1).any(-1).any(0)
    assert set(touched.nonzero().flatten().tolist()) == {int(loc[0]), int(loc[5])}


@pytest.mark.gpu
def test_replay_in_a_graph_follows_new_inputs():
    import paged_kv_attention_out_gb300 as pkv
    pool, q, k, v, w, table, pos, loc = setup(20, 8, 2, 128, 16, 128, True)
    q_out = torch.empty(q.shape, dtype=q.dtype, device="cuda")

    def call():
        pkv.pkv_norm_rope_kv_store(pool, 1, q, k, v, q_out, pos, loc, table, q_norm=w[0],
                                   k_norm=w[1])

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    q.copy_(q.flip(0))
    k.copy_(k.flip(0))
    loc.copy_(loc.flip(0))
    graph.replay()
    got_q, got_pool = q_out.clone(), pool.clone()
    call()
    assert torch.equal(got_q, q_out) and torch.equal(got_pool, pool)
    check(q_out, *reference(q, w[0], 1e-6, table, pos, False), "q")


def _call(lib, pool, **kw):
    a = dict(layer=0, q=1 << 20, qs=256, q_out=2 << 20, hq=2, k=3 << 20, v=4 << 20, kvs=128,
             qn=None, kn=None, eps=1e-6, table=5 << 20, rows=100, rot=64, inter=0, pos=6 << 20,
             loc=7 << 20, n=1)
    a.update(kw)
    return lib.pkv_norm_rope_kv_store(
        ctypes.byref(pool), a["layer"], a["q"], a["qs"], a["q_out"], a["hq"], a["k"], a["v"],
        a["kvs"], a["qn"], a["kn"], ctypes.c_float(a["eps"]), a["table"], a["rows"], a["rot"],
        a["inter"], a["pos"], a["loc"], a["n"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(layer=2), 1), (dict(n=-1), 1), (dict(n=1 << 31), 2), (dict(hq=-1), 1),
    (dict(rot=8), 1), (dict(rot=80), 1), (dict(rot=-16), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(k=None), 1), (dict(q_out=None), 1), (dict(table=None), 1),
    (dict(pos=None), 1), (dict(rows=0), 1), (dict(k=(3 << 20) + 2), 1), (dict(qn=8), 1),
    (dict(kvs=64), 1), (dict(kvs=130), 1), (dict(qs=64), 1), (dict(loc=2), 1),
    (dict(q_out=1 << 20), 1),  # in place needs contiguous rows
    (dict(q_out=(3 << 20) - 128), 1),  # q_out runs into k
    (dict(k=1 << 30), 1), (dict(q=1 << 30), 1),  # k, q inside the pool
])
def test_refusals(kw, status):
    ensure_built()
    from paged_kv_attention_out_gb300 import binding
    pool = binding.PkvPool(1 << 30, 2, 10, 16, 2, 64)
    assert _call(binding.load(), pool, **kw) == status


def test_no_tokens_is_a_no_op():
    ensure_built()
    from paged_kv_attention_out_gb300 import binding
    pool = binding.PkvPool(1 << 30, 2, 10, 16, 2, 64)
    assert _call(binding.load(), pool, n=0, k=None, v=None, q=None) == 0


@pytest.mark.gpu
def test_binding_checks_tensors_before_the_library():
    import paged_kv_attention_out_gb300 as pkv
    pool, q, k, v, w, table, pos, loc = setup(6, 4, 2, 64, 1, 64, True)
    q_out = torch.empty(q.shape, dtype=q.dtype, device="cuda")

    def call(**kw):
        a = dict(pool=pool, q=q, k=k, v=v, q_out=q_out, positions=pos, out_loc=loc, cos_sin=table)
        a.update(kw)
        pkv.pkv_norm_rope_kv_store(layer=0, **a)

    for kw in (dict(k=k.cpu()), dict(v=v.float()), dict(out_loc=loc.long()),
               dict(cos_sin=table.double()), dict(pool=pool.half())):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(k=k[:5]), dict(v=v[:, :1]), dict(out_loc=loc[:5]), dict(positions=pos[::2]),
               dict(q_out=q_out[:, :2].contiguous()), dict(q_out=q_out.transpose(0, 1)),
               dict(k=k.transpose(1, 2).contiguous().transpose(1, 2)), dict(q_norm=w[0][:32])):
        with pytest.raises(ValueError):
            call(**kw)
