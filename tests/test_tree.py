"""Attention of drafted token trees over the paged cache (pkv_paged_tree_attn), against the
definition in 64 bits (attn_reference.py derives the tolerances)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from attn_reference import attend, check, stored_inputs
from helpers import ensure_built, gpu_inputs, nan_outputs
from paged_kv_attention_out_gb300 import workloads as W

INDPTR, SEQ, PAGE, TREE, TABLE_IDX = 0x8, 0x4, 0x2, 0x80, 0x10


def tree_case(seed, cached, drafts, **kw):
    """cached and drafted tokens per request, and a random tree for each."""
    cached, drafts = np.asarray(cached), np.asarray(drafts)
    case = W.random_case(seed, kind="extend", seq_lens=cached + drafts, chunk_lens=drafts, **kw)
    rng = np.random.default_rng(seed)
    parents = np.concatenate([[rng.integers(-1, j) if j else -1 for j in range(c)]
                              for c in drafts] or [[]]).astype(np.int32)
    return case, parents


def ancestors(case, parents):
    """visible(r, j, n) of the tree rule."""
    qo = case.qo_indptr

    def visible(r, j, n):
        first = n - int(qo[r + 1] - qo[r])
        vis = np.arange(n) < first
        while j >= 0:
            vis[first + j] = True
            par = parents[qo[r] + j]
            j = par if par < j else -1
        return vis

    return visible


def tree_run(case, parents, max_tree=None, hint=None, inputs=None, lse=True, scale=None):
    import paged_kv_attention_out_gb300 as pkv
    pool, k, v, q, t = inputs or gpu_inputs(case)
    pkv.pkv_kv_store(pool, case.layer, k, v, t["out_loc"])
    o, l = nan_outputs(q, lse)
    mt = case.max_chunk if max_tree is None else max_tree
    h = case.max_seq_len if hint is None else hint
    cap = h if h >= 1 else case.page_table.shape[1] * case.P
    n = pkv.pkv_tree_workspace_size(case.B, case.Hq, case.Hkv, case.D, mt, cap)
    ws = torch.full((max(n, 1),), 0xff, dtype=torch.uint8, device="cuda")
    pkv.pkv_paged_tree_attn(pool, case.layer, q, t["qo_indptr"],
                            torch.as_tensor(parents, dtype=torch.int32, device="cuda"), o, l,
                            t["page_table"], t["seq_lens"],
                            case.scale if scale is None else scale, mt, h, ws,
                            table_idx=t.get("table_idx"))
    torch.cuda.synchronize()
    return o, l


def tree_check(case, parents, **kw):
    import paged_kv_attention_out_gb300 as pkv
    ensure_built()
    pkv.pkv_read_device_errors()
    o, lse = tree_run(case, parents, **kw)
    assert pkv.pkv_read_device_errors() == 0
    kv, q = stored_inputs(case)
    scale = case.scale if kw.get("scale") is None else kw["scale"]
    check(o, lse, attend(kv, q, case.qo_indptr, scale, ancestors(case, parents)))
    return o, lse


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [1, 16, 7])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (4, 4), (28, 4), (16, 1)])
def test_tree_sweep(D, P, Hq, Hkv):
    case, parents = tree_case(3, [0, 1, 130, 500, 127, 300], [5, 1, 17, 3, 33, 1], Hq=Hq, Hkv=Hkv,
                              D=D, P=P)
    tree_check(case, parents)


@pytest.mark.gpu
@pytest.mark.parametrize("P", [8, 64, 128, 256])
def test_page_sizes_of_the_tma_boxes(P):
    case, parents = tree_case(4, [700, 128, 255, 63], [9, 20, 1, 40], Hq=8, Hkv=2, D=128, P=P)
    tree_check(case, parents)


@pytest.mark.gpu
@pytest.mark.parametrize("P", [1, 16])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 1)])
def test_trees_of_several_blocks(P, Hq, Hkv):
    """256 drafted tokens: several query blocks per request, the drafted keys in several tiles."""
    case, parents = tree_case(5, [1000, 0, 37], [256, 255, 129], Hq=Hq, Hkv=Hkv, D=64, P=P)
    tree_check(case, parents)


@pytest.mark.gpu
@pytest.mark.parametrize("cached", [127 - 8, 128 - 8, 129 - 8, 256 - 4, 384])
def test_drafts_around_a_tile_boundary(cached):
    case, parents = tree_case(6, [cached, cached + 1], [8, 64], Hq=16, Hkv=4, D=128, P=16)
    tree_check(case, parents)


@pytest.mark.gpu
@pytest.mark.parametrize("P", [1, 16])
@pytest.mark.parametrize("drafts", [[4, 2, 3], [64, 33, 50]])
def test_long_caches_are_shared_by_groups(P, drafts):
    """Blocks cut over many groups (one and two query tiles), merged from partial states."""
    case, parents = tree_case(7, [9000, 150, 4001], drafts, Hq=8, Hkv=2, D=128, P=P)
    tree_check(case, parents)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [1, 16, 7])
@pytest.mark.parametrize("Hq,Hkv,B,most", [(8, 2, 39, 64), (28, 4, 20, 36)])
@pytest.mark.parametrize("longest", [300, 2900])
def test_two_query_tiles_to_a_block(D, P, Hq, Hkv, B, most, longest):
    """More query tiles than groups: two to a block, a block to a group (short rows) or shared."""
    rng = np.random.default_rng(B + longest)
    drafts = [most, 1, most // 2, most // 2 + 1, 0] + list(rng.integers(1, most + 1, B - 5))
    cached = [longest, 0, 128, 127, 40] + list(rng.integers(0, 300, B - 5))
    case, parents = tree_case(16, cached, drafts, Hq=Hq, Hkv=Hkv, D=D, P=P)
    tree_check(case, parents)


@pytest.mark.gpu
@pytest.mark.parametrize("hint", [0, 100, 100000])
def test_the_hint_changes_only_the_schedule(hint):
    case, parents = tree_case(8, [900, 20, 333], [6, 7, 1], Hq=8, Hkv=2, D=64, P=16)
    tree_check(case, parents, hint=hint, max_tree=31)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [-0.11, 0.0, 1.5])
def test_any_finite_scale(scale):
    case, parents = tree_case(9, [300, 77], [9, 40], Hq=8, Hkv=2, D=64, P=1)
    o, lse = tree_run(case, parents, scale=scale)
    kv, q = stored_inputs(case)
    want_o, want_l, mag = attend(kv, q, case.qo_indptr, scale, ancestors(case, parents))
    # the score error grows with the scale (1.5 against 0.125 here): 12 times the usual part
    tol = (2 ** -8 + 12 * 2 ** -10) * mag + 2 ** -8 * np.abs(want_o) + 1e-30
    assert (np.abs(o.float().cpu().double().numpy() - want_o) <= tol).all()
    assert np.abs(lse.cpu().double().numpy() - want_l).max() <= 12 * 2 ** -11


@pytest.mark.gpu
def test_requests_without_drafts_and_rows_behind_the_last_one():
    """c_r = 0 computes nothing; rows of q past qo_indptr[batch] stay as they were."""
    import paged_kv_attention_out_gb300 as pkv
    case, parents = tree_case(10, [40, 300, 0, 9], [3, 0, 0, 5], Hq=8, Hkv=2, D=128, P=16,
                              use_table_idx=True)
    tree_check(case, parents, max_tree=5)
    pool, k, v, q, t = gpu_inputs(case)
    pkv.pkv_kv_store(pool, case.layer, k, v, t["out_loc"])
    more = torch.cat([q, q[:4]])
    o, lse = nan_outputs(more)
    par = torch.as_tensor(np.concatenate([parents, [-1] * 4]), dtype=torch.int32, device="cuda")
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    pkv.pkv_paged_tree_attn(pool, case.layer, more, t["qo_indptr"], par, o, lse, t["page_table"],
                            t["seq_lens"], case.scale, 5, case.max_seq_len, ws,
                            table_idx=t["table_idx"])
    assert torch.isfinite(o[:8].float()).all() and torch.isnan(o[8:].float()).all()
    assert torch.isfinite(lse[:8]).all() and torch.isnan(lse[8:]).all()


@pytest.mark.gpu
def test_a_chain_is_causal_extend():
    from helpers import compare, lse_compare, oracle_run
    case, _ = tree_case(11, [500, 64, 3], [70, 64, 9], Hq=8, Hkv=2, D=128, P=16)
    parents = np.concatenate([np.arange(c) - 1 for c in (70, 64, 9)])
    o, lse = tree_check(case, parents)
    want_o, want_l, _ = oracle_run(case)
    compare(o.float().cpu().double().numpy(), want_o)
    lse_compare(lse.cpu().double().numpy(), want_l)


@pytest.mark.gpu
def test_hundreds_of_requests():
    """More requests than a CTA has threads: the schedule's scan takes several rounds."""
    rng = np.random.default_rng(0)
    case, parents = tree_case(12, rng.integers(0, 200, 900), rng.integers(0, 5, 900), Hq=2, Hkv=1,
                              D=64, P=16)
    tree_check(case, parents)


@pytest.mark.gpu
def test_lse_is_optional_and_repeats_are_bitwise_equal():
    case, parents = tree_case(13, [2000, 60], [10, 30], Hq=8, Hkv=4, D=128, P=16)
    o1, _ = tree_run(case, parents, lse=False)
    o2, _ = tree_run(case, parents)
    assert torch.equal(o1, o2)


@pytest.mark.gpu
def test_bad_requests_are_flagged_and_the_others_computed():
    import paged_kv_attention_out_gb300 as pkv
    case, parents = tree_case(14, [100, 300, 20, 64], [9, 12, 5, 3], Hq=8, Hkv=2, D=64, P=16,
                              use_table_idx=True)
    kv, q = stored_inputs(case)
    qo = case.qo_indptr

    def flagged(bit, ok_requests, max_tree=None, par=parents, **tables):
        inputs = gpu_inputs(case)
        for name, (at, value) in tables.items():
            inputs[4][name][at] = value
        pkv.pkv_read_device_errors()
        # kv_store sees good tables: only the attention's are changed
        o, lse = tree_run(case, par, inputs=inputs, max_tree=max_tree)
        assert pkv.pkv_read_device_errors() == bit
        rows = np.concatenate([np.arange(qo[r], qo[r + 1]) for r in ok_requests])
        check(o, lse, attend(kv, q, qo, case.scale, ancestors(case, parents)), rows)

    flagged(TREE, [0, 2, 3], max_tree=9)  # request 1 has twelve
    flagged(SEQ, [0, 1, 3], seq_lens=(2, case.page_table.shape[1] * 16 + 1))
    flagged(INDPTR, [0, 2, 3], seq_lens=(1, 11))  # fewer keys than drafted tokens
    flagged(TABLE_IDX, [1, 2, 3], table_idx=(0, -1))
    bad = parents.copy()
    bad[qo[1] + 4] = 4  # its own parent: taken as a root, the token's row differs
    flagged(TREE, [0, 2, 3], par=bad)


@pytest.mark.gpu
@pytest.mark.parametrize("P", [1, 16])
def test_a_bad_page_reads_as_zeros(P):
    import paged_kv_attention_out_gb300 as pkv
    case, parents = tree_case(15, [200, 40], [6, 8], Hq=4, Hkv=2, D=64, P=P)
    inputs = gpu_inputs(case)
    pkv.pkv_kv_store(inputs[0], 0, inputs[1], inputs[2], inputs[4]["out_loc"])
    inputs[4]["page_table"][0, 3] = case.NP + 7
    pkv.pkv_read_device_errors()
    o, lse = tree_run(case, parents, inputs=inputs)
    assert pkv.pkv_read_device_errors() == PAGE
    kv, q = stored_inputs(case)
    for x in kv[0]:
        x[3 * P:4 * P] = 0
    check(o, lse, attend(kv, q, case.qo_indptr, case.scale, ancestors(case, parents)))


@pytest.mark.gpu
def test_two_graphs_replay_with_their_own_inputs():
    import paged_kv_attention_out_gb300 as pkv
    graphs = []
    for seed in (16, 17):
        case, parents = tree_case(seed, [900, 33, 250], [8, 40, 1], Hq=8, Hkv=2, D=128, P=16)
        pool, k, v, q, t = gpu_inputs(case)
        pkv.pkv_kv_store(pool, case.layer, k, v, t["out_loc"])
        par = torch.as_tensor(parents, device="cuda")
        o, lse = nan_outputs(q)
        n = pkv.pkv_tree_workspace_size(case.B, 8, 2, 128, 40, 1000)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")

        def call(o=o, lse=lse, case=case, pool=pool, q=q, t=t, par=par, ws=ws):
            pkv.pkv_paged_tree_attn(pool, case.layer, q, t["qo_indptr"], par, o, lse,
                                    t["page_table"], t["seq_lens"], case.scale, 40, 1000, ws)

        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append((g, case, parents, q, t, o, lse, call))
    for _ in range(3):
        for g, *_ in graphs:
            g.replay()
    for g, case, parents, q, t, o, lse, call in graphs:
        kv, hq = stored_inputs(case)
        check(o, lse, attend(kv, hq, case.qo_indptr, case.scale, ancestors(case, parents)))
        q.copy_(q.flip(0))
        t["seq_lens"][0] -= 300  # another schedule from the same captured launch
        o.fill_(float("nan"))
        g.replay()
        first = o.clone()
        call()
        assert torch.equal(first, o) and torch.isfinite(o.float()).all()


def _call(lib, pool, **kw):
    a = dict(layer=0, q=1 << 20, qo=64, par=64, o=1 << 20, lse=None, pt=64, stride=8, ti=None,
             sl=64, batch=1, total=4, hq=4, scale=1.0, max_tree=4, hint=16, ws=None, ws_bytes=0)
    a.update(kw)
    return lib.pkv_paged_tree_attn(
        ctypes.byref(pool), a["layer"], a["q"], a["qo"], a["par"], a["o"], a["lse"], a["pt"],
        a["stride"], a["ti"], a["sl"], a["batch"], a["total"], a["hq"],
        ctypes.c_float(a["scale"]), a["max_tree"], a["hint"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(layer=1), 1), (dict(batch=-1), 1), (dict(total=-1), 1), (dict(hq=3), 1),
    (dict(hq=34), 2), (dict(max_tree=0), 1), (dict(max_tree=257), 2), (dict(batch=65536), 2),
    (dict(stride=0), 1), (dict(scale=float("inf")), 1), (dict(q=None), 1), (dict(par=None), 1),
    (dict(q=(1 << 20) + 8), 1), (dict(qo=2), 1), (dict(stride=1 << 31), 2),
])
def test_refusals(kw, status):
    ensure_built()
    from paged_kv_attention_out_gb300 import binding
    pool = binding.PkvPool(1 << 30, 1, 10, 16, 2, 64)
    assert _call(binding.load(), pool, **kw) == status


def test_nothing_to_do_and_workspace_of_bad_sizes():
    ensure_built()
    from paged_kv_attention_out_gb300 import binding
    lib = binding.load()
    pool = binding.PkvPool(1 << 30, 1, 10, 16, 2, 64)
    assert _call(lib, pool, batch=0, q=None) == 0
    assert _call(lib, pool, total=0, q=None) == 0
    for bad in ((0, 8, 2, 64, 4, 9), (1, 9, 2, 64, 4, 9), (1, 8, 2, 96, 4, 9), (1, 8, 2, 64, 0, 9),
                (1, 8, 2, 64, 257, 9), (1, 8, 2, 64, 4, 0), (1, 64, 2, 64, 4, 9)):
        assert lib.pkv_tree_workspace_size(*bad) == 0


@pytest.mark.gpu
def test_a_small_workspace_is_refused():
    import paged_kv_attention_out_gb300 as pkv
    case, parents = tree_case(18, [5000], [8], Hq=8, Hkv=2, D=64, P=16)
    pool, k, v, q, t = gpu_inputs(case)
    o, lse = nan_outputs(q)
    n = pkv.pkv_tree_workspace_size(1, 8, 2, 64, 8, 5008)
    assert n > 0
    for ws in (None, torch.empty(n - 1, dtype=torch.uint8, device="cuda")):
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_paged_tree_attn(pool, 0, q, t["qo_indptr"], torch.as_tensor(parents).cuda(), o,
                                    lse, t["page_table"], t["seq_lens"], case.scale, 8, 5008, ws)
        assert e.value.status == 3
