"""Decode and extend attention under score rules (pkv_paged_decode_attn_mod,
pkv_paged_extend_attn_mod) against the definition in 64 bits (attn_reference.py derives the
tolerances)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from attn_reference import attend, check, stored_inputs
from helpers import ensure_built, gpu_inputs, nan_outputs
from paged_kv_attention_out_gb300 import workloads as W

PAGE = 0x2


class Rules:
    """The rules of a call, as its keyword arguments and as the reference's functions."""

    def __init__(self, case, cap=0.0, alibi=False, window=0, prefix=None):
        self.case, self.cap, self.window = case, cap, window
        self.slopes = 2.0 ** (-8.0 * np.arange(1, case.Hq + 1) / case.Hq) if alibi else None
        if alibi:
            self.slopes = self.slopes.astype(np.float32)
        self.prefix = None if prefix is None else np.resize(np.asarray(prefix, np.int32), case.B)

    def first(self, r):
        """Position of request r's first query."""
        n = int(self.case.seq_lens[r])
        if self.case.kind == "decode":
            return n - 1
        return n - int(self.case.qo_indptr[r + 1] - self.case.qo_indptr[r])

    def visible(self, r, j, n):
        i, t = np.arange(n), self.first(r) + j
        vis = i <= t
        if self.window:
            vis &= t - i < self.window
        return vis if self.prefix is None else vis | (i < self.prefix[r])

    def rule(self, s, r, j, h, idx):
        if self.cap:
            s = self.cap * np.tanh(s / self.cap)
        if self.slopes is not None:
            s = s - float(self.slopes[h]) * np.abs(self.first(r) + j - idx)
        return s

    def kwargs(self):
        return dict(soft_cap=self.cap, window=self.window,
                    alibi_slopes=None if self.slopes is None else torch.as_tensor(self.slopes).cuda(),
                    prefix_lens=None if self.prefix is None else torch.as_tensor(self.prefix).cuda())

    def max_keys(self):
        """A bound on the keys a decode query sees."""
        n = self.case.max_seq_len
        if not self.window:
            return n
        return min(n, self.window + (0 if self.prefix is None else max(0, int(self.prefix.max()))))

    def want(self, scale=None):
        case = self.case
        kv, q = stored_inputs(case)
        qo = np.arange(case.B + 1) if case.kind == "decode" else case.qo_indptr
        return attend(kv, q, qo, case.scale if scale is None else scale, self.visible, self.rule)


def mod_run(rules, inputs=None, hint=None, scale=None, lse=True, before=None, stale=None):
    import paged_kv_attention_out_gb300 as pkv
    case = rules.case
    pool, k, v, q, t = inputs or gpu_inputs(case)
    pkv.pkv_kv_store(pool, case.layer, k, v, t["out_loc"])
    if before is not None:
        before(pool, t)
    o, l = nan_outputs(q, lse)
    scale = case.scale if scale is None else scale
    if case.kind == "decode":
        h = rules.max_keys() if hint is None else hint
        n = pkv.pkv_decode_mod_workspace_size(case.B, case.Hq, case.Hkv, case.D, h)
        ws = torch.full((max(n, 1),), 0xff, dtype=torch.uint8, device="cuda")
        pkv.pkv_paged_decode_attn_mod(pool, case.layer, q, o, l, t["page_table"], t["seq_lens"],
                                      scale, h, ws, table_idx=t.get("table_idx"), **rules.kwargs())
    else:
        h, total = case.max_seq_len, int(case.seq_lens.sum())
        n = pkv.pkv_extend_mod_workspace_size(case.B, case.total_q, case.Hq, case.Hkv, case.D, h,
                                              total)
        ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")  # NaN bits
        if stale is not None:  # what an earlier call may have left
            ws[:n // 16 * 16].view(torch.int32).view(-1, 4)[:] = torch.tensor(stale).cuda()
        pkv.pkv_paged_extend_attn_mod(pool, case.layer, q, t["qo_indptr"], o, l, t["page_table"],
                                      t["seq_lens"], scale, h, ws, table_idx=t.get("table_idx"),
                                      max_total_keys_hint=total, **rules.kwargs())
    torch.cuda.synchronize()
    return o, l


def mod_check(rules, **kw):
    import paged_kv_attention_out_gb300 as pkv
    ensure_built()
    pkv.pkv_read_device_errors()
    o, lse = mod_run(rules, **kw)
    assert pkv.pkv_read_device_errors() == 0
    check(o, lse, rules.want(kw.get("scale")))
    return o, lse


RULES = [
    dict(cap=30.0), dict(cap=2.0), dict(alibi=True), dict(window=100), dict(window=1),
    dict(window=1000), dict(prefix=[40, 0, 700]), dict(window=64, prefix=[5, 0, 130, 300]),
    dict(cap=1.0, alibi=True), dict(cap=50.0, window=200), dict(alibi=True, window=90, prefix=[17]),
    dict(cap=20.0, alibi=True, window=129, prefix=[128, 1000]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("rule", RULES, ids=str)
@pytest.mark.parametrize("D,P,Hq,Hkv", [(64, 1, 8, 2), (128, 16, 32, 8), (128, 7, 7, 1)])
def test_decode_rules(rule, D, P, Hq, Hkv):
    case = W.random_case(3, seq_lens=[1, 40, 513, 900, 130, 64], Hq=Hq, Hkv=Hkv, D=D, P=P,
                         use_table_idx=True)
    mod_check(Rules(case, **rule))


@pytest.mark.gpu
@pytest.mark.parametrize("rule", RULES, ids=str)
@pytest.mark.parametrize("D,P,Hq,Hkv", [(64, 1, 4, 4), (128, 16, 8, 2), (128, 7, 7, 1)])
def test_extend_rules(rule, D, P, Hq, Hkv):
    case = W.random_case(4, kind="extend", seq_lens=[1, 160, 513, 260, 700],
                         chunk_lens=[1, 160, 13, 129, 70], Hq=Hq, Hkv=Hkv, D=D, P=P,
                         use_table_idx=True)
    mod_check(Rules(case, **rule))


@pytest.mark.gpu
@pytest.mark.parametrize("rule", RULES, ids=str)
@pytest.mark.parametrize("D,P,Hq,Hkv", [(64, 1, 4, 4), (128, 16, 8, 2)])
def test_extend_rules_of_many_requests(rule, D, P, Hq, Hkv):
    """More requests than the direct form takes: keys gathered first, blocks in order of cost."""
    rng = np.random.default_rng(1)
    chunks = np.concatenate([[129, 70], rng.integers(1, 3, 270)])
    seqs = np.concatenate([[513, 300], chunks[2:] + rng.integers(0, 40, 270)])
    case = W.random_case(16, kind="extend", seq_lens=seqs, chunk_lens=chunks, Hq=Hq, Hkv=Hkv, D=D,
                         P=P)
    mod_check(Rules(case, **rule))


@pytest.mark.gpu
@pytest.mark.parametrize("rule", [dict(cap=3.0, alibi=True, window=50), dict(prefix=[30])], ids=str)
@pytest.mark.parametrize("scale", [-0.125, 0.0])
def test_scales_of_many_requests(rule, scale):
    case = W.random_case(17, kind="extend", seq_lens=[150] + [5] * 260, chunk_lens=[64] + [2] * 260,
                         Hq=4, Hkv=2, D=64, P=16)
    mod_check(Rules(case, **rule), scale=scale)


@pytest.mark.gpu
def test_extend_tables_are_checked_in_both_forms():
    """Malformed qo_indptr, lengths past the row and bad pages are flagged; others are computed."""
    import paged_kv_attention_out_gb300 as pkv
    for more in (0, 260):
        case = W.random_case(18, kind="extend", seq_lens=[100, 300, 64] + [3] * more,
                             chunk_lens=[40, 100, 20] + [2] * more, Hq=4, Hkv=2, D=64, P=16)
        rules = Rules(case, window=70, cap=20.0)
        want = rules.want()
        qo = case.qo_indptr

        def flagged(bit, ok, change):
            pkv.pkv_read_device_errors()
            o, lse = mod_run(rules, before=change)
            assert pkv.pkv_read_device_errors() == bit
            check(o, lse, want, np.concatenate([np.arange(qo[r], qo[r + 1]) for r in ok]))

        def set_(name, at, value):
            def change(pool, t):
                t[name][at] = value
            return change

        flagged(0x4, [0], set_("seq_lens", 1, case.page_table.shape[1] * 16 + 1))
        flagged(0x8, [0], set_("seq_lens", 1, 50))
        flagged(PAGE, [0, 2], set_("page_table", (1, 18), case.NP + 3))


LONG_RULES = [
    dict(cap=30.0), dict(cap=2.0), dict(alibi=True), dict(window=2000), dict(prefix=[40, 2700]),
    dict(window=64, prefix=[5, 2900, 130]), dict(cap=1.0, alibi=True), dict(cap=50.0, window=2500),
    dict(alibi=True, window=90, prefix=[17]), dict(cap=20.0, alibi=True, window=129, prefix=[128, 1000]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("rule", LONG_RULES, ids=str)
@pytest.mark.parametrize("D,P,Hq,Hkv", [(64, 1, 4, 2), (128, 16, 8, 2), (128, 7, 7, 1),
                                        (64, 64, 16, 1)])
def test_few_queries_over_long_rows(rule, D, P, Hq, Hkv):
    """The direct form: blocks of one and of two query tiles, shared by groups of CTAs."""
    case = W.random_case(21, kind="extend", seq_lens=[3000, 2817, 1], chunk_lens=[37, 1, 1], Hq=Hq,
                         Hkv=Hkv, D=D, P=P, use_table_idx=True)
    mod_check(Rules(case, **rule))


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [-0.125, 0.0])
@pytest.mark.parametrize("rule", [dict(cap=3.0), dict(cap=3.0, alibi=True), dict(prefix=[900])],
                         ids=str)
def test_scales_of_few_queries_over_long_rows(scale, rule):
    case = W.random_case(22, kind="extend", seq_lens=[3000, 500], chunk_lens=[9, 40], Hq=4, Hkv=2,
                         D=64, P=16)
    mod_check(Rules(case, **rule), scale=scale)


@pytest.mark.gpu
def test_pages_outside_the_rules_are_never_read_over_long_rows():
    case = W.random_case(23, kind="extend", seq_lens=[4000, 3500], chunk_lens=[40, 13], Hq=8, Hkv=2,
                         D=64, P=16)
    rules = Rules(case, window=1900, prefix=[20, 0], cap=10.0)

    def free(pool, t):
        for r in range(case.B):
            first_seen = rules.first(r) - 1899
            gone = np.arange(int(rules.prefix[r]), first_seen)
            slots = torch.as_tensor(np.asarray(case.token_slots[r])[gone].astype(np.int64)).cuda()
            pool[:, 0].flatten(1, 2)[:, slots] = float("nan")
            for pg in range(int(rules.prefix[r] + 15) // 16, first_seen // 16):
                t["page_table"][r, pg] = -7 - pg

    mod_check(rules, before=free)


@pytest.mark.gpu
@pytest.mark.parametrize("P", [1, 16])
@pytest.mark.parametrize("rule", [dict(cap=30.0), dict(window=1000, prefix=[200]),
                                  dict(alibi=True)], ids=str)
def test_a_short_chunk_over_a_long_prefix_is_shared_by_the_whole_gpu(rule, P):
    case = W.random_case(19, kind="extend", seq_lens=[9000, 130], chunk_lens=[20, 3], Hq=8, Hkv=2,
                         D=128, P=P)
    mod_check(Rules(case, **rule))


@pytest.mark.gpu
@pytest.mark.parametrize("rule", [dict(window=300), dict(cap=25.0, window=2000, prefix=[700]),
                                  dict(alibi=True)], ids=str)
def test_long_rows(rule):
    """Splits and their merge in decode, many key tiles behind a gap in extend."""
    case = W.random_case(5, seq_lens=[9000, 300, 4097], Hq=8, Hkv=2, D=128, P=16)
    mod_check(Rules(case, **rule))
    case = W.random_case(6, kind="extend", seq_lens=[5000, 2049, 300], chunk_lens=[40, 129, 9],
                         Hq=8, Hkv=2, D=128, P=16)
    mod_check(Rules(case, **rule))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["decode", "extend"])
@pytest.mark.parametrize("scale", [-0.125, 0.0])
@pytest.mark.parametrize("rule", [dict(cap=3.0), dict(cap=3.0, alibi=True, window=50),
                                  dict(alibi=True, prefix=[200])], ids=str)
def test_negative_and_zero_scales(kind, scale, rule):
    kw = dict(chunk_lens=[30, 64]) if kind == "extend" else {}
    case = W.random_case(7, kind=kind, seq_lens=[150, 260], Hq=8, Hkv=2, D=64, P=16, **kw)
    mod_check(Rules(case, **rule), scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["decode", "extend"])
@pytest.mark.parametrize("cap", [1e-2, 0.5, 7.5, 1e4, 1e8])
def test_caps_of_any_size(kind, cap):
    """Caps that saturate every score, caps at the border of the two tanh forms, and caps far above
    every score."""
    kw = dict(chunk_lens=[30, 64]) if kind == "extend" else {}
    case = W.random_case(8, kind=kind, seq_lens=[150, 400], Hq=8, Hkv=2, D=128, P=1, **kw)
    mod_check(Rules(case, cap=cap))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["decode", "extend"])
def test_no_rules_equal_the_plain_call_bitwise(kind):
    import paged_kv_attention_out_gb300 as pkv
    from helpers import gpu_attention
    kw = dict(chunk_lens=[30, 300]) if kind == "extend" else {}
    case = W.random_case(9, kind=kind, seq_lens=[1500, 400], Hq=8, Hkv=2, D=128, P=16, **kw)
    inputs = gpu_inputs(case)
    o, lse = mod_run(Rules(case), inputs=inputs)
    o2, lse2 = gpu_attention(case, inputs[0], inputs[3], inputs[4])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # a window nobody reaches changes nothing but the kernel
    check(*mod_run(Rules(case, window=100000), inputs=inputs), Rules(case).want())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["decode", "extend"])
def test_pages_outside_the_rules_are_never_read(kind):
    """Freed pages: table entries outside the window and prefix are garbage, their rows NaN."""
    kw = dict(chunk_lens=[40, 130]) if kind == "extend" else {}
    case = W.random_case(10, kind=kind, seq_lens=[900, 700], Hq=8, Hkv=2, D=64, P=16, **kw)
    rules = Rules(case, window=100, prefix=[20, 0], cap=10.0)

    def free(pool, t):
        for r in range(case.B):
            n = int(case.seq_lens[r])
            first_seen = max(0, rules.first(r) - 99)
            for pg in range(n // 16 + 1):
                if pg * 16 >= rules.prefix[r] and pg * 16 + 16 <= first_seen:
                    t["page_table"][r, pg] = -12345 - pg
                    for off in range(16):
                        s = int(case.token_slots[r][pg * 16 + off])
                        pool[:, 0].flatten(1, 2)[:, s] = float("nan")
                elif pg * 16 < first_seen:  # rows of a page in use, outside the rules
                    for off in range(16):
                        i = pg * 16 + off
                        if rules.prefix[r] <= i < first_seen:
                            s = int(case.token_slots[r][i])
                            pool[:, 0].flatten(1, 2)[:, s] = float("nan")

    mod_check(rules, before=free)


@pytest.mark.gpu
def test_empty_rows_and_prefix_clipping():
    case = W.random_case(11, seq_lens=[4, 3, 50], Hq=8, Hkv=2, D=64, P=16)
    rules = Rules(case, window=5, prefix=[7, -3, 1 << 30])

    def empty(pool, t):
        t["seq_lens"][0] = 0

    o, lse = mod_run(rules, before=empty)
    rules.prefix = np.array([0, 0, 50])
    check(o, lse, rules.want(), rows=[1, 2])
    assert not o[0].any() and torch.isneginf(lse[0]).all()


@pytest.mark.gpu
def test_a_workspace_of_any_contents():
    """The block table's entries past the call's last block must not be taken for blocks: here
    they would name token 0 (and its group's states), which a later block would overwrite."""
    case = W.random_case(20, kind="extend", seq_lens=[3900, 300, 700, 5],
                         chunk_lens=[70, 1, 33, 5], Hq=8, Hkv=2, D=64, P=16)
    mod_check(Rules(case, cap=20.0), stale=[0, 0, 0, 1])


@pytest.mark.gpu
@pytest.mark.parametrize("hint", [0, 16, 5000])
def test_decode_hint_changes_only_the_splits(hint):
    case = W.random_case(12, seq_lens=[2000, 100], Hq=8, Hkv=2, D=64, P=16)
    mod_check(Rules(case, window=700, cap=5.0), hint=hint)


@pytest.mark.gpu
@pytest.mark.parametrize("rule", [dict(alibi=True), dict(cap=3.0, window=9000, prefix=[40, 0])],
                         ids=str)
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 7, 1), (128, 4, 4), (128, 8, 1)])
def test_decode_of_long_rows_merges_many_states(D, Hq, Hkv, rule):
    """Over a hundred splits of one row, a few or one of the others; with and without lse."""
    case = W.random_case(18, seq_lens=[20011, 1, 129, 2500], Hq=Hq, Hkv=Hkv, D=D, P=16)
    rules = Rules(case, **rule)
    o, _ = mod_check(rules)
    same, _ = mod_run(rules, lse=False)
    assert torch.equal(o, same)


@pytest.mark.gpu
@pytest.mark.parametrize("rule", [dict(cap=20.0), dict(alibi=True, prefix=[200, 0]),
                                  dict(cap=2.0, alibi=True, window=900), dict(window=2500)], ids=str)
@pytest.mark.parametrize("D,P", [(64, 16), (128, 7)])
def test_extend_with_blocks_shared_by_groups(D, P, rule):
    """More blocks than groups and long rows: blocks of one and of two query tiles, cut and merged."""
    case = W.random_case(20, kind="extend", seq_lens=[3900, 2000, 300, 1500, 800, 3000],
                         chunk_lens=[150, 130, 20, 3, 140, 129], Hq=16, Hkv=16, D=D, P=P)
    mod_check(Rules(case, **rule))


@pytest.mark.gpu
def test_a_chunked_prompt_equals_the_whole():
    """A prefix-LM prompt in one chunk, and its causal rest in two: the second chunk sees the
    prefix that the first one stored."""
    whole = W.random_case(13, kind="extend", seq_lens=[300], chunk_lens=[300], Hq=8, Hkv=2, D=128,
                          P=16)
    rules = Rules(whole, window=64, prefix=[90], cap=30.0)
    o, lse = mod_check(rules)
    import paged_kv_attention_out_gb300 as pkv
    pool, k, v, q, t = gpu_inputs(whole)
    pkv.pkv_kv_store(pool, 0, k, v, t["out_loc"])
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    parts = []
    for a, b in ((0, 130), (130, 300)):
        qo = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        n = torch.tensor([b], dtype=torch.int32, device="cuda")
        po, pl = nan_outputs(q[a:b])
        pkv.pkv_paged_extend_attn_mod(pool, 0, q[a:b].contiguous(), qo, po, pl, t["page_table"], n,
                                      whole.scale, b, ws, **rules.kwargs())
        parts.append((po, pl))
    check(torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts]), rules.want())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["decode", "extend"])
def test_replay_in_a_graph_follows_new_lengths(kind):
    import paged_kv_attention_out_gb300 as pkv
    kw = dict(chunk_lens=[40, 130]) if kind == "extend" else {}
    case = W.random_case(14, kind=kind, seq_lens=[900, 700], Hq=8, Hkv=2, D=128, P=16, **kw)
    rules = Rules(case, cap=20.0, alibi=True, window=300, prefix=[10, 40])
    pool, k, v, q, t = gpu_inputs(case)
    pkv.pkv_kv_store(pool, 0, k, v, t["out_loc"])
    o, lse = nan_outputs(q)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    args = rules.kwargs()

    def call():
        if kind == "decode":
            pkv.pkv_paged_decode_attn_mod(pool, 0, q, o, lse, t["page_table"], t["seq_lens"],
                                          case.scale, 900, ws, **args)
        else:
            pkv.pkv_paged_extend_attn_mod(pool, 0, q, t["qo_indptr"], o, lse, t["page_table"],
                                          t["seq_lens"], case.scale, 900, ws, **args)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    t["seq_lens"] -= 200
    args["prefix_lens"] += 100
    args["alibi_slopes"] *= 2
    o.fill_(float("nan"))
    g.replay()
    first = o.clone(), lse.clone()
    call()
    assert torch.equal(first[0], o) and torch.equal(first[1], lse)
    assert torch.isfinite(o.float()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2500, 700])
def test_malformed_tables_with_more_blocks_than_tokens(n):
    """Pairs that overlap hold more query blocks than the call has tokens for: the rest is left out
    and nothing is written behind the workspace (blocks that share groups, then one to a group)."""
    import paged_kv_attention_out_gb300 as pkv
    ensure_built()
    case = W.random_case(17, kind="extend", seq_lens=[n] * 5, chunk_lens=[160] + [1] * 4, Hq=16,
                         Hkv=1, D=64, P=16)
    rules = Rules(case, cap=20.0)
    pool, k, v, q, t = gpu_inputs(case)
    pkv.pkv_kv_store(pool, case.layer, k, v, t["out_loc"])
    pkv.pkv_read_device_errors()
    o, lse = nan_outputs(q)
    size = pkv.pkv_extend_mod_workspace_size(5, case.total_q, 16, 1, 64, n, 5 * n)
    ws = torch.full((size + 65536,), 0x5a, dtype=torch.uint8, device="cuda")
    bad = torch.tensor([0, 160, 0, 160, 0, 160], dtype=torch.int32, device="cuda")
    pkv.pkv_paged_extend_attn_mod(pool, case.layer, q, bad, o, lse, t["page_table"], t["seq_lens"],
                                  case.scale, n, ws[:size], max_total_keys_hint=5 * n,
                                  **rules.kwargs())
    assert pkv.pkv_read_device_errors() == 0x8  # malformed pairs
    assert bool((ws[size:] == 0x5a).all())


@pytest.mark.gpu
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 256, 2 ** 31 - 257, 2 ** 30])
@pytest.mark.parametrize("kind", ["decode", "extend", "few"])
def test_a_window_longer_than_every_row(kind, window):
    """Nothing is masked, and no distance leaves 32 bits: the causal answer."""
    seq, chunks = [1, 700, 129, 400], [1, 300, 129, 200]
    if kind == "few":  # the direct form
        seq, chunks = [3900, 1], [40, 1]
    case = W.random_case(9, kind="decode" if kind == "decode" else "extend", seq_lens=seq,
                         chunk_lens=None if kind == "decode" else chunks, Hq=8, Hkv=2, D=64, P=16)
    o, lse = mod_check(Rules(case, cap=20.0, window=window))
    want, lse0 = mod_run(Rules(case, cap=20.0))
    assert torch.equal(o, want) and torch.equal(lse, lse0)


def test_a_window_past_32_bits_is_refused():
    from paged_kv_attention_out_gb300 import binding
    with pytest.raises(ValueError):
        binding._score_mod(0.0, None, 2 ** 32 + 5, None, 1, 1, 0)


def _decode(lib, pool, mod, hint=16):
    return lib.pkv_paged_decode_attn_mod(ctypes.byref(pool), 0, 1 << 20, 1 << 20, None, 64, 8, None,
                                         64, 1, 4, ctypes.c_float(0.125), ctypes.byref(mod), hint,
                                         None, 0, None)


def _extend(lib, pool, mod):
    return lib.pkv_paged_extend_attn_mod(ctypes.byref(pool), 0, 1 << 20, 64, 1 << 20, None, 64, 8,
                                         None, 64, 1, 4, 4, ctypes.c_float(0.125),
                                         ctypes.byref(mod), 16, 0, None, 0, None)


@pytest.mark.parametrize("mod", [(-1.0, None, 0, None), (float("inf"), None, 0, None),
                                 (float("nan"), None, 0, None), (1e-39, None, 0, None),
                                 (0.0, 2, 0, None), (0.0, None, -1, None), (0.0, None, 0, 6)])
@pytest.mark.parametrize("call", [_decode, _extend])
def test_refusals(call, mod):
    ensure_built()
    from paged_kv_attention_out_gb300 import binding
    pool = binding.PkvPool(1 << 30, 1, 10, 16, 2, 64)
    assert call(binding.load(), pool, binding.PkvScoreMod(*mod)) == 1
    assert b"pool" not in binding.load().pkv_last_error()


@pytest.mark.gpu
def test_the_workspace_covers_both_plans_and_a_smaller_one_is_refused():
    import paged_kv_attention_out_gb300 as pkv
    case = W.random_case(15, seq_lens=[5000, 300], Hq=8, Hkv=2, D=64, P=16)
    pool, k, v, q, t = gpu_inputs(case)
    o, lse = nan_outputs(q)
    n = pkv.pkv_decode_mod_workspace_size(2, 8, 2, 64, 5000)
    assert n >= pkv.pkv_decode_workspace_size(2, 8, 2, 64, 5000) > 0
    ws = torch.empty(n - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_paged_decode_attn_mod(pool, 0, q, o, lse, t["page_table"], t["seq_lens"],
                                      case.scale, 5000, ws, soft_cap=5.0)
    assert e.value.status == 3
    assert pkv.pkv_decode_mod_workspace_size(0, 8, 2, 64, 5000) == 0


@pytest.mark.gpu
def test_a_workspace_for_larger_sizes_serves_smaller_ones():
    import paged_kv_attention_out_gb300 as pkv
    decode = lambda b, n, hq=8, hkv=2: pkv.pkv_decode_mod_workspace_size(b, hq, hkv, 64, n)
    extend = lambda b, t, n, k: pkv.pkv_extend_mod_workspace_size(b, t, 8, 1, 64, n, k)
    tree = lambda b, t, n: pkv.pkv_tree_workspace_size(b, 8, 2, 64, t, n)
    grid = [1, 2, 3, 7, 16, 60, 200, 300]
    keys = [1, 128, 129, 1000, 2000, 5000, 40000]
    for a, b in zip(grid, grid[1:]):
        for m, n in zip(keys, keys[1:]):
            assert decode(a, m) <= decode(b, m) <= decode(b, n) and decode(a, m) <= decode(a, n)
            assert decode(a, n) >= pkv.pkv_decode_workspace_size(a, 8, 2, 64, n)
            assert extend(a, 2 * a, m, 100) <= extend(b, 2 * b, m, 100) <= extend(b, 2 * b, n, 5000)
            assert tree(a, 5, m) <= tree(b, 5, m) <= tree(b, 70, n)
    # a batch whose plan differs from that of the larger one, in its workspace
    big = W.random_case(19, seq_lens=[2000] * 4, Hq=32, Hkv=8, D=64, P=16)
    ws = torch.empty(pkv.pkv_decode_mod_workspace_size(4, 32, 8, 64, 2000), dtype=torch.uint8,
                     device="cuda")
    pool, k, v, q, t = gpu_inputs(big)
    pkv.pkv_kv_store(pool, big.layer, k, v, t["out_loc"])
    o, lse = nan_outputs(q)
    want = Rules(big, window=1500).want()
    for b in (1, 2, 3, 4):
        pkv.pkv_paged_decode_attn_mod(pool, big.layer, q[:b], o[:b], lse[:b], t["page_table"][:b],
                                      t["seq_lens"][:b], big.scale, 2000, ws, window=1500)
        check(o[:b], lse[:b], tuple(x[:b] for x in want))
