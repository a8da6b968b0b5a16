"""Score rules at the ends of their ranges: scores from far below a soft cap to far past it in one
tile, caps of any size, distance slopes that are steep, zero, negative or mixed within a kv head.

The tolerance follows each score's own size. A score q.k is an fp32 sum of D products, off by at
most D 2^-23 of the sum of their magnitudes; a cap (slope at most one) adds a relative 2^-20 of the
capped score; a bias is two fp32 terms of at most slope * (distance + 256), a few 2^-24 of each; the
exponential's argument and value, and a rounding of the row's reference, are at most 2^-18 and
2^-22 of the row's largest score. With e_i the sum of these for key i, its weight is off by a factor
of at most exp(e_i): with w_i = exp(e_i) - 1 and W = sum p_i w_i < 1 the quotient is off by at most
(sum p_i w_i |v_i| + |o| W) / (1 - W). On top, each probability and the result are rounded to bf16
(2^-8), and the fp32 sum of n probabilities is off by at most n 2^-24."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from attn_reference import stored_inputs
from helpers import ensure_built, gpu_inputs
from paged_kv_attention_out_gb300 import workloads as W
from test_score_rules import Rules, mod_run


def case_of(form, seed, D=128, Hq=8, Hkv=2, P=16):
    if form == "decode":
        return W.random_case(seed, seq_lens=[900, 130, 2500], Hq=Hq, Hkv=Hkv, D=D, P=P)
    if form == "direct":  # few query tiles over longer rows
        seqs, chunks = [1100, 300, 2], [37, 9, 2]
    elif form == "shared":  # blocks cut over groups of CTAs
        seqs, chunks = [3000, 600], [20, 3]
    else:  # gathered: more requests than the direct form takes
        seqs, chunks = [900, 300] + [6] * 260, [129, 20] + [2] * 260
    return W.random_case(seed, kind="extend", seq_lens=seqs, chunk_lens=chunks, Hq=Hq, Hkv=Hkv,
                         D=D, P=P)


def check_ranges(rules, factors=None, spikes=None, scale=None):
    """Runs the call with q rows scaled by factors [T, Hq] and the keys spikes[r] = {key: factor}
    of request r scaled (powers of two: exact), and compares it with the definition in 64 bits."""
    import paged_kv_attention_out_gb300 as pkv
    ensure_built()
    case = rules.case
    scale = case.scale if scale is None else scale
    kv, q = stored_inputs(case)
    pool, k, v, gq, t = gpu_inputs(case)
    if factors is not None:
        q = q * factors[:, :, None]
        gq = (gq.float() * torch.as_tensor(factors, dtype=torch.float32).cuda()[:, :, None])
        gq = gq.bfloat16()
    assert torch.equal(gq.double().cpu(), torch.as_tensor(q))

    def spike(pool, t):
        rows = pool[0, case.layer].flatten(0, 1)
        for r, keys in (spikes or {}).items():
            for i, f in keys.items():
                rows[int(case.token_slots[r][i])] *= f
                kv[r][0][i] *= f

    pkv.pkv_read_device_errors()
    o, lse = mod_run(rules, inputs=(pool, k, v, gq, t), scale=scale, before=spike)
    assert pkv.pkv_read_device_errors() == 0
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(o).all() and np.isfinite(lse).all()
    qo = np.arange(case.B + 1) if case.kind == "decode" else case.qo_indptr
    g = case.Hq // case.Hkv
    worst = 0.0
    for r, (kk, vv) in enumerate(kv):
        n = kk.shape[0]
        for j in range(int(qo[r + 1] - qo[r])):
            tok = int(qo[r]) + j
            idx = np.flatnonzero(rules.visible(r, j, n))
            dist = np.abs(rules.first(r) + j - idx)
            for h in range(case.Hq):
                x, y = kk[idx, h // g], vv[idx, h // g]
                s = scale * (x @ q[tok, h])
                e = case.D * 2.0 ** -23 * abs(scale) * (np.abs(x) @ np.abs(q[tok, h]))
                if rules.cap:
                    s = rules.cap * np.tanh(s / rules.cap)
                    e += 2.0 ** -20 * np.abs(s)
                if rules.slopes is not None:
                    s = s - float(rules.slopes[h]) * dist
                    e += 2.0 ** -22 * abs(float(rules.slopes[h])) * (dist + 256)
                e += 2.0 ** -18 + 2.0 ** -22 * np.abs(s).max()
                p = np.exp(s - s.max())
                want_lse = s.max() + np.log(p.sum())
                p /= p.sum()
                w = np.expm1(e)
                big_w = float(p @ w)
                sums = len(idx) * 2.0 ** -24
                want = p @ y
                if big_w < 1:
                    tol = (2.0 ** -8 + sums) * (p @ np.abs(y)) + 2.0 ** -8 * np.abs(want) + 1e-30
                    tol += ((p * w) @ np.abs(y) + np.abs(want) * big_w) / (1 - big_w)
                    worst = max(worst, float((np.abs(o[tok, h] - want) / tol).max()))
                    lse_tol = -np.log1p(-big_w) + sums + 2.0 ** -20 * abs(want_lse)
                    worst = max(worst, float(abs(lse[tok, h] - want_lse) / lse_tol))
    assert worst <= 1, f"{worst:.2f} times the tolerance"


FORMS = ["decode", "direct", "shared", "gathered"]


def some_rows(case, large, seed):
    """Nine rows in ten as they are, the others times one of `large`."""
    rng = np.random.default_rng(seed)
    T = case.B if case.kind == "decode" else case.total_q
    f = rng.choice(np.asarray(large, float), size=(T, case.Hq))
    return np.where(rng.random((T, case.Hq)) < 0.9, 1.0, f)


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("cap,large", [(30.0, [4, 8, 64]), (50.0, [8]), (50.0, [2, 8, 64]),
                                       (1e3, [8, 64, 1024]), (1e4, [8, 64]), (1e4, [8, 2048]),
                                       (1e6, [8, 64]), (1e8, [8, 64]), (1e30, [8])], ids=str)
def test_caps_of_any_size_with_scores_of_any_size(form, cap, large):
    case = case_of(form, 31)
    check_ranges(Rules(case, cap=cap), some_rows(case, large, 1))


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rule", [dict(cap=1e4, window=200), dict(cap=1e5, alibi=True),
                                  dict(cap=50.0, alibi=True, window=300)], ids=str)
@pytest.mark.parametrize("scale", [None, -0.125])
def test_large_scores_under_a_cap_and_other_rules(form, rule, scale):
    case = case_of(form, 32, D=64, P=7)
    check_ranges(Rules(case, **rule), some_rows(case, [8, 16], 2), scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("cap", [50.0, 1e4, 1e6])
def test_one_key_with_large_scores_among_small_ones(form, cap):
    """Its scores are large and of either sign; where they are negative, the others decide."""
    case = case_of(form, 33)
    check_ranges(Rules(case, cap=cap), spikes={0: {5: 64.0, 700: 16.0}, 1: {100: 64.0}})


SLOPES = {"steep": [2.0, 8.0], "zero": [0.0], "negative": [-0.05], "steep negative": [-2.5],
          "mixed": [0.0, 2.0, -0.05, 0.01], "border": [1.0285, 1.0287, -1.0287, -1.0285]}


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("slopes", list(SLOPES.values()), ids=list(SLOPES))
@pytest.mark.parametrize("rule", [{}, dict(cap=20.0), dict(window=300, prefix=[200, 40])], ids=str)
def test_slopes_of_any_size_and_sign(form, slopes, rule):
    """Steep ones (past what a bound of 32 columns may be off), none, ones that favour far keys."""
    case = case_of(form, 34)
    rules = Rules(case, alibi=True, **rule)
    rules.slopes = np.resize(np.asarray(slopes, np.float32), case.Hq)
    check_ranges(rules)


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("scale,cap", [(1e30, 1e26), (-3e37, 1e32), (1e-30, 1e-30)])
def test_scales_at_the_ends_of_their_range_under_a_cap(form, scale, cap):
    """A request whose q is zero scores zero: the mean of its visible values, whatever the scale."""
    ensure_built()
    case = case_of(form, 35)
    rules = Rules(case, cap=cap)
    pool, k, v, q, t = gpu_inputs(case)
    tokens = 1 if case.kind == "decode" else int(case.qo_indptr[1])
    q[:tokens] = 0
    o, lse = mod_run(rules, inputs=(pool, k, v, q, t), scale=scale)
    v, g = stored_inputs(case)[0][0][1], case.Hq // case.Hkv
    for j in range(tokens):
        n = rules.visible(0, j, v.shape[0]).sum()
        want, mag = (np.repeat(x[:n].mean(0), g, 0) for x in (v, np.abs(v)))
        sums = n * 2.0 ** -24
        tol = (2.0 ** -8 + sums) * mag + 2.0 ** -8 * np.abs(want)
        assert (np.abs(o[j].double().cpu().numpy() - want) <= tol).all()
        assert (np.abs(lse[j].double().cpu().numpy() - np.log(n)) <= 2.0 ** -18 + sums).all()
