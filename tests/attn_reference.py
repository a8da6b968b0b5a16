"""Attention of paged cases in 64 bits for any set of visible keys and score rule, with the
tolerances of the bf16 kernels.

Tolerance of o. The kernels round each probability to bf16 (at most half a step, 2^-8 of it) and
the result (2^-8 of it); the normaliser is the fp32 sum of the unrounded ones. With
A = sum_i softmax_i |v_i|, which bounds |o|, the first is at most 2^-8 A and the second 2^-8 |o|.
A score is an fp32 sum of D <= 128 products: even if each addition lost a whole 2^-23 of the sum of
magnitudes, which for these N(0, 1) inputs is at most 1.5 D scale = 17, it is off by
128 * 2^-23 * 17 = 2.6e-4 < 2^-11.9; that moves numerator and normaliser by as much, together less
than 2^-10.8 A. lse is off by the score's error and the fp32 logarithm's, below 2^-11 in all; score
rules are smooth (their slope is at most one) and computed in fp32, which adds a few 2^-23 of the
largest term (at most 100: 2^-15)."""
from __future__ import annotations

import numpy as np

from helpers import bits_to_f64, oracle_inputs
from paged_kv_attention_out_gb300 import workloads as W
import oracle

P_ROUNDING = 2.0 ** -8
OUT_ROUNDING = 2.0 ** -8
SCORES = 2.0 ** -10
LSE_TOL = 2.0 ** -11 + 2.0 ** -15


def stored_inputs(case: W.Case):
    """(K rows, V rows) of each request in key order [n, Hkv, D] and q [T, Hq, D], in 64 bits, the
    case's new tokens stored."""
    pool, k, v, q = oracle_inputs(case)
    oracle.kv_store(pool, case.layer, k, v, case.out_loc)
    planes = [pool[c, case.layer].reshape(-1, case.Hkv, case.D) for c in (0, 1)]
    kv = [tuple(bits_to_f64(p[np.asarray(case.token_slots[r], np.int64)[:int(case.seq_lens[r])]])
                for p in planes) for r in range(case.B)]
    return kv, bits_to_f64(q)


def attend(kv, q, qo, scale, visible, rule=None):
    """o, lse and A = sum softmax |v| of every query. visible(r, j, n) -> bool [n] for query j of
    request r; rule(s, r, j, h) -> scores."""
    T, Hq, D = q.shape
    o, mag = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -np.inf)
    for r, (k, v) in enumerate(kv):
        n, hkv = k.shape[0], k.shape[1]
        for j in range(int(qo[r + 1] - qo[r])):
            t = int(qo[r]) + j
            idx = np.flatnonzero(visible(r, j, n))
            if not len(idx):
                continue
            for h in range(Hq):
                kh = h // (Hq // hkv)
                s = scale * (k[idx, kh] @ q[t, h])
                if rule is not None:
                    s = rule(s, r, j, h, idx)
                m = s.max()
                p = np.exp(s - m)
                lse[t, h] = m + np.log(p.sum())
                p /= p.sum()
                o[t, h] = p @ v[idx, kh]
                mag[t, h] = p @ np.abs(v[idx, kh])
    return o, lse, mag


def check(got_o, got_lse, want, rows=None):
    o, lse, mag = want
    got_o = got_o.float().cpu().double().numpy()
    sel = slice(None) if rows is None else rows
    got_o, o, mag = got_o[sel], o[sel], mag[sel]
    assert np.isfinite(got_o).all(), "o: non-finite values"
    tol = (P_ROUNDING + SCORES) * mag + OUT_ROUNDING * np.abs(o) + 1e-30
    over = np.abs(got_o - o) - tol
    assert over.max(initial=-1) <= 0, f"o: {over.max():.3e} past the tolerance at " \
                                      f"{np.unravel_index(over.argmax(), over.shape)}"
    if got_lse is not None:
        got, want_l = got_lse.cpu().double().numpy()[sel], lse[sel]
        empty = np.isneginf(want_l)
        assert np.array_equal(np.isneginf(got), empty), "lse: -inf positions differ"
        err = np.abs(got[~empty] - want_l[~empty])
        assert err.max(initial=0) <= LSE_TOL, f"lse: off by {err.max():.3e}"
