"""Scores that are NaN or infinite in decode with weights (pkv_paged_decode_attn_mass): a q head
with a score that is NaN or +inf has NaN for its lse and its output and gives NaN to every key of
the row; -inf is no weight."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from helpers import ensure_built, nan_outputs
from mass_reference import check_mass, received, weights

pytestmark = pytest.mark.gpu


def run(lens, hq=8, hkv=2, d=64, change=lambda k, q: None, cap=0.0):
    """Keys and queries N(0, 1), changed; every output, and (key_mass before, keys, q)."""
    ensure_built()
    import paged_kv_attention_out_gb300 as pkv
    g = torch.Generator().manual_seed(len(lens))
    B, most = len(lens), max(lens)
    k = torch.randn(B, most, hkv, d, generator=g).bfloat16()
    q = torch.randn(B, hq, d, generator=g).bfloat16()
    change(k, q)
    v = torch.randn(k.shape, generator=g).bfloat16()
    pool = torch.stack([k, v]).view(2, 1, B * most, 1, hkv, d)
    table = torch.arange(B * most, dtype=torch.int32).view(B, most).cuda()
    mass = torch.rand(B, hkv, most + 5, generator=g).cuda()
    before = mass.clone()
    o, lse = nan_outputs(q.cuda())
    o.zero_(), lse.zero_()
    ws = torch.empty(pkv.pkv_decode_mass_workspace_size(B, hq, hkv, d, most), dtype=torch.uint8,
                     device="cuda")
    pkv.pkv_paged_decode_attn_mass(pool.cuda(), 0, q.cuda(), o, lse, mass, table,
                                   torch.tensor(lens, dtype=torch.int32, device="cuda"), d ** -0.5,
                                   most, ws, soft_cap=cap)
    assert pkv.pkv_read_device_errors() == 0
    return o.cpu(), lse.cpu(), mass.cpu(), before.cpu(), k.double().numpy(), q.double().numpy()


# one split, a cluster, and many states merged by a warp or a CTA a head
LENS = [[40], [700, 300], [900, 5000] + [3000] * 30, [60000]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_score_that_is_no_number(lens, value):
    key = lens[0] * 2 // 3

    def change(k, q):
        k[0, key, 1] = 0
        k[0, key, 1, 3] = value
        q[0, :, 3] = 1.0  # (+inf or NaN for every head of the group)

    o, lse, mass, before, k, q = run(lens, change=change)
    for b, n in enumerate(lens):
        w, want = weights(np.nan_to_num(k[b, :n], nan=0, posinf=0), q[b:b + 1], n - 1, 0.125)
        for h in range(2):
            mine = slice(4 * h, 4 * h + 4)
            if b == 0 and h == 1:
                assert torch.isnan(lse[b, mine]).all() and torch.isnan(o[b, mine]).all()
                assert torch.isnan(mass[b, h, :n]).all()
                assert torch.equal(mass[b, h, n:], before[b, h, n:])
                continue
            assert torch.isfinite(o[b, mine]).all()
            assert np.abs(lse[b, mine].double().numpy() - want[0, mine]).max() <= 2.0 ** -10
            had = before[b, h:h + 1, :n].double().numpy()
            had[:, n - 1] = 0
            check_mass(mass[b, h:h + 1, :n].double().numpy(), had, received(w[:, mine], 1))


@pytest.mark.parametrize("lens", LENS)
def test_scores_of_minus_infinity_are_no_weight(lens):
    def change(k, q):
        k[:, 1::3] = 0
        k[:, 1::3, :, 3] = float("inf")
        q[:, :, 3] = -1.0
        if lens[0] == 40:  # a row whose every score is -inf
            k[0, :, 0] = 0
            k[0, :, 0, 3] = float("inf")

    o, lse, mass, before, k, q = run(lens, change=change)
    finite = np.nan_to_num(k, posinf=4e6)  # exp(-5e5) = 0
    for b, n in enumerate(lens):
        w, want = weights(finite[b, :n], q[b:b + 1], n - 1, 0.125)
        for h in range(2):
            mine = slice(4 * h, 4 * h + 4)
            had = before[b, h:h + 1, :n].double().numpy()
            had[:, n - 1] = 0
            got = mass[b, h:h + 1, :n].double().numpy()
            if lens[0] == 40 and h == 0:
                assert (lse[b, mine] == -float("inf")).all() and (o[b, mine] == 0).all()
                assert np.array_equal(got, had)
                continue
            assert np.abs(lse[b, mine].double().numpy() - want[0, mine]).max() <= 2.0 ** -10
            assert torch.isfinite(o[b, mine]).all()
            check_mass(got, had, received(w[:, mine], 1))


def test_under_a_cap_only_nan_is_no_number():
    """The cap takes infinite scores to itself."""
    def change(k, q):
        k[0, 7, 1] = 0
        k[0, 7, 1, 3] = float("inf")
        k[0, 9, 0, 5] = float("nan")
        q[0, :, 3] = 1.0

    o, lse, mass, before, k, q = run([200], change=change, cap=20.0)
    assert torch.isnan(lse[0, :4]).all() and torch.isnan(mass[0, 0, :200]).all()
    finite = np.nan_to_num(k, nan=0, posinf=4e6)
    w, want = weights(finite[0, :200], q, 199, 0.125, 20.0)
    assert np.abs(lse[0, 4:].double().numpy() - want[0, 4:]).max() <= 2.0 ** -10
    had = before[0, 1:, :200].double().numpy()
    had[:, 199] = 0
    check_mass(mass[0, 1:, :200].double().numpy(), had, received(w[:, 4:], 1))
