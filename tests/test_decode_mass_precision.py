"""The output of decode with weights (pkv_paged_decode_attn_mass) to the precision of its own
rounding: the probabilities enter the product with the values to more bits than bf16 has.

Inputs for which nothing else rounds: q and keys of -1, 0, 1, so that raw scores are exact,
values of -1 and 1. Tolerance, with sum p |v| / sum p = 1: a probability is the sum of two bf16
terms, the second between 2^-8 and 2^-6.4 of it and rounded by at most 2^-8 of itself: 2^-14.4. A
score in log2 units is at most 64 / 16 log2(e) = 5.8 in magnitude, rounded twice (2^-24 of it
each) and less the maximum once more (2^-24 of 11.6): 2^-20 in all; exp2 adds 2^-22 of its value;
numerator and normaliser are off by as much, together below 2^-18. Fp32 sums: at most 64
sequential steps, each within a product of 16 terms or of a merge, at 2^-23: 2^-17. In all below
2^-14; then half a step of the bf16 result, 2^-8 of it at most. The signs of the values alternate
with the size of the probabilities, so that results are small beside the 2^-8 that probabilities
rounded to bf16 are off by."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from helpers import ensure_built, nan_outputs

BEFORE_ROUNDING, OUT_ROUNDING = 2.0 ** -14, 2.0 ** -8


def make(n, hq, hkv, d, seed):
    """q [hq, d], keys and values [n, hkv, d] in 64 bits; values of dim x alternate by the
    probability of q head x % group."""
    g = np.random.default_rng(seed)
    q = g.integers(-1, 2, (hq, d)).astype(np.float64)
    k = g.integers(-1, 2, (n, hkv, d)).astype(np.float64)
    v = np.empty((n, hkv, d))
    for h in range(hkv):
        for m in range(hq // hkv):
            order = np.argsort(k[:, h] @ q[h * (hq // hkv) + m], kind="stable")
            sign = np.empty(n)
            sign[order] = 1 - 2 * (np.arange(n) % 2)
            v[:, h, m::hq // hkv] = sign[:, None]
    return q, k, v


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (32, 8, 128), (7, 1, 128), (3, 3, 64)])
@pytest.mark.parametrize("lens", [[2, 3, 5, 16, 17, 33], [64, 100, 250], [600, 2500]])
def test_probabilities_keep_their_bits(hq, hkv, d, lens):
    ensure_built()
    import paged_kv_attention_out_gb300 as pkv
    p, scale = 16, 1 / 16
    per_row = -(-max(lens) // p)
    g = torch.Generator().manual_seed(hq)
    table = torch.randperm(len(lens) * per_row, generator=g).int().view(len(lens), per_row)
    pool = torch.full((2, 1, table.numel(), p, hkv, d), float("nan"), dtype=torch.bfloat16)
    qs, rows = [], []
    for r, n in enumerate(lens):
        q, k, v = make(n, hq, hkv, d, seed=n + hq)
        slots = (table[r].long()[:, None] * p + torch.arange(p)).reshape(-1)[:n]
        for c, x in ((0, k), (1, v)):
            pool[c, 0].view(-1, hkv, d)[slots] = torch.tensor(x).bfloat16()
        qs.append(q)
        rows.append((k, v))
    q = torch.tensor(np.stack(qs)).bfloat16().cuda()
    o, lse = nan_outputs(q)
    mass = torch.zeros(len(lens), hkv, max(lens), device="cuda")
    ws = torch.empty(pkv.pkv_decode_mass_workspace_size(len(lens), hq, hkv, d, max(lens)),
                     dtype=torch.uint8, device="cuda")
    pkv.pkv_paged_decode_attn_mass(pool.cuda(), 0, q, o, lse, mass, table.cuda(),
                                   torch.tensor(lens, dtype=torch.int32, device="cuda"), scale,
                                   max(lens), ws)
    assert pkv.pkv_read_device_errors() == 0
    o = o.double().cpu().numpy()
    for r, (k, v) in enumerate(rows):
        for h in range(hq):
            kh = h // (hq // hkv)
            e = np.exp(scale * (k[:, kh] @ qs[r][h]))
            want = e @ v[:, kh] / e.sum()
            over = np.abs(o[r, h] - want) - BEFORE_ROUNDING - OUT_ROUNDING * np.abs(want)
            assert over.max() <= 0, f"{lens[r]} keys, q head {h}: {over.max():.2e} past the tolerance"


@pytest.mark.gpu
def test_infinite_values_stay_infinite():
    """A value of +-inf gives +-inf (not NaN) to what attends it, whatever its probability rounds to."""
    ensure_built()
    import paged_kv_attention_out_gb300 as pkv
    q, k, v = make(300, 8, 2, 64, seed=1)
    pool = torch.zeros(2, 1, 300, 1, 2, 64, dtype=torch.bfloat16)
    pool[0, 0, :, 0] = torch.tensor(k)
    pool[1, 0, :, 0] = torch.tensor(v)
    for i in range(0, 300, 7):
        pool[1, 0, i, 0, 0, i % 64] = float("inf") if i % 64 % 2 else -float("inf")
    top = int(np.argmax(k[:, 1] @ q[5]))  # a probability of one
    pool[1, 0, top, 0, 1, 9] = float("inf")
    q = torch.tensor(q).bfloat16().cuda()[None]
    o, lse = nan_outputs(q)
    ws = torch.empty(pkv.pkv_decode_mass_workspace_size(1, 8, 2, 64, 300), dtype=torch.uint8,
                     device="cuda")
    pkv.pkv_paged_decode_attn_mass(pool.cuda(), 0, q, o, lse, torch.zeros(1, 2, 300, device="cuda"),
                                   torch.arange(300, dtype=torch.int32, device="cuda")[None],
                                   torch.tensor([300], dtype=torch.int32, device="cuda"), 1 / 16,
                                   300, ws)
    o = o[0].cpu()
    assert torch.isfinite(lse).all()
    hit = {i % 64 for i in range(0, 300, 7)}
    for x in range(64):
        want = float("inf") * (1 if x % 2 else -1)
        assert (o[:4, x] == want).all() if x in hit else torch.isfinite(o[:4, x]).all(), x
        assert (o[4:, x] == float("inf")).all() if x == 9 else torch.isfinite(o[4:, x]).all(), x
