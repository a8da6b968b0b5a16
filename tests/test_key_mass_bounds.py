"""Offsets past 32 bits into the scores that decode with weights (pkv_paged_decode_attn_mass) keeps
in its workspace."""
from __future__ import annotations

import math

import pytest
import torch

from attn_reference import LSE_TOL
from helpers import ensure_built, nan_outputs
from test_key_mass import case_on_gpu, decode, mass_buffer
from paged_kv_attention_out_gb300 import workloads as W

pytestmark = pytest.mark.gpu


def test_scores_of_a_batch_past_32_bits():
    """2.7e9 scores in the workspace: the last request has the bits of the first, whose pages and q
    it shares."""
    lens = [300, 5, 77, 260] * 10
    lens[-1] = lens[0]
    case = W.random_case(11, seq_lens=lens, Hq=32, Hkv=8, D=64, P=16)
    pkv, pool, q, t = case_on_gpu(case)
    t["page_table"][-1] = t["page_table"][0]
    q[-1] = q[0]
    mass = mass_buffer(case)
    mass[-1] = mass[0]
    before = mass.clone()
    hint = 1 << 21
    ws = torch.empty(pkv.pkv_decode_mass_workspace_size(case.B, 32, 8, 64, hint), dtype=torch.uint8,
                     device="cuda")
    assert ws.numel() > 4 * 2 ** 31
    o, lse = nan_outputs(q)
    wide = torch.zeros(case.B, hint // 16 + 1, dtype=torch.int32, device="cuda")
    wide[:, :t["page_table"].shape[1]] = t["page_table"]
    pkv.pkv_paged_decode_attn_mass(pool, case.layer, q, o, lse, mass, wide, t["seq_lens"], case.scale,
                                   hint, ws)
    assert pkv.pkv_read_device_errors() == 0
    for x in (o, lse, mass):
        assert torch.equal(x[0], x[-1])
    del ws
    small = before.clone()
    o2, lse2 = decode(pkv, case, pool, q, t, small)
    assert (lse - lse2).abs().max() <= 2 * LSE_TOL
    assert torch.allclose(mass, small, rtol=2 ** -9, atol=0) and not torch.equal(mass, before)


def test_scores_of_a_row_past_32_bits():
    """A row of more than 2^28 keys and eight q heads: 2^31 scores and more. Every table entry is
    the same page, so weights repeat with its size."""
    ensure_built()
    import paged_kv_attention_out_gb300 as pkv
    page, n, hq, d = 65536, 2 ** 28 + 5000, 8, 64
    g = torch.Generator().manual_seed(2)
    pool = torch.randn(2, 1, 1, page, 1, d, generator=g).bfloat16().cuda()
    q = torch.randn(1, hq, d, generator=g).bfloat16().cuda()
    table = torch.zeros(1, -(-n // page), dtype=torch.int32, device="cuda")
    o, lse = nan_outputs(q)
    mass = torch.zeros(1, 1, n + 3, device="cuda")
    ws = torch.empty(pkv.pkv_decode_mass_workspace_size(1, hq, 1, d, n), dtype=torch.uint8,
                     device="cuda")
    pkv.pkv_paged_decode_attn_mass(pool, 0, q, o, lse, mass, table,
                                   torch.tensor([n], dtype=torch.int32, device="cuda"), d ** -0.5, n,
                                   ws)
    assert pkv.pkv_read_device_errors() == 0
    s = (q[0].double() @ pool[0, 0, 0, :, 0].double().T) * d ** -0.5  # [hq, page]
    e, v = s.exp(), pool[1, 0, 0, :, 0].double()
    full, rest = divmod(n, page)
    total = full * e.sum(1) + e[:, :rest].sum(1)
    assert (lse[0].double() - total.log()).abs().max() <= LSE_TOL
    want_o = (full * (e @ v) + e[:, :rest] @ v[:rest]) / total[:, None]
    mag = (full * (e @ v.abs()) + e[:, :rest] @ v[:rest].abs()) / total[:, None]
    # (bf16 probabilities would be allowed as well)
    tol = (2 ** -8 + 2 ** -10) * mag + 2 ** -8 * want_o.abs()
    assert ((o[0].double() - want_o).abs() <= tol).all()
    # a weight is off by its score's and the lse's error (mass_reference), the lse also by fp32 sums
    # of at most 2^11 sequential terms a warp and of 2^12 states: 2^-12 each at worst
    want = (e / total[:, None]).sum(0)
    got = mass[0, 0, :full * page].view(full, page)
    for at in range(0, full, 256):
        assert ((got[at:at + 256].double() - want).abs() <= 2 ** -10 * want).all(), at
    last = mass[0, 0, full * page:n].double()
    assert ((last - want[:rest]).abs() <= 2 ** -10 * want[:rest]).all()
    assert (mass[0, 0, n:] == 0).all()
    assert math.isclose(float(mass.double().sum()), hq, rel_tol=2 ** -10)
