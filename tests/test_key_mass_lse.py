"""A chunk's lse enters its weights to 24 bits, whatever the lse, the scale and the form of the
call.

With q = 0 every score is exactly zero, so a key's weight from a query is exp(-lse), and what is
off is how the lse came there. As -lse / scale in three bf16 terms beside the product: scale in
log2 units, its reciprocal and the quotient are rounded once each, the terms leave 2^-24 of it,
their fp32 sum is off by 2 x 2^-23, the product with the scale by 2^-24, log2(e) by 2^-24:
2^-20.6 of |lse|, which moves the weight by that much relative to it. exp2 adds 2^-22, the sum of
32 equal weights and the store 5 x 2^-24. (Two terms would leave up to 2^-16 of |lse|.)"""
from __future__ import annotations

import pytest
import torch

from helpers import ensure_built


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [0.125, 0.3, -0.0703, 3e-4])
@pytest.mark.parametrize("kw", [{}, {"num_last": 16}, {"soft_cap": 30.0}])
def test_weights_of_far_lse(d, scale, kw):
    ensure_built()
    import paged_kv_attention_out_gb300 as pkv
    rows, chunk, n, hq, hkv = 40, 16, 150, 4, 2
    g = torch.Generator().manual_seed(d)
    given = (torch.rand(rows, generator=g) * 160 - 80).float()
    pool = torch.randn(2, 1, rows * 10, 16, hkv, d, generator=g).bfloat16().cuda()
    table = torch.randperm(rows * 10, generator=g).int().view(rows, 10).cuda()
    q = torch.zeros(rows * chunk, hq, d, dtype=torch.bfloat16, device="cuda")
    lse = given.repeat_interleave(chunk)[:, None].expand(-1, hq).contiguous().cuda()
    mass = torch.empty(rows, hkv, n, device="cuda")
    indptr, seq = torch.arange(rows + 1) * chunk, torch.full((rows,), n)
    pkv.pkv_paged_extend_mass(pool, 0, q, indptr.int().cuda(), lse, mass, table, seq.int().cuda(),
                              scale, n, accumulate=False, **kw)
    assert pkv.pkv_read_device_errors() == 0
    x = given.double()
    # queries that see a key
    queries = torch.cat([torch.full((n - chunk,), chunk), torch.arange(chunk, 0, -1)])
    want = (-x).exp()[:, None] * (queries * (hq // hkv))
    rel = (mass.double().cpu() - want[:, None]).abs() / want[:, None]
    assert (rel <= (x.abs() * 2 ** -20.6 + 2 ** -21)[:, None, None]).all(), float(
        (rel / (x.abs() * 2 ** -20.6 + 2 ** -21)[:, None, None]).max())
