"""The weights of a chunk (pkv_paged_extend_mass) are added in an order that does not depend on
which CTA came to an item when: the same bits from every call, alone or beside other work."""
from __future__ import annotations

import pytest
import torch

from helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d,cap", [(16, 4, 64, 0.0), (28, 4, 128, 0.0), (8, 8, 64, 30.0)])
def test_same_bits_beside_other_work(hq, hkv, d, cap):
    ensure_built()
    import paged_kv_attention_out_gb300 as pkv
    g = torch.Generator().manual_seed(d)
    lens = torch.randint(700, 4500, (12,), generator=g).tolist()
    chunks = [min(n, int(c)) for n, c in zip(lens, torch.randint(200, 1300, (12,), generator=g))]
    p = 16
    per_row = -(-max(lens) // p)
    pool = torch.randn(2, 1, 12 * per_row, p, hkv, d, generator=g).bfloat16().cuda()
    table = torch.randperm(12 * per_row, generator=g).int().view(12, per_row).cuda()
    q = torch.randn(sum(chunks), hq, d, generator=g).bfloat16().cuda()
    lse = (6 + torch.randn(sum(chunks), hq, generator=g)).cuda()
    indptr = torch.tensor([0] + chunks).cumsum(0).int().cuda()
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    mass = torch.empty(12, hkv, max(lens), device="cuda")

    def call():
        mass.zero_()
        pkv.pkv_paged_extend_mass(pool, 0, q, indptr, lse, mass, table, seq, d ** -0.5, max(lens),
                                  soft_cap=cap, max_total_keys_hint=sum(lens))
        return mass.clone()

    first = call()
    assert pkv.pkv_read_device_errors() == 0 and torch.isfinite(first).all()
    other, a = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda").bfloat16()
    torch.cuda.synchronize()
    for i in range(30):
        if i % 2:
            with torch.cuda.stream(other):
                for _ in range(1 + i % 5):
                    a @ a
        assert torch.equal(call(), first), i
    torch.cuda.synchronize()
