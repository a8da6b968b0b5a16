"""The hint of decode with weights (pkv_paged_decode_attn_mass) bounds the rows whose weights are
added to the key."""
from __future__ import annotations

import pytest
import torch

from test_key_mass import case_on_gpu, decode, mass_buffer
from paged_kv_attention_out_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,hint", [([105, 100, 90], 100), ([17, 16, 15], 15),
                                       ([1009, 1008, 1007], 1007), ([2, 1], 1)])
def test_rows_just_past_the_hint_are_flagged(lens, hint):
    """A hint is a bound to the key, in one launch and in two."""
    for copies in (1, 60):
        case = W.random_case(8, seq_lens=lens * copies, Hq=8, Hkv=2, D=64, P=16)
        pkv, pool, q, t = case_on_gpu(case)
        mass = mass_buffer(case)
        before = mass.clone()
        o, lse = decode(pkv, case, pool, q, t, mass, hint=hint)
        assert pkv.pkv_read_device_errors() == 0x4
        long = torch.tensor([n > hint for n in lens * copies], device="cuda")
        assert torch.equal(mass[long], before[long])
        assert torch.isfinite(lse).all()  # all get their attention
        good = mass_buffer(case)
        o2, lse2 = decode(pkv, case, pool, q, t, good)
        assert (o - o2).abs().max() < 2 ** -5 and (lse - lse2).abs().max() < 2 ** -10
        assert torch.allclose(mass[~long], good[~long], rtol=2 ** -10, atol=0)
        assert not torch.equal(mass[~long], before[~long])
