"""Draft-tree calls that share no block need no workspace, as the extend calls of that form."""
from __future__ import annotations

import pytest
import torch

from attn_reference import attend, check, stored_inputs
from helpers import gpu_inputs, nan_outputs
from test_tree import ancestors, tree_case


@pytest.mark.gpu
@pytest.mark.parametrize("cached,drafts,Hq,Hkv", [([512], [8], 32, 8), ([200, 30, 7], [40, 3, 1], 8, 2)])
@pytest.mark.parametrize("room", [None, 1])
def test_a_group_for_each_block_needs_no_workspace(cached, drafts, Hq, Hkv, room):
    import paged_kv_attention_out_gb300 as pkv
    case, parents = tree_case(21, cached, drafts, Hq=Hq, Hkv=Hkv, D=64, P=16)
    pool, k, v, q, t = gpu_inputs(case)
    pkv.pkv_kv_store(pool, case.layer, k, v, t["out_loc"])
    o, lse = nan_outputs(q)
    ws = None if room is None else torch.empty(room, dtype=torch.uint8, device="cuda")
    pkv.pkv_paged_tree_attn(pool, case.layer, q, t["qo_indptr"],
                            torch.as_tensor(parents, device="cuda"), o, lse, t["page_table"],
                            t["seq_lens"], case.scale, case.max_chunk, case.max_seq_len, ws)
    kv, hq = stored_inputs(case)
    check(o, lse, attend(kv, hq, case.qo_indptr, case.scale, ancestors(case, parents)))
