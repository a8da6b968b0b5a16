"""The calls of a serving step together, as an engine strings them: append (norm, rotation, store),
then attention under the layer's score rules; a drafted tree appended, verified and cut back to its
accepted path. Every result is checked against a dense model of the same steps in 64 bits, with
K and V rounded to bf16 where the cache holds them."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from attn_reference import LSE_TOL, OUT_ROUNDING, P_ROUNDING, SCORES
from helpers import ensure_built
from test_norm_rope import reference, rope_table

pytestmark = pytest.mark.gpu
HQ, HKV, D, P, PAGES, STRIDE = 8, 2, 128, 16, 120, 40


class Engine:
    """A one-layer engine: pool, page rows and the bf16 rows its cache must hold."""

    def __init__(self, requests, seed=0):
        import paged_kv_attention_out_gb300 as pkv
        ensure_built()
        self.pkv, self.g = pkv, torch.Generator(device="cuda").manual_seed(seed)
        self.pool = torch.full((2, 2, PAGES, P, HKV, D), float("nan"), device="cuda").bfloat16()
        order = torch.randperm(PAGES, generator=self.g, device="cuda").int()
        self.rows = order[:requests * STRIDE].view(requests, STRIDE).contiguous()
        self.len = [0] * requests
        self.k = [torch.zeros(0, HKV, D, dtype=torch.float64) for _ in range(requests)]
        self.v = [torch.zeros(0, HKV, D, dtype=torch.float64) for _ in range(requests)]
        self.w = [(1 + torch.randn(D, generator=self.g, device="cuda") / 8).bfloat16()
                  for _ in (0, 1)]
        self.table = rope_table(600, D)
        self.ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def append(self, news, positions):
        """news[r] tokens per request at the given positions: returns the rotated q."""
        n = sum(news)
        qkv = torch.randn(n, (HQ + 2 * HKV) * D, generator=self.g, device="cuda").bfloat16()
        q, k, v = (x.view(n, -1, D) for x in qkv.split([HQ * D, HKV * D, HKV * D], 1))
        pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
        loc = []
        for r, c in enumerate(news):
            i = torch.arange(self.len[r], self.len[r] + c, device="cuda")
            loc.append(self.rows[r].long()[i // P] * P + i % P)
        loc = torch.cat(loc).int()
        q_out = torch.empty(n, HQ, D, dtype=torch.bfloat16, device="cuda")
        self.pkv.pkv_norm_rope_kv_store(self.pool, 1, q, k, v, q_out, pos, loc, self.table,
                                        q_norm=self.w[0], k_norm=self.w[1])
        want_k = reference(k, self.w[1], 1e-6, self.table, pos, False)[0]
        stored = self.pool[0, 1].flatten(0, 1)[loc.long()].double().cpu()
        # (the kernel's own rounding of k is tested elsewhere: the model takes the cache's rows)
        assert ((stored - want_k).abs() <= 2 ** -7 * want_k.abs() + 1e-3).all()
        at = 0
        for r, c in enumerate(news):
            self.k[r] = torch.cat([self.k[r], stored[at:at + c]])
            self.v[r] = torch.cat([self.v[r], v[at:at + c].double().cpu()])
            self.len[r] += c
            at += c
        return q_out

    def lens(self):
        return torch.tensor(self.len, dtype=torch.int32, device="cuda")

    def check(self, q, o, lse, news, seen, rule=lambda s, r, j, h, vis: s):
        q, o, lse = q.double().cpu(), o.double().cpu(), lse.double().cpu()
        t = 0
        for r, c in enumerate(news):
            for j in range(c):
                vis = torch.as_tensor(seen(r, j, self.len[r]))
                for h in range(HQ):
                    k, v = self.k[r][vis, h // 4], self.v[r][vis, h // 4]
                    s = rule(k @ q[t, h] * D ** -0.5, r, j, h, vis)
                    p = torch.softmax(s, 0)
                    want, mag = p @ v, p @ v.abs()
                    tol = (P_ROUNDING + SCORES) * mag + OUT_ROUNDING * want.abs()
                    assert ((o[t, h] - want).abs() <= tol).all(), (r, j, h)
                    assert abs(lse[t, h] - torch.logsumexp(s, 0)) <= LSE_TOL
                t += 1


def test_prompt_decode_and_verified_drafts_of_a_windowed_capped_layer():
    e = Engine(3)
    rules = dict(soft_cap=20.0, window=70)

    def cap(s, r, j, h, vis):
        return 20.0 * torch.tanh(s / 20.0)

    def window(first):
        def seen(r, j, n):
            i, t = np.arange(n), first[r] + j
            return (i <= t) & (t - i < 70)
        return seen

    pkv, scale = e.pkv, D ** -0.5
    # two chunks of prompt per request
    for news in ([130, 17, 90], [40, 1, 75]):
        first = list(e.len)
        q = e.append(news, [p for r, c in enumerate(news) for p in range(e.len[r], e.len[r] + c)])
        o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        qo = torch.tensor(np.cumsum([0] + news), dtype=torch.int32, device="cuda")
        pkv.pkv_paged_extend_attn_mod(e.pool, 1, q, qo, o, lse, e.rows, e.lens(), scale, max(e.len),
                                      e.ws, **rules)
        e.check(q, o, lse, news, window(first), cap)
    # two decode steps
    for _ in range(2):
        first = list(e.len)
        q = e.append([1, 1, 1], list(e.len))
        o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        pkv.pkv_paged_decode_attn_mod(e.pool, 1, q, o, lse, e.rows, e.lens(), scale, 70, e.ws,
                                      **rules)
        e.check(q, o, lse, [1, 1, 1], window(first), cap)
    assert pkv.pkv_read_device_errors() == 0


def test_a_tree_is_verified_and_its_accepted_path_goes_on():
    """Trees of drafts at positions cached + depth; the accepted path is re-appended after the
    cached tokens (cache cut back) and a plain decode step sees exactly it."""
    e = Engine(3, seed=1)
    pkv, scale = e.pkv, D ** -0.5
    news = [150, 1, 64]
    e.append(news, [p for c in news for p in range(c)])
    rng = np.random.default_rng(2)
    for step in range(2):
        drafts = [9, 33, 5]
        parents = [[int(rng.integers(-1, j)) if j else -1 for j in range(c)] for c in drafts]
        depth = []
        for r, c in enumerate(drafts):
            d = []
            for j in range(c):
                d.append(0 if parents[r][j] < 0 else d[parents[r][j]] + 1)
            depth += [e.len[r] + x for x in d]
        cached = list(e.len)
        q = e.append(drafts, depth)
        o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        qo = torch.tensor(np.cumsum([0] + drafts), dtype=torch.int32, device="cuda")
        par = torch.tensor(sum(parents, []), dtype=torch.int32, device="cuda")
        pkv.pkv_paged_tree_attn(e.pool, 1, q, qo, par, o, lse, e.rows, e.lens(), scale, 33,
                                max(e.len), e.ws)

        def seen(r, j, n):
            vis = np.arange(n) < cached[r]
            while j >= 0:
                vis[cached[r] + j] = True
                j = parents[r][j]
            return vis

        e.check(q, o, lse, drafts, seen)
        # the cache goes back to the cached tokens; two accepted ones are stored again, in order
        for r in range(3):
            e.len[r] = cached[r]
            e.k[r], e.v[r] = e.k[r][:cached[r]], e.v[r][:cached[r]]
        e.append([2, 2, 2], [p for r in range(3) for p in (e.len[r], e.len[r] + 1)])
        q = e.append([1, 1, 1], list(e.len))
        o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        pkv.pkv_paged_decode_attn(e.pool, 1, q, o, lse, e.rows, e.lens(), scale, max(e.len), e.ws)
        e.check(q, o, lse, [1, 1, 1], lambda r, j, n: np.ones(n, bool))
    assert pkv.pkv_read_device_errors() == 0


def test_steps_on_a_side_stream_and_in_a_graph_give_the_same():
    """append -> decode under rules, eagerly on another stream and replayed from a graph."""
    e = Engine(3, seed=3)
    pkv, scale = e.pkv, D ** -0.5
    news = [200, 33, 120]
    e.append(news, [p for c in news for p in range(c)])
    n = 3
    qkv = torch.randn(n, (HQ + 2 * HKV) * D, generator=e.g, device="cuda").bfloat16()
    q, k, v = (x.view(n, -1, D) for x in qkv.split([HQ * D, HKV * D, HKV * D], 1))
    pos = e.lens()
    seq = pos + 1
    loc = torch.stack([e.rows[r].long()[e.len[r] // P] * P + e.len[r] % P for r in range(n)]).int()
    q_out = torch.empty(n, HQ, D, dtype=torch.bfloat16, device="cuda")
    slopes = torch.linspace(0.01, 0.5, HQ, device="cuda")
    outs = []

    def step(o, lse):
        pkv.pkv_norm_rope_kv_store(e.pool, 1, q, k, v, q_out, pos, loc, e.table, q_norm=e.w[0],
                                   k_norm=e.w[1])
        pkv.pkv_paged_decode_attn_mod(e.pool, 1, q_out, o, lse, e.rows, seq, scale, 300, e.ws,
                                      alibi_slopes=slopes, soft_cap=10.0)

    for how in ("eager", "stream", "graph"):
        o = torch.full((n, HQ, D), float("nan"), device="cuda").bfloat16()
        lse = torch.empty(n, HQ, device="cuda")
        if how == "eager":
            step(o, lse)
        elif how == "stream":
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step(o, lse)
            torch.cuda.current_stream().wait_stream(side)
        else:
            g = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(g):
                step(o, lse)
            g.replay()
        torch.cuda.synchronize()
        outs.append((o, lse))
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])
