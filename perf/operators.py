"""The step of a served model around its paged KV cache, as cases that can be timed and compared.

Four operators, each with the plain form that defines it (elementary torch operations in 32 bits) and the call of this
package that computes it:

  append  per-head RMS norm and position rotation of a step's q and k in one pass, k and v appended to the paged cache
  decode  one query per request over its cached keys, scores capped by a tanh, biased by distance or cut to a window
  extend  the same scores for a chunk of queries after a cached prefix (causal, with an optional bidirectional prefix)
  tree    a tree of drafted tokens over the cache: each attends to the cached keys, its ancestors and itself

A case is a dict of plain values; lengths follow from the case, values, page order and trees from the seed.
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------------------------------------------------------- cases

def listed():
    none = dict(cap=0.0, alibi=False, window=0, bidir=0)
    return [
        # One decode step of 64 requests: latency of a single small launch.
        dict(name="append_step_64", op="append", tokens=64, hq=32, hkv=8, d=128, rot=128, interleaved=False, norm=True, page=1),
        # A prefill chunk of 16384 tokens, q/k/v sliced out of the fused projection: bandwidth.
        dict(name="append_prefill_16384", op="append", tokens=16384, hq=32, hkv=8, d=128, rot=128, interleaved=False, norm=True, page=16),
        # An odd number of tokens, half of each head rotated in neighbouring pairs, no norm.
        dict(name="append_partial_1237", op="append", tokens=1237, hq=28, hkv=4, d=64, rot=32, interleaved=True, norm=False, page=16),
        # The smallest decode batch: latency.
        dict(name="decode_cap_small", op="decode", batch=3, most=600, hq=8, hkv=2, d=64, page=1, **{**none, "cap": 30.0}),
        # A sliding-window layer with capped scores over a mixed batch.
        dict(name="decode_window_cap", op="decode", batch=64, most=16384, hq=32, hkv=8, d=128, page=16, **{**none, "cap": 50.0, "window": 4096}),
        # Long rows of a model with a distance bias and no shared heads.
        dict(name="decode_alibi_long", op="decode", batch=8, most=32768, hq=16, hkv=16, d=128, page=16, **{**none, "alibi": True}),
        # A short chunk after a short prefix: latency.
        dict(name="extend_alibi_small", op="extend", batch=2, chunk=48, most=200, hq=8, hkv=8, d=64, page=1, **{**none, "alibi": True}),
        # Chunked prefill of a sliding-window layer with capped scores: arithmetic.
        dict(name="extend_window_cap", op="extend", batch=4, chunk=2048, most=8192, hq=32, hkv=8, d=128, page=16, **{**none, "cap": 50.0, "window": 4096}),
        # Ragged prompts with a bidirectional prefix, seven query heads to a kv head.
        dict(name="extend_prefix_odd", op="extend", batch=6, chunk=701, most=2201, hq=28, hkv=4, d=128, page=16, **{**none, "bidir": 400}),
        # One request verifies eight drafted tokens: latency.
        dict(name="tree_small", op="tree", batch=1, chunk=8, most=520, hq=32, hkv=8, d=128, page=1),
        # A batch verifies trees of up to 64 drafted tokens over long caches: bandwidth.
        dict(name="tree_batch", op="tree", batch=16, chunk=64, most=32768, hq=32, hkv=8, d=128, page=16),
        # Odd trees, odd group, short heads.
        dict(name="tree_odd", op="tree", batch=7, chunk=61, most=2900, hq=28, hkv=4, d=64, page=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "extend", "tree"])
    d = rng.choice([64, 128])
    hq, hkv = rng.choice([(32, 8), (28, 4), (16, 16), (8, 2), (8, 1), (40, 8), (12, 4)])
    c = dict(op=op, hq=hq, hkv=hkv, d=d, page=rng.choice([1, 16, 64, 7]))
    if op == "append":
        c.update(tokens=_log_int(rng, 1, 16000), rot=rng.choice([d, d // 2, 16]), interleaved=rng.random() < 0.5, norm=rng.random() < 0.5)
        return c
    if op != "tree":
        c.update(cap=rng.choice([0.0, 20.0, 50.0]), alibi=rng.random() < 0.4, window=rng.choice([0, 0, 100, 1024, 4096]), bidir=rng.choice([0, 0, 5, 260]))
    if op == "decode":
        c.update(batch=_log_int(rng, 1, 24), most=_log_int(rng, 1, 12000))
    elif op == "extend":
        c.update(batch=_log_int(rng, 1, 4), chunk=_log_int(rng, 1, 1200))
        c.update(most=c["chunk"] + _log_int(rng, 1, 2900) - 1)
    else:
        c.update(batch=_log_int(rng, 1, 16), chunk=_log_int(rng, 1, 128))
        c.update(most=c["chunk"] + _log_int(rng, 1, 12000) - 1)
    return c


def _lengths(case):
    """(new tokens, keys with them) of each request: the longest first, the others spread down to an eighth of it."""
    rng = random.Random("%s/%s" % (case["batch"], case["most"]))
    chunk = [case.get("chunk", 1)] + [_log_int(rng, max(1, case.get("chunk", 1) // 4), case.get("chunk", 1)) for _ in range(case["batch"] - 1)]
    keys = [case["most"]] + [max(c, _log_int(rng, max(1, case["most"] // 8), case["most"])) for c in chunk[1:]]
    return chunk, keys


def _visible(case, t, n):
    """Keys that the query at position t of n sees."""
    lo = max(0, t - case["window"] + 1) if case["window"] else 0
    return (t - lo + 1) + len(range(min(case["bidir"], n), 0, -1)) - len(range(max(0, lo), min(case["bidir"], t + 1)))


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "append":
        n = case["tokens"]
        table = n * case["rot"] * 4 + n * 8 + (4 * d if case["norm"] else 0)
        return {"bytes": 2 * n * (hq + 2 * hkv) * d * 2 + table, "flops": n * (hq + hkv) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    chunk, keys = _lengths(case)
    queries = sum(chunk)
    if case["op"] == "tree":
        # the cached keys, and at least itself among the drafted ones
        pairs, read = sum(c * (n - c + 1) for c, n in zip(chunk, keys)), sum(keys)
    else:
        pairs = read = 0
        for c, n in zip(chunk, keys):
            first = n - c
            pairs += sum(_visible(case, t, n) for t in range(first, n))
            lo = max(0, first - case["window"] + 1) if case["window"] else 0
            read += n - lo + min(case["bidir"], lo)
    pages = -(-read // case["page"])
    return {"bytes": read * 2 * hkv * d * 2 + pages * 4 + 2 * queries * hq * d * 2 + queries * hq * 4, "flops": 4 * d * hq * pairs}


# --------------------------------------------------------------------------------------------------------------- inputs

def _normal(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)


def _rotation(positions, rot):
    """cos and sin of every position's angles, as a model keeps them: [positions, rot] fp32, cosines first."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    s = {"case": case, "layer": 1, "scale": d ** -0.5}
    if case["op"] == "append":
        n = case["tokens"]
        pages = -(-2 * n // page) + 3
        s["pool"] = _normal(gen, 2, 2, pages, page, hkv, d)
        qkv = _normal(gen, n, (hq + 2 * hkv) * d)
        s["q"] = qkv[:, :hq * d].view(n, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(n, hkv, d)
        s["q_out"] = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
        s["q_norm"] = 1 + _normal(gen, d) / 8 if case["norm"] else None
        s["k_norm"] = 1 + _normal(gen, d) / 8 if case["norm"] else None
        s["cos_sin"] = _rotation(32768, case["rot"])
        s["positions"] = torch.randint(0, 32768, (n,), generator=gen, device="cuda", dtype=torch.int32)
        s["out_loc"] = torch.randperm(pages * page, generator=gen, device="cuda")[:n].int()
        return s
    chunk, keys = _lengths(case)
    per_row = -(-max(keys) // page) + 1
    pages = sum(-(-n // page) for n in keys) + 5
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    rows, at = [], 0
    for n in keys:  # each request's pages, then entries that no call may read
        own_pages = -(-n // page)
        rows.append(torch.cat([order[at:at + own_pages], order[:1].expand(per_row - own_pages)]))
        at += own_pages
    s["page_table"] = torch.stack(rows).contiguous()
    s["pool"] = _normal(gen, 2, 2, pages, page, hkv, d)
    s["seq_lens"] = torch.tensor(keys, dtype=torch.int32, device="cuda")
    queries = sum(chunk)
    s["q"] = _normal(gen, queries, hq, d)
    s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty(queries, hq, device="cuda")
    s["max_keys"], s["total_keys"], s["max_chunk"] = max(keys), sum(keys), max(chunk)
    if case["op"] != "decode":
        s["qo_indptr"] = torch.tensor([0] + chunk, device="cuda").cumsum(0).int()
    if case["op"] == "tree":
        # a drafted token's parent is an earlier one, or the last cached token (-1)
        j = torch.cat([torch.arange(c, device="cuda") for c in chunk])
        s["parents"] = ((torch.rand(queries, generator=gen, device="cuda", dtype=torch.float64) * (j + 1)).long() - 1).int()
    else:
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, hq + 1, device="cuda") / hq) if case["alibi"] else None
        s["prefix_lens"] = torch.tensor([min(case["bidir"], n) for n in keys], dtype=torch.int32, device="cuda") if case["bidir"] else None
        if case["window"]:
            s["max_keys"] = min(s["max_keys"], case["window"] + case["bidir"]) if case["op"] == "decode" else s["max_keys"]
    # one scratch buffer for every call of the program: the gathered keys of an extend call, partial states otherwise
    room = 2 * hkv * d * 2 * (sum(keys) + 256 * (len(keys) + 1)) if case["op"] == "extend" else 256 << 20
    s["workspace"] = torch.empty(room + (64 << 20), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------------------ the passes

def run(s):
    if own:
        return _own(s)
    return {"append": _append, "decode": _decode, "extend": _extend, "tree": _tree}[s["case"]["op"]](s)


def _own(s):
    import paged_kv_attention_out_gb300 as pkv
    case = s["case"]
    if case["op"] == "append":
        pkv.pkv_norm_rope_kv_store(s["pool"], s["layer"], s["q"], s["k"], s["v"], s["q_out"], s["positions"], s["out_loc"], s["cos_sin"],
                                   q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6, interleaved=case["interleaved"])
        return {"q": s["q_out"], "pool": s["pool"]}
    if case["op"] == "decode":
        pkv.pkv_paged_decode_attn_mod(s["pool"], s["layer"], s["q"], s["o"], s["lse"], s["page_table"], s["seq_lens"], s["scale"], s["max_keys"], s["workspace"],
                                      soft_cap=case["cap"], alibi_slopes=s["slopes"], window=case["window"], prefix_lens=s["prefix_lens"])
    elif case["op"] == "extend":
        pkv.pkv_paged_extend_attn_mod(s["pool"], s["layer"], s["q"], s["qo_indptr"], s["o"], s["lse"], s["page_table"], s["seq_lens"], s["scale"], s["max_keys"], s["workspace"],
                                      soft_cap=case["cap"], alibi_slopes=s["slopes"], window=case["window"], prefix_lens=s["prefix_lens"], max_total_keys_hint=s["total_keys"])
    else:
        pkv.pkv_paged_tree_attn(s["pool"], s["layer"], s["q"], s["qo_indptr"], s["parents"], s["o"], s["lse"], s["page_table"], s["seq_lens"], s["scale"],
                                s["max_chunk"], s["max_keys"], s["workspace"])
    return {"o": s["o"], "lse": s["lse"]}


def _normed(x, weight):
    x = x.float()
    return x if weight is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()


def _rotated(x, table, interleaved):
    """x [tokens, heads, d], its first table.shape[1] dims turned by each token's angles."""
    half = table.shape[1] // 2
    cos, sin = table[:, None, :half], table[:, None, half:]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    lo, hi = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([lo, hi], -1).flatten(-2) if interleaved else torch.cat([lo, hi], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _append(s):
    inter, slots = s["case"]["interleaved"], s["out_loc"].long()
    table = s["cos_sin"][s["positions"].long()]
    q = _rotated(_normed(s["q"], s["q_norm"]), table, inter).bfloat16()
    k = _rotated(_normed(s["k"], s["k_norm"]), table, inter).bfloat16()
    s["pool"][0, s["layer"]].flatten(0, 1)[slots] = k
    s["pool"][1, s["layer"]].flatten(0, 1)[slots] = s["v"]
    return {"q": q, "pool": s["pool"]}


def _cached(s):
    """Every request's keys and values in order, padded to the longest: [batch, hkv, keys, d] fp32."""
    page = s["case"]["page"]
    i = torch.arange(int(s["page_table"].shape[1] * page), device="cuda")
    i = i[:max(_lengths(s["case"])[1])]
    slot = s["page_table"].long()[:, i // page] * page + i % page
    return tuple(s["pool"][c, s["layer"]].flatten(0, 1)[slot].transpose(1, 2).float() for c in (0, 1))


def _attend(q, k, v, seen, scale, bias=None, cap=0.0):
    """q [batch, queries, hq, d]; k, v [batch, hkv, keys, d]; seen [batch, queries, keys]; bias: None, or slopes [hq]
    and distances [batch, queries, keys] whose product is taken off the scores. Returns o and lse."""
    batch, n, hq, d = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    rows = q.float().view(batch, n, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, g * n, d)
    x = (rows @ k.transpose(2, 3)).view(batch, hkv, g, n, -1) * scale
    if cap:
        x = cap * torch.tanh(x / cap)
    if bias is not None:
        x = x - bias[0].view(1, hkv, g, 1, 1) * bias[1][:, None, None]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    o = (e.view(batch, hkv, g * n, -1) @ v).view(batch, hkv, g, n, d) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total))[..., 0]
    return o.permute(0, 3, 1, 2, 4).reshape(batch, n, hq, d), lse.permute(0, 3, 1, 2).reshape(batch, n, hq)


def _masked(s, q, t):
    """Attention of the padded queries q at positions t [batch, queries] under the case's score rules."""
    case = s["case"]
    k, v = _cached(s)
    i = torch.arange(k.shape[2], device="cuda")
    seen = i <= t[..., None]
    if case["window"]:
        seen &= i > t[..., None] - case["window"]
    if s["prefix_lens"] is not None:
        seen = seen | (i < s["prefix_lens"].long()[:, None, None])
    seen &= i < s["seq_lens"].long()[:, None, None]
    bias = None if s["slopes"] is None else (s["slopes"], (t[..., None] - i).abs().float())
    return _attend(q, k, v, seen, s["scale"], bias, case["cap"])


def _decode(s):
    o, lse = _masked(s, s["q"][:, None], s["seq_lens"].long()[:, None] - 1)
    return {"o": o[:, 0].bfloat16(), "lse": lse[:, 0]}


def _padded(s):
    """Where each query goes in [batch, longest chunk], and the queries there."""
    start = s["qo_indptr"].long()
    token = torch.arange(s["q"].shape[0], device="cuda")
    request = torch.searchsorted(start, token, right=True) - 1
    j = token - start[request]
    q = s["q"].new_zeros(start.shape[0] - 1, s["max_chunk"], *s["q"].shape[1:])
    q[request, j] = s["q"]
    return request, j, q


def _extend(s):
    request, j, q = _padded(s)
    first = s["seq_lens"].long() - s["qo_indptr"].long().diff()
    o, lse = _masked(s, q, first[:, None] + torch.arange(s["max_chunk"], device="cuda"))
    return {"o": o[request, j].bfloat16(), "lse": lse[request, j]}


def _tree(s):
    request, j, q = _padded(s)
    n = s["max_chunk"]
    first = s["seq_lens"].long() - s["qo_indptr"].long().diff()
    # ancestor-or-self by repeated squaring of "self or parent"; column n takes the roots' -1
    kin = torch.zeros(q.shape[0], n, n + 1, device="cuda")
    kin[:, range(n), range(n)] = 1
    kin[request, j, s["parents"].long() % (n + 1)] = 1
    kin = kin[..., :n]
    for _ in range(max(1, (n - 1).bit_length())):
        kin = (kin @ kin > 0).float()
    k, v = _cached(s)
    i = torch.arange(k.shape[2], device="cuda")
    drafted = i - first[:, None]  # index among the drafted tokens, negative for cached ones
    at = drafted.clamp(0, n - 1)[:, None].expand(-1, n, -1)
    seen = (drafted < 0)[:, None] | (kin.gather(2, at) > 0) & (drafted < n)[:, None]
    seen &= i < s["seq_lens"].long()[:, None, None]
    o, lse = _attend(q, k, v, seen, s["scale"])
    return {"o": o[request, j].bfloat16(), "lse": lse[request, j]}


# ------------------------------------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The definition in 64 bits, token by token or request by request."""
    s = prepare(case, seed)
    pool = s["pool"]
    if case["op"] == "append":
        pos = s["positions"].long()
        half = case["rot"] // 2
        pair = [(2 * m, 2 * m + 1) if case["interleaved"] else (m, m + half) for m in range(half)]
        first, second = [p[0] for p in pair], [p[1] for p in pair]
        turn = torch.complex(s["cos_sin"][pos, :half].double(), s["cos_sin"][pos, half:].double())[:, None]

        def place(x, w):
            x = x.double()
            if w is not None:
                x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * w.double()
            z = torch.complex(x[..., first], x[..., second]) * turn
            y = x.clone()
            y[..., first], y[..., second] = z.real, z.imag
            return y

        want = pool.double()
        want[0, 1].view(-1, case["hkv"], case["d"]).index_copy_(0, s["out_loc"].long(), place(s["k"], s["k_norm"]))
        want[1, 1].view(-1, case["hkv"], case["d"]).index_copy_(0, s["out_loc"].long(), s["v"].double())
        return {"q": place(s["q"], s["q_norm"]), "pool": want}
    o, lse = s["q"].double() * 0, s["lse"].double() * 0
    chunk, keys = _lengths(case)
    at = 0
    for r, (c, n) in enumerate(zip(chunk, keys)):
        slot = [int(p) * case["page"] + x for p in s["page_table"][r].tolist() for x in range(case["page"])][:n]
        slot = torch.tensor(slot, device="cuda")
        k, v = (pool[x, 1].reshape(-1, case["hkv"], case["d"])[slot].double() for x in (0, 1))
        t = torch.arange(n - c, n, device="cuda")[:, None]
        i = torch.arange(n, device="cuda")[None]
        if case["op"] == "tree":
            up = s["parents"][at:at + c].tolist()
            hide = (i >= n - c).repeat(c, 1)
            for x in range(c):
                y = x
                while y >= 0:
                    hide[x, n - c + y] = False
                    y = up[y]
        else:
            hide = i > t
            if case["window"]:
                hide = hide | (t - i >= case["window"])
            hide = hide & (i >= case["bidir"])
        for h in range(case["hq"]):
            kv = h * case["hkv"] // case["hq"]
            x = torch.einsum("qd,kd->qk", s["q"][at:at + c, h].double(), k[:, kv]) * s["scale"]
            if case.get("cap"):
                x = case["cap"] * torch.tanh(x / case["cap"])
            if case.get("alibi"):
                x = x - s["slopes"][h].double() * (t - i).abs()
            x = x.masked_fill(hide, -math.inf)
            lse[at:at + c, h] = torch.logsumexp(x, 1)
            o[at:at + c, h] = torch.einsum("qk,kd->qd", torch.exp(x - lse[at:at + c, h, None]), v[:, kv])
        at += c
    return {"o": o, "lse": lse}
