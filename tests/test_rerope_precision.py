"""Re-rotation (pkv_kv_rerope) where the two products of a pair cancel, so that bf16 rounding hides
nothing.

Tolerance: sine and cosine are off by 2^-23.2 at most, the angle (cut to 2^-32 of a turn, from a
fraction kept to 2^-52 of a frequency and 2^-64) by 2^-28, so the turned value by 2^0.5 (2^-23.2 +
2^-28) of the pair's radius R; the product with the factor, the products with a and b and their sum
add 4 x 2^-24 R: 2^-21.28 R in all. Where positions differ by kv head the hardware's sine and cosine
are used, with the bound of test_rerope. Then half a bf16 step of the value, 2^-8 of it at most. a
and b are the bf16 numbers, of 2^14 pairs, that bring the value nearest to zero: below 2^-13 R
mostly."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from test_rerope import FP32_PART, HALF_BF16, freqs, make

ONE_POSITION = 2.0 ** -21.28


@pytest.mark.gpu
@pytest.mark.parametrize("by_head", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_values_that_cancel(interleaved, by_head):
    import paged_kv_attention_out_gb300 as pkv
    n, rot, hkv, p = 300, 128, 2, 16
    f = freqs(rot)
    g = np.random.default_rng(2)
    pos = g.integers(1, 5000, (1, hkv if by_head else 1, n))
    pool, table = make([n], hkv=hkv, d=128, p=p)
    slots = (table[0].cpu().long()[:, None] * p + torch.arange(p)).reshape(-1)[:n]
    mantissas = 1 + np.arange(128) / 128
    a, b = (x.ravel() for x in np.meshgrid(mantissas, mantissas))
    order = np.argsort(b / a)
    a, b = a[order], b[order]
    want = np.empty((n, hkv, rot // 2, 2))
    radius = np.empty((n, hkv, rot // 2))
    x = np.empty((n, hkv, rot // 2, 2))
    for h in range(hkv):
        angle = np.outer(pos[0, h % pos.shape[1]], f.double().numpy())
        c, s = np.cos(angle), np.sin(angle)
        # a c = b s: b / a = c / s, its size brought into [1/2, 2) by a power of two on b
        t = np.clip(np.abs(c / s), 2.0 ** -60, 2.0 ** 60)
        shift = np.exp2(np.floor(np.log2(t) + 0.5))
        at = np.clip(np.searchsorted((b / a), t / shift), 1, len(a) - 1)
        at -= np.abs((b / a)[at - 1] - t / shift) < np.abs((b / a)[at] - t / shift)
        x[:, h, :, 0], x[:, h, :, 1] = a[at], b[at] * shift * np.sign(c * s)
        want[:, h, :, 0] = x[:, h, :, 0] * c - x[:, h, :, 1] * s
        want[:, h, :, 1] = x[:, h, :, 1] * c + x[:, h, :, 0] * s
        radius[:, h] = np.hypot(x[:, h, :, 0], x[:, h, :, 1])
    keys = x.reshape(n, hkv, rot) if interleaved else x.transpose(0, 1, 3, 2).reshape(n, hkv, rot)
    pool[0, 1].view(-1, hkv, 128)[slots.cuda()] = torch.tensor(keys).bfloat16().cuda()
    assert np.median(np.abs(want[..., 0]) / radius) < 2.0 ** -13
    pkv.pkv_kv_rerope(pool, 1, table, torch.tensor([n], dtype=torch.int32, device="cuda"), None,
                      f.cuda(), new_positions=torch.tensor(pos, dtype=torch.int32, device="cuda"),
                      interleaved=interleaved)
    assert pkv.pkv_read_device_errors() == 0
    got = pool[0, 1].view(-1, hkv, 128)[slots.cuda()].double().cpu().numpy()
    got = (got.reshape(n, hkv, -1, 2) if interleaved else
           got.reshape(n, hkv, 2, -1).transpose(0, 1, 3, 2))
    off = np.abs(got - want) - HALF_BF16 * np.abs(want)
    worst = (off / radius[..., None]).max()
    assert worst <= (FP32_PART if by_head else ONE_POSITION), \
        f"off by 2^{np.log2(worst):.2f} of the pair's radius"
