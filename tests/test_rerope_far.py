"""Re-rotation (pkv_kv_rerope) at positions over the whole of 32 bits, against angles reduced in
exact arithmetic.

Tolerance: that of test_rerope, and what its angles are off by at such positions. A frequency is
kept as a fraction of a turn, off by 2^-52 of its value (the rounded 1 / (2 pi) and a product in
64 bits) and by 2^-64 (cut off): with frequencies of up to 1 radian and positions, or a distance,
of up to 2^32, by 2^32 (2^-52 / (2 pi) + 2^-64) turns for the one product and as much for the
other: 2^-18.99 radians together, which move each of the pair's two products by that much of |a|
or |b|: 2^-18.49 of its radius."""
from __future__ import annotations

from decimal import Decimal, getcontext
from fractions import Fraction
import math

import numpy as np
import pytest
import torch

from test_rerope import FP32_PART, HALF_BF16, freqs, make, turned

FAR = 2.0 ** -18.49


def two_pi():
    """2 pi to 60 digits (Machin's formula)."""
    getcontext().prec = 70

    def arctan_of_inverse(x):
        total, term, k = Decimal(0), Decimal(1) / x, 0
        while abs(term) > Decimal(10) ** -68:
            total += term / (2 * k + 1) * (-1) ** k
            term /= x * x
            k += 1
        return total

    return 8 * (4 * arctan_of_inverse(Decimal(5)) - arctan_of_inverse(Decimal(239)))


def reduced(positions, freq):
    """positions [n] times freq [m] modulo a turn, in 64 bits: [n, m]."""
    turn = Fraction(two_pi())
    out = np.empty((len(positions), len(freq)))
    for j, f in enumerate(freq.tolist()):
        f = Fraction(f)
        for i, p in enumerate(positions):
            x = (f * p) % turn
            out[i, j] = float(x if x <= turn / 2 else x - turn)
    return out


def test_the_reduction_itself():
    assert float(two_pi()) == 2 * math.pi
    x = reduced([-3, 0, 2, 1000], np.float32([1.0, 0.1]))
    want = np.outer([-3, 0, 2, 1000], np.float32([1.0, 0.1]).astype(np.float64))
    assert np.abs(np.exp(1j * x) - np.exp(1j * want)).max() < 1e-12


LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("sides", ["both", "old", "new"])
def test_whole_range_of_positions(same, sides, interleaved):
    import paged_kv_attention_out_gb300 as pkv
    n, rot, hkv = 90, 64, 2
    g = torch.Generator().manual_seed(5)
    old, new = (torch.randint(LOW, HIGH + 1, (1, hkv, n), generator=g) for _ in range(2))
    for i, (a, b) in enumerate([(LOW, HIGH), (HIGH, LOW), (LOW, LOW), (HIGH, HIGH), (0, LOW),
                                (HIGH, 0), (-1, HIGH)]):
        old[0, :, i], new[0, :, i] = a, b
    pool, table = make([n], hkv=hkv, d=128)
    before = pool.cpu()
    fo = freqs(rot)
    fn = fo if same else freqs(rot, 40000.0)
    i = torch.arange(n).expand(1, hkv, n)
    pkv.pkv_read_device_errors()
    pkv.pkv_kv_rerope(pool, 1, table, torch.tensor([n], dtype=torch.int32, device="cuda"),
                      fo.cuda(), fn.cuda(),
                      old_positions=old.int().cuda() if sides != "new" else None,
                      new_positions=new.int().cuda() if sides != "old" else None,
                      interleaved=interleaved)
    assert pkv.pkv_read_device_errors() == 0
    old, new = (i if sides == "new" else old), (i if sides == "old" else new)
    slots = (table[0].cpu().long()[:, None] * 16 + torch.arange(16)).reshape(-1)[:n]
    was = before[0, 1].flatten(0, 1)[slots].double().numpy()
    got = pool.cpu()[0, 1].flatten(0, 1)[slots].double().numpy()
    for h in range(hkv):
        angle = reduced(new[0, h].tolist(), fn) - reduced(old[0, h].tolist(), fo)
        y, radius = turned(was[:, h], angle, rot, interleaved, 1.0)
        over = np.abs(got[:, h] - y) - HALF_BF16 * np.abs(y) - (FP32_PART + FAR) * radius
        assert over.max() <= 0, np.unravel_index(over.argmax(), over.shape)
