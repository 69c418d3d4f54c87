"""The AdamW update of one layer, bit for bit: every operation rounded to float32 as the update is written,

    m <- fma(c1, g, b1 m)      v <- fma(c2 g, g, b2 v)      L <- fma(L, decay, -(step m / fma(sqrt(v), r, eps)))

with the coefficients formed in float64 and rounded once.  The fused multiply-adds are worked out here in
float64: the product of two float32 values is exact there, and a sum that is not is rounded to odd, so that
rounding it to float32 is the only rounding (float64 has more than twice float32's digits, and two more)."""
import math

import numpy as np
import pytest
import torch

from learnable_channel_permutation_b200 import binding as b

F, D = np.float32, np.float64


def _fma(a, x, c):
    p, c = a.astype(D) * x.astype(D), c.astype(D)
    s = p + c
    t = s - p
    err = (p - (s - t)) + (c - t)                            # what the sum lost, exactly
    bits = s.view(np.int64)
    even = (bits & 1) == 0
    toward = np.where((err > 0) == (s > 0), 1, -1)           # the neighbour on the side of the exact sum
    odd = np.where((err != 0) & even, bits + toward, bits).view(D)
    return odd.astype(F)


def _update(L, g, m, v, t, lr, b1, b2, eps, wd):
    c = lambda x: np.full(L.shape, F(x))
    m = _fma(c(1 - b1), g, c(b1) * m)
    v = _fma(c(1 - b2) * g, g, c(b2) * v)
    den = _fma(np.sqrt(v), c(1 / math.sqrt(1 - b2 ** t)), c(eps))
    return _fma(L, c(1 - lr * wd), -(c(lr / (1 - b1 ** t)) * m / den)), m, v


def test_the_emulated_multiply_add():
    """Against whole numbers: 24-bit factors and addends of every distance, ties among them."""
    rng = np.random.default_rng(0)
    a, x = (rng.integers(1 << 23, 1 << 24, 20000) for _ in range(2))
    c = rng.integers(-(1 << 24), 1 << 24, 20000) * (1 << rng.integers(0, 30, 20000))
    c[:2000] = (1 << 23) - a[:2000] * x[:2000] % (1 << 24)   # halfway between two float32 values
    c[:2000] -= c[:2000] % 2
    keep = np.array([F(int(k)) == k for k in c])
    got = _fma(a.astype(F), x.astype(F), c.astype(F))

    def nearest(n):
        k = max(abs(n).bit_length() - 24, 0)
        q, r = divmod(abs(n), 1 << k)
        q += 1 if 2 * r > (1 << k) or (2 * r == (1 << k) and q & 1) else 0
        return math.copysign(q * 2.0 ** k, n)

    want = np.array([nearest(int(i) * int(j) + int(k)) for i, j, k in zip(a, x, c)])
    assert keep.sum() > 15000 and np.array_equal(got.astype(D)[keep], want[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("t", [1, 2, 30, 4000])
@pytest.mark.parametrize("scale", [1e-6, 1e-3, 10.0])
@pytest.mark.parametrize("wd", [0.0, 0.01])
def test_adamw_bit_for_bit(gpu_lib, t, scale, wd):
    rng = np.random.default_rng(t)
    n = 40000
    spread = lambda s: (rng.normal(size=n) * s * np.exp2(rng.integers(-6, 7, n))).astype(F)
    L, g, m, v = spread(1e-2), spread(scale), spread(0.1 * scale) * F(t > 1), np.square(spread(0.1 * scale)) * F(t > 1)
    g[:50] = 0
    dev = [torch.from_numpy(x.copy()).cuda() for x in (L, g, m, v)]
    b.adamw(*dev, b.adamw_params(lr=5e-3, weight_decay=wd), t)
    want = _update(L, g, m, v, t, 5e-3, 0.9, 0.999, 1e-8, wd)
    for got, w in zip((dev[0], dev[2], dev[3]), want):
        assert np.array_equal(got.cpu().numpy(), w)
