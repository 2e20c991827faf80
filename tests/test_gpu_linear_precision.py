"""16-bit outputs of linear attention and gradients of v are fp32 sums rounded once: how often they fall to another side of the last
rounding than 64 bits do, where nothing but a block's own rows and the skip weight makes them."""
import numpy as np
import pytest
import torch

from layer_harness import TINY_STEP, Linear, f64
from oracle import layer as oracle

pytestmark = pytest.mark.gpu

BITS = {"bf16": 8, "f16": 11}


def _step(x, dtype):
    """The distance of the type's neighbouring values around x."""
    exponent = np.floor(np.log2(np.maximum(np.abs(x), 1e-300)))
    return np.maximum(2.0 ** (exponent + 1 - BITS[dtype]), TINY_STEP[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_the_skip_weight_is_held_in_24_bits(dtype):
    """Where the scores are zero a result is skip times a row: the products of parts are exact, and at most five of them are added, each
    rounded (or cut off) to 24 bits, one left out below 2^-24: within 2^-21 of the product before the last rounding. (Many heads: a row's
    elements have few different mantissas.)"""
    b = Linear([64, 30, 6], H=512, Hk=2, dk=32, dv=64, dtype=dtype, seed=40, s0=False, wide=False)
    q, k = b.q, b.k
    for zero, what, rows in (("q", "out", b.v), ("k", "dv", b.do)):
        b.q, b.k = q, k
        setattr(b, zero, torch.zeros_like(q))
        got = f64(b.forward()[0] if what == "out" else b.backward()["dv"])
        want = f64(rows) * f64(b.skip)[None, :, None]
        off = int((np.abs(got - want) > _step(want, dtype) / 2 + 2.0 ** -21 * np.abs(want)).sum())
        assert off == 0, (what, off, want.size)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_pairs_are_held_in_24_bits(dtype):
    """Prompts of one and two tokens from empty states without decays: scores are sums of 16 products of inputs (four of parts each in fp16),
    and a result adds two rows by three parts (five) of a score. Roundings are as often up as down, so that the sum of n of them is off by
    about sqrt(n) 2^-25 of its terms' magnitude: 5 * 2^-25 for 16 + 6, 9 * 2^-25 for 64 + 10. An error e makes a value fall to the
    other side of a rounding in e / step of all cases, where step is the type's; twice the sum of these and ten more are allowed."""
    n = {"bf16": 5, "f16": 9}[dtype]
    b = Linear([1, 2] * 400, H=4, Hk=2, dk=16, dv=64, dtype=dtype, seed=41, s0=False, beta=False, skip=False, wide=False, scale=1.0)
    b.g.zero_()
    out = f64(b.forward()[0])
    want, mag = np.empty_like(out), np.empty_like(out)
    for s in range(b.N):
        for h in range(b.H):
            a, at, _ = b.head(s, h)
            want[at, h] = oracle.linear(**a)[0]
            mag[at, h] = oracle.linear(**{x: np.abs(y) for x, y in a.items()})[0]
    step = _step(want, dtype)
    others = int((np.abs(out - want) > step / 2 * (1 + 1e-9)).sum())
    expected = float(np.minimum(1.0, n * 2.0 ** -25 * mag / step).sum())
    print(dtype, others, expected, out.size)
    assert others <= 2 * expected + 10
