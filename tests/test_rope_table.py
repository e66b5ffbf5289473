"""The rotary table against w_i = base^(-2 i / rotary_dim) / 2 pi in integers:
w_i by an integer root, pi by Machin's arctangents. No GPU."""
import math
from fractions import Fraction

import pytest

import global_soft_capped_b200 as g2

BITS = 300


def pi():
    def arctan_inverse(x):  # of 1 / x, times 2^BITS
        total, term, n = 0, (1 << BITS) // x, 1
        while term:
            total += term // n if n % 4 == 1 else -(term // n)
            term, n = term // (x * x), n + 2
        return total
    return Fraction(4 * (4 * arctan_inverse(5) - arctan_inverse(239)), 1 << BITS)


PI = pi()


def root(n, k):
    """The integer part of the k-th root of n, by bisection."""
    lo, hi = 0, 1 << (n.bit_length() // k + 1)
    while lo < hi:
        mid = (lo + hi + 1) // 2
        if mid ** k <= n:
            lo = mid
        else:
            hi = mid - 1
    return lo


def turns(i, rot, base):
    """base^(-2 i / rot) / 2 pi to some 2^-200."""
    k = rot // 2
    up = Fraction(root(base ** i << (200 * k), k), 1 << 200)   # base^(i / k)
    return 1 / up / (2 * PI)


def table(plan):
    return [f % 2 ** 64 for f in plan.freqs.tolist()]


def test_pi():
    assert float(PI) == math.pi and abs(PI - Fraction(355, 113)) < Fraction(3, 10 ** 7)


@pytest.mark.parametrize("rot,base", [(16, 10000), (64, 10000), (128, 10000), (256, 10000),
                                      (128, 1000000), (96, 500000)])
def test_table_is_rounded_once(rot, base):
    """Within half a unit (2^-65 turns per position; the roots are a little off)."""
    got = table(g2.rope_plan(rot, device="cpu", base=float(base)))
    linear = table(g2.rope_plan(rot, device="cpu", base=float(base), scaling="linear", factor=8.0))
    half = Fraction(1, 2) + Fraction(1, 10 ** 6)
    for i in range(rot // 2):
        want = turns(i, rot, base) * 2 ** 64
        assert abs(got[i] - want) <= half, i
        assert abs(linear[i] - want / 8) <= half, i


def test_far_positions():
    """Phases of the farthest positions, pair 0 and all others, to 2^-34 turns."""
    rot = 128
    got = table(g2.rope_plan(rot, device="cpu"))
    for p in (2 ** 31 - 1, -2 ** 31, 123456789):
        for i in range(rot // 2):
            off = Fraction(got[i] * p, 2 ** 64) - turns(i, rot, 10000) * p
            assert abs(off - round(off)) <= Fraction(1, 2 ** 34) * Fraction(1001, 1000), (p, i)


def test_given_frequencies_are_taken_exactly():
    """Doubles, as they are: each is the number of radians it stands for."""
    given = [1.0, 0.3, -0.7, 5.25, 1e-9, 2.0 ** -60, 0.0, 40000.5]
    got = table(g2.rope_plan(16, device="cpu", frequencies=given))
    for f, w in zip(got, given):
        off = Fraction(f) - Fraction(w) / (2 * PI) * 2 ** 64
        assert abs(off - round(off / 2 ** 64) * 2 ** 64) <= Fraction(1, 2) + Fraction(1, 10 ** 6)


@pytest.mark.parametrize("scaling", [dict(), dict(scaling="linear", factor=4.0),
                                     dict(scaling="ntk", factor=8.0),
                                     dict(scaling="yarn", factor=16.0, trained_len=4096)])
def test_table_and_frequencies_agree(scaling):
    """The doubles of rope_frequencies are the same numbers, rounded."""
    inv, m = g2.rope_frequencies(64, **scaling)
    plan = g2.rope_plan(64, device="cpu", **scaling)
    assert plan.mscale == m
    for f, w in zip(table(plan), inv):
        assert abs(Fraction(f, 2 ** 64) - Fraction(w) / (2 * PI)) <= Fraction(w) * 2 / 2 ** 54 + \
            Fraction(1, 2 ** 64)


def test_numbers_of_any_kind():
    """numpy and torch scalars, as sizes read from a configuration may be."""
    import numpy as np
    import torch
    want = g2.rope_plan(64, device="cpu", base=500000.0, scaling="ntk", factor=4.0)
    for n, b, f in ((np.int64(64), np.float32(500000), np.float64(4)),
                    (64, torch.tensor(500000.0), 4)):
        got = g2.rope_plan(n, device="cpu", base=b, scaling="ntk", factor=f)
        assert torch.equal(got.freqs, want.freqs) and got.rotary_dim == 64
    inv, _ = g2.rope_frequencies(np.int32(8), scaling="yarn", factor=np.float32(2))
    assert inv == g2.rope_frequencies(8, scaling="yarn", factor=2.0)[0]
    given = g2.rope_plan(np.int64(4), device="cpu", frequencies=np.array([1.0, 0.5]))
    assert torch.equal(given.freqs, g2.rope_plan(4, device="cpu", frequencies=[1.0, 0.5]).freqs)
