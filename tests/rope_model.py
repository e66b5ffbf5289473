"""Rotary positions in 64 bits, from the definition."""
import numpy as np


def turn(x, pos, inv, rot, interleaved, m=1.0, sign=1):
    """x (tokens, heads, d) float64 at positions pos; inv radians per position."""
    y = np.array(x, dtype=np.float64)
    a = sign * np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(inv)[None, :]
    c, s = m * np.cos(a)[:, None], m * np.sin(a)[:, None]
    i = np.arange(rot // 2)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    x1, x2 = y[..., one].copy(), y[..., two].copy()
    y[..., one] = x1 * c - x2 * s
    y[..., two] = x2 * c + x1 * s
    return y


def check(got, x, want, m, what=""):
    """bf16 results within their bound of the 64-bit ones.

    One rounding to bf16: 2^-8 of the value. Before it, fp32: the phase is
    right to 2^-32 turns and its conversion to 2^-25 half turns (2e-7 rad with
    the sine's own 2 ulp), the products and the sum add 3 roundings of 2^-24:
    below 1e-6 m (|x1| + |x2|), bounded here by the head's largest element.
    """
    got, x = got.double().cpu().numpy(), np.asarray(x, dtype=np.float64)
    big = np.abs(x).max(axis=-1, keepdims=True)
    bound = np.abs(want) * 2.0 ** -8 + 2e-6 * abs(m) * big
    bad = np.abs(got - want) > bound
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(got - want).max()))
