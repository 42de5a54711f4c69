"""Plain 64-bit forms of rotary positions, on the CPU, with the error bound the
GPU results are held to.

Sines and cosines are off by at most 2^-23: 2^-24.35 radians from the fp32 rounding of
the angle left after the nearest quarter turn (at most 1/8 of a turn), 2^-24 from
one unit in the last place of a value below 1.  A turned value is two fp32
products and a sum: two roundings of 2^-24 of |a cos| + |b sin|.  In all (|a| + |b|)
(2^-23 + 2^-23), and half a step of the output's type."""
import math
from fractions import Fraction

import torch

ANGLE = 2.0 ** -22


def frequencies(n, base=10000.0):
    return base ** (-torch.arange(n, dtype=torch.float64) / n)


def angles(positions, freq, axis=None):
    """[rows, pairs] angles in 64 bits of positions [axes, rows], less whole turns: the turns of a step are taken in
    whole numbers of 2^-96 turns, three words of 32 bits, so that the farthest positions lose nothing."""
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    out = torch.zeros((positions.shape[1], len(freq)), dtype=torch.float64)
    word = 2 ** 32
    for i, w in enumerate(freq.tolist()):
        steps = round(Fraction(w) / (2 * pi) * 2 ** 96) % 2 ** 96
        w0, w1, w2 = steps >> 64, steps >> 32 & word - 1, steps & word - 1
        p = positions[0 if axis is None else axis[i]].long()
        low = p * w1 + torch.div(p * w2, word, rounding_mode="floor")      # in 2^-64 turns
        high = (p * w0 + torch.div(low, word, rounding_mode="floor")) % word
        turns = (high.double() + (low % word).double() / word) / word
        out[:, i] = torch.where(turns > 0.5, turns - 1, turns) * 2 * math.pi
    return out


def turn(x, positions, freq, axis=None, adjacent=False, inverse=False):
    """Turned rows x [n, heads, D] in 64 bits, and the bound of their fp32 arithmetic."""
    n = len(freq)
    t = angles(positions, freq, axis) * (-1 if inverse else 1)
    c, s = t.cos()[:, None], t.sin()[:, None]
    x = x.double()
    y, tol = x.clone(), torch.zeros_like(x)
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if adjacent else (slice(0, n), slice(n, 2 * n))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    tol[..., a] = tol[..., b] = (x[..., a].abs() + x[..., b].abs()) * ANGLE
    return y, tol
