"""Plain 64-bit forms of rotary positions, on the CPU, with the error bound the
GPU results are held to.

Sines and cosines are off by at most 2^-23: 2^-24.35 radians from the fp32 rounding of
the angle left after the nearest quarter turn (at most 1/8 of a turn), 2^-24 from
one unit in the last place of a value below 1.  A turned value is two fp32
products and a sum: two roundings of 2^-24 of |a cos| + |b sin|.  In all (|a| + |b|)
(2^-23 + 2^-23), and half a step of the output's type."""
import math

import torch

ANGLE = 2.0 ** -22


def frequencies(n, base=10000.0):
    return base ** (-torch.arange(n, dtype=torch.float64) / n)


def angles(positions, freq, axis=None):
    """[rows, pairs] angles in 64 bits of positions [axes, rows]: less whole turns by integers, so that the farthest
    positions lose nothing."""
    from fractions import Fraction
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    out = torch.zeros((positions.shape[1], len(freq)), dtype=torch.float64)
    for i, w in enumerate(freq.tolist()):
        turns = Fraction(w) / (2 * pi)
        for r, p in enumerate(positions[0 if axis is None else axis[i]].tolist()):
            t = p * turns
            out[r, i] = float(t - round(t)) * 2 * math.pi
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
