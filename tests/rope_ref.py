"""Rotary positions in 64 bits, from their definition: the angle of a pair from whole numbers (a position times a 64-bit fraction of
a turn), cosine and sine in double, layouts by explicit channel lists."""

import math

import numpy as np

EPS = 2.0 ** -24  # fp32: half a step


def angles(turns, positions):
    """[T][pairs] radians in [0, 2 pi), exact before the conversion to a double."""
    f = [int(t) % 2 ** 64 for t in turns]
    return np.array([[2 * math.pi * (int(p) * t % 2 ** 64 / 2.0 ** 64) for t in f] for p in positions]).reshape(len(positions), len(f))


def pairs(rotary, interleaved):
    n = rotary // 2
    return [(2 * i, 2 * i + 1) if interleaved else (i, i + n) for i in range(n)]


def rotate(x, positions, rope):
    """x float64 [T][heads][D] -> (rotated, error of fp32 arithmetic).

    Cosine and sine: the angle's conversion to fp32 (half a step of at most pi / 4), the function's step (2^-23), what lies below
    2^-32 of a turn, the product with the magnitude (half a step): under 2^-22 (1 + 2^-1) of the magnitude.  The two products
    and the sum: a fused one and one of its own, two half steps of each term at most.  All of it: 2^-21 M (|a| + |b|)."""
    y, err = x.copy(), np.zeros_like(x)
    th, M = angles(rope.turns.cpu().numpy(), positions), rope.magnitude
    for i, (a, b) in enumerate(pairs(rope.rotary_dim, rope.interleaved)):
        c, s = M * np.cos(th[:, i])[:, None], M * np.sin(th[:, i])[:, None]
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        err[..., a] = err[..., b] = 2.0 ** -21 * abs(M) * (abs(x[..., a]) + abs(x[..., b]))
    return y, err
