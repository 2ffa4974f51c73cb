"""Plain references of the rotary operators in numpy float64: turns of a rotation's pairs, the rotation of part of a
vector, and the normalised and rotated latents that an append quantizes."""
from __future__ import annotations

import math

import numpy as np


def turns(n_rot, base, scaling=None):
    """Angle of each pair per position.  scaling: None, ("linear", s) or ("yarn", s, original, fast, slow)."""
    out = []
    for i in range(n_rot // 2):
        t = base ** (-2.0 * i / n_rot)
        if scaling and scaling[0] == "linear":
            t /= scaling[1]
        elif scaling:
            _, s, original, fast, slow = scaling
            edge = lambda b: n_rot * math.log(original / (2 * math.pi * b)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(math.floor(edge(fast)), 0), min(math.ceil(edge(slow)), n_rot - 1)
            r = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            t = t * (1 - r) + t / s * r
        out.append(t)
    return np.array(out)


def rotate(x, pos, n_rot, first, halves, base, scaling=None, inverse=False, magnitude=1.0):
    """x [rows, .., dim] float64 with its pairs turned by pos [rows] and multiplied by magnitude."""
    angle = np.asarray(pos, np.float64).reshape(-1, *[1] * (x.ndim - 1)) * turns(n_rot, base, scaling)
    c, s = magnitude * np.cos(angle), magnitude * np.sin(angle) * (-1 if inverse else 1)
    y, h = x.copy(), n_rot // 2
    a = slice(first, first + h) if halves else slice(first, first + n_rot, 2)
    b = slice(first + h, first + n_rot) if halves else slice(first + 1, first + n_rot, 2)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def partners(x, n_rot, first, halves):
    """|x| with each rotated channel's partner's added: what bounds the error of a rotated channel."""
    y, h = np.abs(x), n_rot // 2
    a = slice(first, first + h) if halves else slice(first, first + n_rot, 2)
    b = slice(first + h, first + n_rot) if halves else slice(first + 1, first + n_rot, 2)
    y[..., a] = y[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y
