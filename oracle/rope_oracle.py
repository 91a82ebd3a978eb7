"""CPU oracle of the rotary positions, in 64 bits with exact angles, from the
definitions in include/oscar.h (test infrastructure only)."""
from __future__ import annotations

from fractions import Fraction

import numpy as np

D = 128
PLAIN, LINEAR, NTK, BANDS, YARN = range(5)


def speeds(dims, theta, scaling=PLAIN, factor=1.0, trained=0.0, low=0.0, high=0.0):
    """Radians a position of each pair."""
    n = dims // 2
    if scaling == NTK:
        theta = theta * factor ** (dims / (dims - 2))
    w = np.array([theta ** (-2.0 * i / dims) for i in range(n)])
    if scaling == LINEAR:
        return w / factor
    if scaling in (BANDS, YARN):
        if low == 0 and high == 0:
            low, high = 1.0, 4.0 if scaling == BANDS else 32.0
        if scaling == BANDS:
            keep = (trained * w / (2 * np.pi) - low) / (high - low)
        else:
            pair = lambda t: dims * np.log(trained / (2 * np.pi * t)) / (2 * np.log(theta))  # noqa: E731
            a, b = max(np.floor(pair(high)), 0.0), min(np.ceil(pair(low)), dims - 1.0)
            keep = 1.0 - (np.arange(n) - a) / max(b - a, 0.001)
        keep = np.clip(keep, 0.0, 1.0)
        return w / factor * (1 - keep) + w * keep
    return w


def size(scaling=PLAIN, factor=1.0, given=0.0):
    if given:
        return given
    return 0.1 * np.log(factor) + 1.0 if scaling == YARN and factor > 1 else 1.0


def angles(pos, w):
    """pos·w modulo a turn, from the exact product of the position and the speed in turns as a double."""
    turns = [Fraction(float(x / (2 * np.pi))) for x in w]
    return np.array([[float((int(p) * t) % 1) * 2 * np.pi for t in turns] for p in pos])


def rope(x, pos, w, interleaved, gamma=None, eps=0.0, m=1.0):
    """x [n][heads][128] float64 at positions pos [n]."""
    x = x.astype(np.float64)
    if gamma is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gamma
    n = len(w)
    i = np.arange(n)
    p, r = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    a = angles(pos, w)[:, None]
    out = x.copy()
    out[..., p] = (x[..., p] * np.cos(a) - x[..., r] * np.sin(a)) * m
    out[..., r] = (x[..., r] * np.cos(a) + x[..., p] * np.sin(a)) * m
    return out
