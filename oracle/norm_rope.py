"""The oracle of the normed rotation and its other layouts: the definition pair
by pair in fp64 numpy, sharing no code with the kernels."""

from __future__ import annotations

import math

import numpy as np


def frequency(base, index, pairs, kind=None, factor=1.0, original_max=None, fast=32.0, slow=1.0):
    """Radians per position of pair `index` of a spectrum of `pairs`."""
    f = base ** -(index / pairs)
    if kind == "linear":
        f = f / factor
    elif kind == "ntk":                                  # another base, whose last pair has a factor'th of the frequency
        f = (base * factor ** (pairs / (pairs - 1))) ** -(index / pairs) if pairs > 1 else f
    elif kind == "yarn":
        turns = original_max / (2 * math.pi / f)
        if turns < slow:
            f = f / factor
        elif turns <= fast:
            keep = (turns - slow) / (fast - slow)
            f = (1 - keep) * f / factor + keep * f
    return f


def pairs_of(d, rotary_dim, layout):
    """[(first, second)] element of every turned pair."""
    half = rotary_dim // 2
    return [(p, p + half) if layout == "half" else (2 * p, 2 * p + 1) for p in range(half)]


def turn(x, positions, sections, base=10000.0, spectrum="joint", rotary_dim=None, layout="half", inverse=False,
         amplitude=1.0, **scaling):
    """x [n, l, h, d], positions [axes, n, l]."""
    x = np.asarray(x, dtype=np.float64)
    rotary_dim = x.shape[-1] if rotary_dim is None else rotary_dim
    where = pairs_of(x.shape[-1], rotary_dim, layout)
    y = x.copy()
    p = 0
    for a, count in enumerate(sections):
        for j in range(count):
            f = frequency(base, p, rotary_dim // 2, **scaling) if spectrum == "joint" else frequency(base, j, count, **scaling)
            ang = np.asarray(positions[a], dtype=np.float64)[:, :, None] * f * (-1 if inverse else 1)
            i, k = where[p]
            y[..., i] = amplitude * (x[..., i] * np.cos(ang) - x[..., k] * np.sin(ang))
            y[..., k] = amplitude * (x[..., k] * np.cos(ang) + x[..., i] * np.sin(ang))
            p += 1
    return y


def norm_turn(x, w, eps, positions, sections, **how):
    x = np.asarray(x, dtype=np.float64)
    r = 1 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    return turn(x * r * (1.0 if w is None else np.asarray(w, dtype=np.float64)), positions, sections, **how)


def norm_turn_bwd(x, w, eps, g, positions, sections, **how):
    """(dx, dw) for the output's gradient g."""
    x = np.asarray(x, dtype=np.float64)
    w = np.ones(x.shape[-1]) if w is None else np.asarray(w, dtype=np.float64)
    d = x.shape[-1]
    r = 1 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    back = turn(g, positions, sections, inverse=True, **how)
    dw = (back * x * r).reshape(-1, d).sum(0)
    gy = back * w
    return r * gy - x * r ** 3 * (gy * x).sum(-1, keepdims=True) / d, dw


def spread(x, rotary_dim, layout, amplitude=1.0):
    """|x| of an element, and of both where it belongs to a turned pair: what rounding bounds are proportional to."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    y = a.copy()
    for i, k in pairs_of(a.shape[-1], rotary_dim, layout):
        y[..., i] = y[..., k] = abs(amplitude) * (a[..., i] + a[..., k])
    return y
