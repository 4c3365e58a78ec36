"""Rotary positions with one or several axes (time, height, width ...).

Rotate-half pairs (x_p, x_{p+d/2}) as in ``workloads.rotary``; pair p belongs to
one axis and turns by that axis' position times the pair's frequency.
``rope_axes`` is the plain call, ``rotary_axes`` the same for autograd: the
gradient of a rotation is the rotation back.
"""

from __future__ import annotations

import functools
import math
import struct

from . import _lib


def _table(sections: tuple, base: float, spectrum: str, d: int) -> tuple[bytes, bytes, int]:
    """(axis, frequency) of every pair, as the int32 and double arrays the library reads, and the number of axes."""
    return _built_table(sections, (*map(type, sections),), base, spectrum, d)


# To a cache 16.0 is 16, so the arguments' types are part of its key.
@functools.lru_cache(maxsize=128, typed=True)
def _built_table(sections: tuple, types: tuple, base: float, spectrum: str, d: int) -> tuple[bytes, bytes, int]:
    half = d // 2
    if not all(isinstance(s, int) and s >= 0 for s in sections) or sum(sections) != half:
        raise ValueError(f"sections {sections} are not numbers of pairs that sum to d / 2 = {half}")
    if not (math.isfinite(base) and base > 0):
        raise ValueError(f"base {base} is not a positive number")
    if spectrum not in ("joint", "axis"):
        raise ValueError(f"spectrum {spectrum!r}: 'joint' or 'axis'")
    axis, freq = [], []
    for a, pairs in enumerate(sections):
        for j in range(pairs):
            freq.append(base ** -(len(freq) / half if spectrum == "joint" else j / pairs))
            axis.append(a)
    return struct.pack(f"={half}i", *axis), struct.pack(f"={half}d", *freq), len(sections)


def rope_axes(q, k, positions, sections, base=10000.0, spectrum="joint", inverse=False, q_out=None, k_out=None):
    """Turn q [n, l, h, d] and k [n, l, h_k, d] (or None) by their positions.

    ``positions`` [axes, n, l] int32; ``sections``: how many of the d/2 pairs
    belong to each axis, first axis first. ``spectrum`` "joint": pair p has
    frequency base**(-2p/d) whatever its axis; "axis": the pairs of an axis
    with s pairs have base**(-j/s), j = 0 .. s-1. One axis with all pairs is
    the ordinary rotary embedding. ``inverse`` turns back (the gradient).
    Returns (q_out, k_out); either may be its input, turned in place."""
    table = _table(tuple(sections), base, spectrum, q.shape[-1])
    return _lib.bind().rope_axes(q, k, positions, table, inverse, q_out, k_out)


def rotary_axes(q, k, positions, sections, base=10000.0, spectrum="joint"):
    """Differentiable ``rope_axes``: (q, k) -> (q_out, k_out), k may be None.

    Captured into a CUDA graph, it refuses a leaf tensor on which a graph made on
    the default stream is still alive: autograd would wait for that stream in the
    middle of the capture. Delete the earlier outputs first."""
    return _lib.bind().rotary_axes(q, k, positions, _table(tuple(sections), base, spectrum, q.shape[-1]))
