"""Rotary positions with one or several axes (time, height, width ...).

Rotate-half pairs (x_p, x_{p+d/2}) as in ``workloads.rotary``; pair p belongs to
one axis and turns by that axis' position times the pair's frequency.
``rope_axes`` is the plain call, ``rotary_axes`` the same for autograd: the
gradient of a rotation is the rotation back. Both also take interleaved pairs
(x_{2p}, x_{2p+1}), a part of the head, and frequencies scaled for long contexts
(``RopeScaling``). ``norm_rope_axes`` and ``norm_rotary_axes`` put the RMS norm
of every head of q and k before it, in the same pass.
"""

from __future__ import annotations

import functools
import math
import struct
from typing import NamedTuple

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


class RopeScaling(NamedTuple):
    """Frequencies for sequences ``factor`` times as long as the trained ones.

    ``kind`` "linear": every frequency divided by the factor (positions
    interpolated). "ntk": the base times factor ** (P / (P - 1)), P the number of
    pairs of the spectrum, so that the first pair keeps its frequency and the last
    has a factor'th of it. "yarn": by parts (Peng et al., "YaRN", 2023): a pair
    that turns more than ``beta_fast`` times within ``original_max`` positions
    keeps its frequency, one that turns less than ``beta_slow`` times has a
    factor'th of it, with a ramp linear in the turns between, as the paper's formula
    has it; and the turned pairs are multiplied by ``amplitude`` (default
    0.1 log(factor) + 1, the natural logarithm; 1 for the other kinds).

    Models were also trained under the name "yarn" with a ramp linear in the pair's
    index between two rounded borders. Between the borders their frequencies are
    others, in places by more than a factor of two: this kind is not for their
    weights."""
    kind: str
    factor: float
    original_max: int | None = None
    beta_fast: float = 32.0
    beta_slow: float = 1.0
    amplitude: float | None = None

    def checked(self) -> RopeScaling:
        if self.kind not in ("linear", "ntk", "yarn"):
            raise ValueError(f"scaling kind {self.kind!r}: 'linear', 'ntk' or 'yarn'")
        if not (math.isfinite(self.factor) and self.factor >= 1):
            raise ValueError(f"scaling factor {self.factor} is not a number of at least 1")
        if self.kind == "yarn":
            if self.original_max is None or not self.original_max > 0:
                raise ValueError(f"scaling 'yarn' needs original_max > 0, got {self.original_max}")
            if not (math.isfinite(self.beta_fast) and 0 < self.beta_slow < self.beta_fast):
                raise ValueError(f"scaling 'yarn' needs 0 < beta_slow < beta_fast, got {self.beta_slow}, {self.beta_fast}")
        if self.amplitude is not None and not math.isfinite(self.amplitude):
            raise ValueError(f"scaling amplitude {self.amplitude} is not finite")
        return self

    def frequency(self, base: float, index: int, pairs: int) -> float:
        """Of pair ``index`` of a spectrum of ``pairs``."""
        f = base ** -(index / pairs)
        if self.kind == "linear":
            return f / self.factor
        if self.kind == "ntk":
            return f * self.factor ** -(index / (pairs - 1)) if pairs > 1 else f
        turns = self.original_max * f / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - self.beta_slow) / (self.beta_fast - self.beta_slow)))
        return f * keep + f / self.factor * (1 - keep)

    def size(self) -> float:
        if self.amplitude is not None:
            return float(self.amplitude)
        return 0.1 * math.log(self.factor) + 1.0 if self.kind == "yarn" else 1.0


def _laid_out(sections, base, spectrum, rotary_dim, layout, scaling, d):
    """The table of a rotation with a layout: (axis, frequency) of every turned pair, the number of axes, the amplitude
    and whether pairs are interleaved."""
    if scaling is not None and not isinstance(scaling, RopeScaling):
        raise TypeError(f"scaling {scaling!r} is not a RopeScaling")
    return _built_layout(sections, (*map(type, sections),), base, spectrum, rotary_dim, layout, scaling, d)


@functools.lru_cache(maxsize=128, typed=True)
def _built_layout(sections, types, base, spectrum, rotary_dim, layout, scaling, d):
    rotary_dim = d if rotary_dim is None else rotary_dim
    if not isinstance(rotary_dim, int) or rotary_dim < 0 or rotary_dim > d or rotary_dim % 2 != 0:
        raise ValueError(f"rotary_dim {rotary_dim} is not an even number of elements of a head of {d}")
    if layout not in ("half", "interleaved"):
        raise ValueError(f"layout {layout!r}: 'half' or 'interleaved'")
    axis, freq, axes = _built_table(sections, types, base, spectrum, rotary_dim)
    interleaved = int(layout == "interleaved")
    if scaling is None:
        return axis, freq, axes, 1.0, interleaved
    scaling.checked()
    half = rotary_dim // 2
    freq = []
    for pairs in sections:
        for j in range(pairs):
            freq.append(scaling.frequency(base, len(freq), half) if spectrum == "joint" else scaling.frequency(base, j, pairs))
    return axis, struct.pack(f"={half}d", *freq), axes, scaling.size(), interleaved


def _plainly(q, rotary_dim, layout, scaling) -> bool:
    return (rotary_dim is None or rotary_dim == q.shape[-1]) and layout == "half" and scaling is None


def rope_axes(q, k, positions, sections, base=10000.0, spectrum="joint", inverse=False, q_out=None, k_out=None,
              rotary_dim=None, layout="half", scaling=None):
    """Turn q [n, l, h, d] and k [n, l, h_k, d] (or None) by their positions.

    ``positions`` [axes, n, l] int32; ``sections``: how many of the d/2 pairs
    belong to each axis, first axis first. ``spectrum`` "joint": pair p has
    frequency base**(-2p/d) whatever its axis; "axis": the pairs of an axis
    with s pairs have base**(-j/s), j = 0 .. s-1. One axis with all pairs is
    the ordinary rotary embedding. ``inverse`` turns back (the gradient).
    Returns (q_out, k_out); either may be its input, turned in place.

    ``rotary_dim``: only the first so many elements of a head are turned, and
    stand for d above. ``layout``: pairs are (x_p, x_{p + rotary_dim/2}) ("half")
    or (x_{2p}, x_{2p+1}) ("interleaved"). ``scaling``: a RopeScaling; with an
    amplitude other than 1 ``inverse`` is the adjoint, still the gradient."""
    if _plainly(q, rotary_dim, layout, scaling):
        table = _table(tuple(sections), base, spectrum, q.shape[-1])
        return _lib.bind().rope_axes(q, k, positions, table, inverse, q_out, k_out)
    table = _laid_out(tuple(sections), base, spectrum, rotary_dim, layout, scaling, q.shape[-1])
    return _lib.bind().norm_rope_axes(q, k, positions, table, inverse, None, None, 0, 0.0, q_out, k_out)


def rotary_axes(q, k, positions, sections, base=10000.0, spectrum="joint", rotary_dim=None, layout="half", scaling=None):
    """Differentiable ``rope_axes``: (q, k) -> (q_out, k_out), k may be None.

    Captured into a CUDA graph, it refuses a leaf tensor on which a graph made on
    the default stream is still alive: autograd would wait for that stream in the
    middle of the capture. Delete the earlier outputs first."""
    if _plainly(q, rotary_dim, layout, scaling):
        return _lib.bind().rotary_axes(q, k, positions, _table(tuple(sections), base, spectrum, q.shape[-1]))
    table = _laid_out(tuple(sections), base, spectrum, rotary_dim, layout, scaling, q.shape[-1])
    return _lib.bind().norm_rotary_axes(q, k, positions, table, None, None, 0, 0.0)


def norm_rope_axes(q, k, positions, sections, q_weight=None, k_weight=None, eps=1e-6, base=10000.0, spectrum="joint",
                   q_out=None, k_out=None, rotary_dim=None, layout="half", scaling=None):
    """``rope_axes`` of the RMS-normed heads: every row x of q and k becomes
    weight * x / sqrt(mean(x**2) + eps) before it is turned, in the same pass.

    ``q_weight``, ``k_weight`` [d], bf16 or f32 (None: ones). The norm is over the
    whole head, also where only a part of it is turned; sections (0,) with
    rotary_dim 0 is the norm alone. Returns (q_out, k_out); either may be its
    input."""
    table = _laid_out(tuple(sections), base, spectrum, rotary_dim, layout, scaling, q.shape[-1])
    return _lib.bind().norm_rope_axes(q, k, positions, table, 0, q_weight, k_weight, 1, eps, q_out, k_out)


def norm_rotary_axes(q, k, positions, sections, q_weight=None, k_weight=None, eps=1e-6, base=10000.0, spectrum="joint",
                     rotary_dim=None, layout="half", scaling=None):
    """Differentiable ``norm_rope_axes``, in q, k and the weights; once.

    In a CUDA graph it refuses what ``rotary_axes`` refuses, of the weights too."""
    table = _laid_out(tuple(sections), base, spectrum, rotary_dim, layout, scaling, q.shape[-1])
    return _lib.bind().norm_rotary_axes(q, k, positions, table, q_weight, k_weight, 1, eps)
