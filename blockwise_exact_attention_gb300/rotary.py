"""Rotary positions with one or several axes (time, height, width ...).

Rotate-half pairs (x_p, x_{p+d/2}) as in ``workloads.rotary``; pair p belongs to
one axis and turns by that axis' position times the pair's frequency.
``rope_axes`` is the plain call, ``rotary_axes`` the same for autograd: the
gradient of a rotation is the rotation back.
"""

from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import _lib, ops


@functools.lru_cache(maxsize=128)
def _table(sections: tuple, base: float, spectrum: str, half: int):
    """(axis, frequency) of every pair, as the host arrays the library reads."""
    if not all(isinstance(s, int) and s >= 0 for s in sections) or sum(sections) != half:
        raise ValueError(f"sections {sections} are not numbers of pairs that sum to d / 2 = {half}")
    if not (math.isfinite(base) and base > 0):
        raise ValueError(f"base {base} is not a positive number")
    axis, freq = [], []
    for a, pairs in enumerate(sections):
        for j in range(pairs):
            freq.append(base ** -(len(freq) / half if spectrum == "joint" else j / pairs))
            axis.append(a)
    if spectrum not in ("joint", "axis"):
        raise ValueError(f"spectrum {spectrum!r}: 'joint' or 'axis'")
    return (ctypes.c_int32 * half)(*axis), (ctypes.c_double * half)(*freq)


def rope_axes(q, k, positions, sections, base=10000.0, spectrum="joint", inverse=False, q_out=None, k_out=None):
    """Turn q [n, l, h, d] and k [n, l, h_k, d] (or None) by their positions.

    ``positions`` [axes, n, l] int32; ``sections``: how many of the d/2 pairs
    belong to each axis, first axis first. ``spectrum`` "joint": pair p has
    frequency base**(-2p/d) whatever its axis; "axis": the pairs of an axis
    with s pairs have base**(-j/s), j = 0 .. s-1. One axis with all pairs is
    the ordinary rotary embedding. ``inverse`` turns back (the gradient).
    Returns (q_out, k_out); either may be its input, turned in place."""
    table = _table(tuple(sections), float(base), spectrum, q.shape[-1] // 2)
    if positions.ndim != 3 or positions.shape[0] != len(sections):
        raise ValueError(f"positions {tuple(positions.shape)}: [{len(sections)}, n, l] for sections {tuple(sections)}")
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if k is not None and k_out is None:
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    (qr, kr, pr, qo, ko), stream = ops._records(q, k, positions, q_out, k_out)
    rc = _lib.load().bea_rope_axes(qr, kr, pr, *table, 1 if inverse else 0, qo, ko, stream)
    _lib.check(rc, "rope_axes")
    ops._count()
    return q_out, k_out


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, sections, base, spectrum, inverse):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(positions)
        ctx.args = (sections, base, spectrum, inverse)
        ctx.dtypes = (q.dtype, None if k is None else k.dtype)
        return rope_axes(q, k, positions, sections, base, spectrum, inverse)

    @staticmethod
    def backward(ctx, dq, dk):
        (positions,) = ctx.saved_tensors
        sections, base, spectrum, inverse = ctx.args
        # a gradient that autograd hands back may be expanded or of another layout
        dq, dk = (None if g is None or not need else g.to(dt).contiguous()
                  for g, need, dt in zip((dq, dk), ctx.needs_input_grad, ctx.dtypes))
        if dq is not None or dk is not None:
            # through the Function itself, so that the gradient has a gradient too
            first, second = (dk, None) if dq is None else (dq, dk)
            first, second = _Rotary.apply(first, second, positions, sections, base, spectrum, not inverse)
            dq, dk = (None, first) if dq is None else (first, second)
        return dq, dk, None, None, None, None, None


def _check_capture(*outs) -> None:
    """A leaf's accumulation node is shared by all graphs that live on the leaf and
    keeps the stream it was made on. If that is the legacy default stream, a
    backward pass captured on another stream makes autograd wait there in the
    middle of the capture, which ends the process. So a call on the default
    stream leaves a mark at its leaves' nodes, and a captured call that meets the
    mark is refused."""
    if torch.cuda.is_current_stream_capturing():
        def visit(node):
            if node.metadata.get("bea_default_stream"):
                raise RuntimeError("rotary_axes: captured into a CUDA graph while an earlier graph of the same leaf "
                                   "tensors, made on the default stream, is alive; delete its outputs first")
    elif torch.cuda.current_stream().cuda_stream == 0:
        def visit(node):
            node.metadata["bea_default_stream"] = True
    else:
        return
    for out in outs:
        if out is not None and out.grad_fn is not None:
            for node, _ in out.grad_fn.next_functions:
                if node is not None and hasattr(node, "variable"):  # a leaf's accumulation node
                    visit(node)


def rotary_axes(q, k, positions, sections, base=10000.0, spectrum="joint"):
    """Differentiable ``rope_axes``: (q, k) -> (q_out, k_out), k may be None."""
    q_out, k_out = _Rotary.apply(q, k, positions, tuple(sections), float(base), spectrum, False)
    _check_capture(q_out, k_out)
    return q_out, k_out
