"""The normed rotation's oracle against what is known of it, the scaled
frequencies, and the refusals of the entry points, all without a GPU."""

import ctypes
import math

import numpy as np
import pytest

from oracle import norm_rope as on
from oracle import paged as op
from blockwise_exact_attention_gb300 import RopeScaling, _lib, rotary

OK, ARG, SHAPE, DTYPE, ALIGN, UNSUP, WS = 0, -1, -2, -3, -4, -5, -8
BF16, F32, I32 = 0, 1, 2
FAKE = 0x7F0000000000  # never dereferenced: the checks fail first


# ---- the oracle ----------------------------------------------------------------


def test_whole_half_layout_is_the_plain_rotation():
    rng = np.random.default_rng(0)
    x, pos = rng.standard_normal((2, 5, 3, 32)), rng.integers(-50, 900, (2, 2, 5))
    for spectrum in ("joint", "axis"):
        assert np.allclose(on.turn(x, pos, (4, 12), spectrum=spectrum), op.rope_axes(x, pos, (4, 12), spectrum=spectrum),
                           atol=1e-14)


def test_interleaved_is_half_with_the_elements_in_another_order():
    rng = np.random.default_rng(1)
    x, pos = rng.standard_normal((1, 7, 2, 24)), rng.integers(0, 99, (1, 1, 7))
    order = [*range(0, 16, 2), *range(1, 16, 2), *range(16, 24)]
    y = on.turn(x, pos, (8,), rotary_dim=16, layout="interleaved")
    assert np.array_equal(y[..., order], on.turn(x[..., order], pos, (8,), rotary_dim=16))
    assert np.array_equal(y[..., 16:], x[..., 16:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient_by_differences(layout):
    rng = np.random.default_rng(2)
    x, g = rng.standard_normal((2, 1, 3, 2, 16))
    w, pos = rng.standard_normal(16), rng.integers(0, 50, (1, 1, 3))
    how = dict(rotary_dim=8, layout=layout, amplitude=1.3)
    dx, dw = on.norm_turn_bwd(x, w, 1e-3, g, pos, (4,), **how)

    def loss(x, w):
        return (on.norm_turn(x, w, 1e-3, pos, (4,), **how) * g).sum()

    e = 1e-6
    for at in [(0, 0, 0, 0), (0, 1, 1, 5), (0, 2, 0, 15)]:
        d = np.zeros_like(x)
        d[at] = e
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * e) - dx[at]) <= 1e-8
    for c in (0, 7, 9):
        d = np.zeros_like(w)
        d[c] = e
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * e) - dw[c]) <= 1e-8


# ---- scaled frequencies ----------------------------------------------------------

SCALINGS = [dict(kind="linear", factor=4.0), dict(kind="ntk", factor=8.0), dict(kind="yarn", factor=16.0, original_max=2048),
            dict(kind="yarn", factor=2.5, original_max=100, beta_fast=8.0, beta_slow=0.5)]


def table_of(sections, rotary_dim, d, scaling, spectrum="joint", layout="half"):
    axis, freq, axes, size, inter = rotary._laid_out(sections, 10000.0, spectrum, rotary_dim, layout, scaling, d)
    return np.frombuffer(axis, dtype=np.int32), np.frombuffer(freq), axes, size, inter


@pytest.mark.parametrize("kw", SCALINGS)
@pytest.mark.parametrize("spectrum", ["joint", "axis"])
def test_scaled_frequencies(kw, spectrum):
    axis, freq, axes, size, inter = table_of((3, 0, 13), 32, 64, RopeScaling(**kw), spectrum, "interleaved")
    assert axis.tolist() == [0] * 3 + [2] * 13 and axes == 3 and inter == 1
    names = dict(original_max=kw.get("original_max"), fast=kw.get("beta_fast", 32.0), slow=kw.get("beta_slow", 1.0))
    want = []
    for pairs in (3, 0, 13):
        for j in range(pairs):
            at, of = (len(want), 16) if spectrum == "joint" else (j, pairs)
            want.append(on.frequency(10000.0, at, of, kw["kind"], kw["factor"], **names))
    assert np.allclose(freq, want, rtol=1e-14)
    assert math.isclose(size, 0.1 * math.log(kw["factor"]) + 1 if kw["kind"] == "yarn" else 1.0)


def test_scaling_ends():
    """What the kinds promise of the fastest and the slowest pair."""
    plain = table_of((32,), 64, 64, None)[1]
    assert plain[0] == 1.0 and math.isclose(plain[-1], 10000.0 ** -(31 / 32))
    ntk = table_of((32,), 64, 64, RopeScaling("ntk", 4.0))[1]
    assert ntk[0] == 1.0 and math.isclose(ntk[-1], plain[-1] / 4)
    yarn = table_of((32,), 64, 64, RopeScaling("yarn", 4.0, 4096))[1]
    assert yarn[0] == plain[0] and math.isclose(yarn[-1], plain[-1] / 4) and (np.diff(yarn) < 0).all()
    assert table_of((32,), 64, 64, RopeScaling("linear", 4.0, amplitude=0.5))[3] == 0.5
    assert table_of((1,), 2, 64, RopeScaling("ntk", 4.0))[1].tolist() == [1.0]


@pytest.mark.parametrize("kw,names", [
    (dict(scaling=RopeScaling("dynamic", 2.0)), "kind"), (dict(scaling=RopeScaling("linear", 0.5)), "factor"),
    (dict(scaling=RopeScaling("linear", math.nan)), "factor"), (dict(scaling=RopeScaling("yarn", 2.0)), "original_max"),
    (dict(scaling=RopeScaling("yarn", 2.0, 64, 1.0, 1.0)), "beta"), (dict(scaling=RopeScaling("ntk", 2.0, amplitude=math.inf)), "amplitude"),
    (dict(layout="both"), "layout"), (dict(rotary_dim=31), "rotary_dim"), (dict(rotary_dim=66), "rotary_dim"),
    (dict(rotary_dim=-2), "rotary_dim"), (dict(rotary_dim=32), "sections"), (dict(rotary_dim=64.0), "rotary_dim")])
def test_python_refusals(kw, names):
    torch = pytest.importorskip("torch")
    import blockwise_exact_attention_gb300 as bea
    q = torch.zeros(1, 1, 1, 64)
    pos = torch.zeros(1, 1, 1, dtype=torch.int32)
    for call in (bea.norm_rope_axes, bea.norm_rotary_axes, bea.rope_axes, bea.rotary_axes):
        if kw == dict(rotary_dim=64.0) and call in (bea.rope_axes, bea.rotary_axes):
            continue                                     # equal to d: the plain call
        with pytest.raises(ValueError, match=names):
            call(q, None, pos, (32,), **kw)
    with pytest.raises(TypeError, match="RopeScaling"):
        bea.norm_rope_axes(q, None, pos, (32,), scaling={"kind": "linear"})
    with pytest.raises(ValueError, match="CUDA"):
        bea.norm_rope_axes(q, None, pos, (32,))


# ---- the C entry points ------------------------------------------------------------


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    return _lib.load()


def t(shape, dtype=BF16, ptr=FAKE, strides=None):
    if strides is None:
        strides, s = [], 1
        for x in reversed(shape):
            strides.insert(0, s)
            s *= x
    return _lib.describe(ptr, dtype, shape, strides)


def args(**over):
    a = dict(q=t((2, 3, 4, 64)), k=t((2, 3, 2, 64)), pos=t((1, 2, 3), I32), axis=(ctypes.c_int32 * 32)(),
             freq=(ctypes.c_double * 32)(*[1.0] * 32), pairs=32, inter=0, amp=1.0, inverse=0, qw=t((64,), F32), kw=t((64,)),
             norm=1, eps=1e-6, qo=t((2, 3, 4, 64), ptr=FAKE + 4096), ko=t((2, 3, 2, 64), ptr=FAKE + 8192))
    a.update(over)
    return a


def ref(x):
    return None if x is None else ctypes.byref(x)


def fwd(lib, **over):
    a = args(**over)
    return lib.bea_norm_rope_axes(ref(a["q"]), ref(a["k"]), ref(a["pos"]), a["axis"], a["freq"], a["pairs"], a["inter"],
                                  a["amp"], a["inverse"], ref(a["qw"]), ref(a["kw"]), a["norm"], a["eps"], ref(a["qo"]),
                                  ref(a["ko"]), None)


def bwd(lib, ws=FAKE, size=None, gq=t((2, 3, 4, 64)), gk=t((2, 3, 2, 64)), dqw=t((64,), F32), dkw=t((64,)), **over):
    a = args(**over)
    size = lib.bea_norm_rope_axes_bwd_workspace_size(64) if size is None else size
    return lib.bea_norm_rope_axes_bwd(ref(a["q"]), ref(a["k"]), ref(gq), ref(gk), ref(a["pos"]), a["axis"], a["freq"],
                                      a["pairs"], a["inter"], a["amp"], ref(a["qw"]), ref(a["kw"]), a["eps"], ref(a["qo"]),
                                      ref(a["ko"]), ref(dqw), ref(dkw), ws, size, None)


BAD = [
    (dict(q=None), ARG), (dict(qo=None), ARG), (dict(ko=None), ARG), (dict(k=None, ko=None), ARG), (dict(inter=2), ARG),
    (dict(amp=math.inf), ARG), (dict(eps=-1.0), ARG), (dict(eps=math.nan), ARG), (dict(pairs=33), ARG), (dict(pairs=-1), ARG),
    (dict(axis=None), ARG), (dict(freq=None), ARG), (dict(freq=(ctypes.c_double * 32)(math.nan)), ARG),
    (dict(axis=(ctypes.c_int32 * 32)(1)), ARG), (dict(pairs=30), UNSUP), (dict(q=t((2, 3, 4, 72)), qo=t((2, 3, 4, 72)), k=None, ko=None, kw=None, qw=None), UNSUP),
    (dict(qw=t((32,))), SHAPE), (dict(kw=t((1, 64))), SHAPE), (dict(qw=t((64,), I32)), DTYPE), (dict(qw=t((64,), F32, FAKE + 2)), ALIGN),
    (dict(qw=t((64,), F32, strides=[2])), ALIGN), (dict(qo=t((2, 3, 4, 64), F32)), DTYPE), (dict(pos=t((2, 3), I32)), SHAPE),
    (dict(pos=t((1, 2, 4), I32)), SHAPE), (dict(pos=t((9, 2, 3), I32)), SHAPE), (dict(pos=t((1, 2, 3), F32)), DTYPE),
    (dict(qo=t((2, 3, 4, 64), strides=[768, 0, 64, 1])), ARG), (dict(q=t((2, 3, 4, 64), ptr=FAKE + 8)), ALIGN),
]


@pytest.mark.parametrize("over,code", BAD)
def test_refusals(lib, over, code):
    assert fwd(lib, **over) == code
    assert bwd(lib, **over) in ((code, ARG) if "qw" in over or "kw" in over or over.get("k", 1) is None else (code,))


def test_refusals_of_one_call(lib):
    assert fwd(lib, norm=0) == ARG                       # weights without a norm
    assert fwd(lib, norm=2) == ARG
    assert fwd(lib, inverse=1) == ARG                    # no inverse of a norm
    assert fwd(lib, inverse=2, norm=0, qw=None, kw=None) == ARG
    assert bwd(lib, ws=None) == WS and bwd(lib, ws=FAKE + 16) == WS and bwd(lib, size=100) == WS
    assert bwd(lib, gq=None) == ARG and bwd(lib, gk=None) == ARG
    assert bwd(lib, gq=t((2, 3, 4, 64), F32)) == DTYPE and bwd(lib, gk=t((2, 3, 1, 64))) == SHAPE
    assert bwd(lib, dqw=t((64,))) == DTYPE and bwd(lib, dqw=t((32,), F32)) == SHAPE
    assert bwd(lib, qw=None) == ARG                      # a gradient of no weight
    assert lib.bea_norm_rope_axes_bwd_workspace_size(0) == 0 and lib.bea_norm_rope_axes_bwd_workspace_size(-4) == 0
