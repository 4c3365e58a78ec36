"""The paged cache's and the rotary embedding's oracle against what is known of
them, and the refusals of their entry points, all without a GPU."""

import ctypes
import math
import random

import numpy as np
import pytest

import oracle
from oracle import paged as op
from blockwise_exact_attention_gb300 import _lib, workloads

OK, ARG, SHAPE, DTYPE, ALIGN, UNSUP, CUDA, TIMEOUT, WS, PAGES = 0, -1, -2, -3, -4, -5, -6, -7, -8, -9
BF16, F32, I32 = 0, 1, 2
FAKE = 0x7F0000000000  # never dereferenced: the checks fail first


# ---- the oracle ----------------------------------------------------------------


def test_rope_one_axis_is_the_workloads_rotary():
    x = np.random.default_rng(0).standard_normal((2, 50, 3, 64)).astype(np.float32)
    pos = np.broadcast_to(np.arange(50), (1, 2, 50))
    assert np.abs(op.rope_axes(x, pos, (32,)) - workloads.rotary(x)).max() <= 2 ** -22 * np.abs(x).max()


def test_rope_axes_turn_their_own_pairs_only():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((1, 4, 2, 32))
    pos = rng.integers(-9, 9, (3, 1, 4))
    for spectrum in ("joint", "axis"):
        y = op.rope_axes(x, pos, (4, 0, 12), spectrum=spectrum)
        moved = pos.copy()
        moved[1] += 5                                    # an axis without pairs
        assert np.array_equal(y, op.rope_axes(x, moved, (4, 0, 12), spectrum=spectrum))
        moved[2] += 1
        z = op.rope_axes(x, moved, (4, 0, 12), spectrum=spectrum)
        same = [p for p in range(32) if p % 16 < 4]
        assert np.array_equal(y[..., same], z[..., same]) and not np.isclose(y, z).all()


def test_rope_inverse_is_inverse_and_adjoint():
    rng = np.random.default_rng(2)
    x, g = rng.standard_normal((2, 1, 5, 3, 16))[:, :, :, None, :].reshape(2, 1, 5, 3, 16)
    pos = rng.integers(0, 1000, (2, 1, 5))
    y = op.rope_axes(x, pos, (3, 5))
    back = op.rope_axes(g, pos, (3, 5), inverse=True)
    assert np.allclose(op.rope_axes(y, pos, (3, 5), inverse=True), x, atol=1e-13)
    assert math.isclose((y * g).sum(), (x * back).sum(), rel_tol=1e-12)
    eps = 1e-6                                           # and the gradient by differences
    for at in [(0, 2, 1, 3), (0, 4, 0, 11)]:
        d = np.zeros_like(x)
        d[at] = eps
        diff = ((op.rope_axes(x + d, pos, (3, 5)) - op.rope_axes(x - d, pos, (3, 5))) * g).sum() / (2 * eps)
        assert abs(diff - back[at]) <= 1e-8


@pytest.mark.parametrize("left", [-1, 0, 5])
def test_decode_is_the_attention_of_the_last_query(left):
    rng = np.random.default_rng(3)
    h, h_kv, d, page, length = 4, 2, 16, 3, 11
    k, v = rng.standard_normal((2, 1, length, h_kv, d))
    q = rng.standard_normal((1, 1, h, d))
    table = np.array([[5, 0, 3, 6, -1]])
    kc, vc = np.full((2, 7, page, h_kv, d), np.nan)
    for j in range(length):
        kc[table[0, j // page], j % page], vc[table[0, j // page], j % page] = k[0, j], v[0, j]
    out, lse, a, s = op.decode(q, kc, vc, table, [length], 0.3, left)
    ref_o, ref_l = oracle.attention_fwd(q, k, v, 0.3, True, (left, 0))
    assert np.allclose(out, ref_o, atol=1e-13) and np.allclose(lse, ref_l, atol=1e-13)
    assert (np.abs(out) <= a + 1e-15).all() and (s > 0).all()


def test_plan_keeps_every_page_once():
    rng = random.Random(4)
    n, width, page, pool_len = 6, 5, 4, 20
    lens, table, pool, free = [0] * n, [[-1] * width for _ in range(n)], list(range(pool_len)), pool_len
    done = 0
    for _ in range(300):
        new = [rng.choice([0, 1, 1, 3, 7, -1]) for _ in range(n)]
        before = (list(lens), [list(r) for r in table], list(pool), free)
        slots, pos, cu, cup, lens, free, table, pool, ok = op.plan(lens, new, table, pool, free, page, 16)
        if not ok:
            assert (lens, table, pool, free) == before and slots == [-1] * 16
            lens, free, table, pool = [0] * n, pool_len, [[-1] * width for _ in range(n)], list(range(pool_len))
            continue
        done += 1
        owned = [table[r][j] for r in range(n) for j in range(-(-lens[r] // page))]
        assert sorted(owned + pool[:free]) == list(range(pool_len))
        used = [s for s in slots if s >= 0]
        assert len(set(used)) == len(used) == cu[-1] == sum(max(a, 0) for a in new)
        assert cup[-1] == cup[-2] + (cup[-1] - cup[-2]) and len(cu) == len(cup) == n + 1
    assert done > 100


# ---- refusals --------------------------------------------------------------------


@pytest.fixture(scope="module")
def lib():
    from blockwise_exact_attention_gb300 import build
    build.build()
    return _lib.load()


def T(shape, dtype=BF16, ptr=FAKE, strides=None):
    if strides is None:
        strides, acc = [], 1
        for s in reversed(shape):
            strides.insert(0, acc)
            acc *= s
    return _lib.describe(ptr, dtype, shape, strides)


def I(*shape, **kw):
    return T(shape, I32, **kw)


def test_status_strings(lib):
    assert lib.bea_status_string(PAGES) not in (b"unknown status", b"")


def test_int_tensors_stay_refused_by_the_attention_calls(lib):
    q = _lib.describe(FAKE, I32, [1, 256, 4, 128], [256 * 512, 512, 128, 1])
    r = ctypes.byref
    assert lib.bea_flash_mha_fwd(r(q), r(q), r(q), r(q), r(q), 0.1, 0, -1, -1, None) == DTYPE


def rope(lib, q=T([2, 6, 4, 64]), k=T([2, 6, 1, 64]), pos=I(2, 2, 6), axis=None, freq=None, inv=0, qo=T([2, 6, 4, 64]),
         ko=T([2, 6, 1, 64]), half=32):
    axis = (ctypes.c_int32 * half)(*([0] * half)) if axis is None else axis
    freq = (ctypes.c_double * half)(*([1.0] * half)) if freq is None else freq
    return lib.bea_rope_axes(q, k, pos, axis, freq, inv, qo, ko, None)


def test_rope_rejects_bad_arguments(lib):
    i32, f64 = ctypes.c_int32 * 32, ctypes.c_double * 32
    assert rope(lib, q=None) == ARG
    assert rope(lib, k=None) == ARG and rope(lib, ko=None) == ARG
    assert rope(lib, inv=2) == ARG
    assert rope(lib, axis=i32(*([0] * 31 + [2]))) == ARG
    assert rope(lib, axis=i32(*([-1] * 32))) == ARG
    assert rope(lib, freq=f64(*([math.inf] * 32))) == ARG
    assert rope(lib, freq=f64(*([math.nan] * 32))) == ARG
    assert rope(lib, pos=T([2, 2, 6], F32)) == DTYPE
    assert rope(lib, pos=I(2, 6)) == SHAPE and rope(lib, pos=I(2, 2, 7)) == SHAPE and rope(lib, pos=I(9, 2, 6)) == SHAPE
    assert rope(lib, pos=I(2, 2, 6, ptr=FAKE + 2)) == ALIGN
    assert rope(lib, pos=I(2, 2, 6, strides=[24, 12, 2])) == ALIGN
    assert rope(lib, k=T([2, 6, 1, 64], F32), ko=T([2, 6, 1, 64], F32)) == DTYPE
    assert rope(lib, qo=T([2, 6, 4, 64], F32)) == DTYPE
    assert rope(lib, q=T([2, 6, 4, 64], I32), qo=T([2, 6, 4, 64], I32)) == DTYPE
    assert rope(lib, qo=T([2, 6, 5, 64])) == SHAPE and rope(lib, ko=T([2, 6, 4, 64])) == SHAPE
    assert rope(lib, k=T([2, 7, 1, 64]), ko=T([2, 7, 1, 64])) == SHAPE
    assert rope(lib, q=T([2, 6, 4, 64], ptr=FAKE + 8)) == ALIGN
    assert rope(lib, q=T([2, 6, 4, 64], strides=[1536, 256, 64, 2])) == ALIGN
    assert rope(lib, qo=T([2, 6, 4, 64], ptr=FAKE + 512, strides=[0, 256, 64, 1])) == ARG      # broadcast output
    assert rope(lib, qo=T([2, 6, 4, 64], strides=[2048, 256, 64, 1])) == ARG                   # half in place
    one = dict(k=None, ko=None, half=160)
    assert rope(lib, q=T([2, 6, 4, 24]), qo=T([2, 6, 4, 24]), **one) == UNSUP
    assert rope(lib, q=T([2, 6, 4, 20], F32), qo=T([2, 6, 4, 20], F32), **one) == UNSUP
    assert rope(lib, q=T([2, 6, 4, 320]), qo=T([2, 6, 4, 320]), **one) == UNSUP
    assert rope(lib, q=T([2, 0, 4, 64]), qo=T([2, 0, 4, 64]), pos=I(2, 2, 0), k=None, ko=None) == OK  # nothing to do


def plan(lib, n=4, lens=None, new=None, table=None, pool=I(40), n_free=I(1), page=16, slots=I(8), pos=I(8), cu=None,
         cup=None, lo=None, nf=I(1)):
    z = lambda x, d: d if x is None else x  # noqa: E731
    return lib.bea_paged_plan(z(lens, I(n)), z(new, I(n)), z(table, I(n, 5)), pool, n_free, page, slots, pos,
                              z(cu, I(n + 1)), z(cup, I(n + 1)), z(lo, I(n)), nf, None)


def test_plan_rejects_bad_arguments(lib):
    assert plan(lib, pool=None) == ARG
    assert plan(lib, lens=I(4, ptr=0)) == ARG
    assert plan(lib, page=0) == ARG and plan(lib, page=(1 << 20) + 1) == ARG
    assert plan(lib, new=I(5)) == SHAPE and plan(lib, table=I(5, 5)) == SHAPE and plan(lib, lo=I(3)) == SHAPE
    assert plan(lib, cu=I(4)) == SHAPE and plan(lib, cup=I(6)) == SHAPE
    assert plan(lib, n_free=I(2)) == SHAPE and plan(lib, nf=I(0)) == SHAPE
    assert plan(lib, pos=I(9)) == SHAPE and plan(lib, table=I(4)) == SHAPE
    assert plan(lib, table=I(4, 1 << 27)) == SHAPE                         # 2^31 tokens a row
    assert plan(lib, lens=T([4], F32)) == DTYPE and plan(lib, slots=T([8], BF16)) == DTYPE
    assert plan(lib, lens=I(4, strides=[2])) == ALIGN and plan(lib, pool=I(40, ptr=FAKE + 1)) == ALIGN
    assert plan(lib, table=I(4, 5, strides=[0, 1])) == ARG and plan(lib, table=I(4, 5, strides=[4, 1])) == ARG


def write(lib, k=T([1, 6, 2, 64]), v=T([1, 6, 2, 64]), slots=I(6), kc=T([9, 16, 2, 64]), vc=T([9, 16, 2, 64])):
    return lib.bea_paged_write(k, v, slots, kc, vc, None)


def test_write_rejects_bad_arguments(lib):
    assert write(lib, slots=None) == ARG
    assert write(lib, kc=T([9, 16, 2, 64], strides=[0, 128, 64, 1])) == ARG
    assert write(lib, v=T([1, 5, 2, 64])) == SHAPE and write(lib, slots=I(5)) == SHAPE and write(lib, slots=I(1, 6)) == SHAPE
    assert write(lib, kc=T([9, 16, 1, 64]), vc=T([9, 16, 1, 64])) == SHAPE
    assert write(lib, kc=T([9, 16, 2, 128]), vc=T([9, 16, 2, 128])) == SHAPE
    assert write(lib, vc=T([8, 16, 2, 64])) == SHAPE
    assert write(lib, kc=T([9, 0, 2, 64]), vc=T([9, 0, 2, 64])) == SHAPE
    assert write(lib, kc=T([1 << 27, 16, 2, 64]), vc=T([1 << 27, 16, 2, 64])) == SHAPE      # 2^31 slots
    assert write(lib, k=T([1, 6, 2, 64], F32)) == DTYPE and write(lib, vc=T([9, 16, 2, 64], F32)) == DTYPE
    assert write(lib, slots=T([6], F32)) == DTYPE
    assert write(lib, k=T([1, 6, 2, 64], ptr=FAKE + 8)) == ALIGN
    f = dict(k=T([1, 6, 2, 12]), v=T([1, 6, 2, 12]), kc=T([9, 16, 2, 12], strides=[512, 32, 16, 1]),
             vc=T([9, 16, 2, 12], strides=[512, 32, 16, 1]))
    f["k"] = f["v"] = T([1, 6, 2, 12], strides=[256, 32, 16, 1])
    assert write(lib, **f) == UNSUP
    assert write(lib, k=T([1, 0, 2, 64]), v=T([1, 0, 2, 64]), slots=I(0)) == OK


def decode(lib, q=None, kc=None, vc=None, table=I(3, 7), lens=I(3), out=None, lse=T([3, 8, 1], F32), scale=0.1, left=-1,
           d=128, dt=BF16, ws=None, nbytes=0, page=16):
    q = T([3, 1, 8, d], dt) if q is None else q
    kc = T([40, page, 2, d], dt) if kc is None else kc
    vc = T([40, page, 2, d], dt) if vc is None else vc
    out = T([3, 1, 8, d], dt) if out is None else out
    return lib.bea_paged_decode(q, kc, vc, table, lens, out, lse, scale, left, ws, nbytes, None)


def test_decode_rejects_bad_arguments(lib):
    assert decode(lib, table=None) == ARG
    assert decode(lib, scale=0.0) == ARG and decode(lib, scale=math.nan) == ARG and decode(lib, left=-2) == ARG
    assert decode(lib, out=T([3, 1, 8, 128], strides=[0, 1024, 128, 1])) == ARG
    assert decode(lib, lse=T([3, 8, 1], F32, strides=[0, 1, 1])) == ARG
    assert decode(lib, q=T([3, 2, 8, 128]), out=T([3, 2, 8, 128])) == SHAPE                 # one new token only
    assert decode(lib, kc=T([40, 16, 3, 128]), vc=T([40, 16, 3, 128])) == SHAPE             # 8 % 3
    assert decode(lib, kc=T([40, 16, 0, 128]), vc=T([40, 16, 0, 128])) == SHAPE
    assert decode(lib, vc=T([40, 8, 2, 128])) == SHAPE and decode(lib, kc=T([40, 16, 2, 64]), vc=T([40, 16, 2, 64])) == SHAPE
    assert decode(lib, table=I(2, 7)) == SHAPE and decode(lib, lens=I(4)) == SHAPE and decode(lib, lse=T([3, 8, 2], F32)) == SHAPE
    assert decode(lib, lens=I(3, 1)) == SHAPE and decode(lib, out=T([3, 1, 4, 128])) == SHAPE
    assert decode(lib, table=I(3, 1 << 26)) == SHAPE                                        # 2^30 keys
    assert decode(lib, kc=T([40, 16, 2, 128], F32)) == DTYPE and decode(lib, lens=T([3], F32)) == DTYPE
    assert decode(lib, lse=T([3, 8, 1], BF16)) == DTYPE
    assert decode(lib, dt=F32, out=T([3, 1, 8, 128], BF16)) == DTYPE
    assert decode(lib, q=T([3, 1, 8, 128], ptr=FAKE + 8)) == ALIGN and decode(lib, table=I(3, 7, ptr=FAKE + 2)) == ALIGN
    assert decode(lib, kc=T([40, 16, 2, 128], strides=[4100, 256, 128, 1])) == ALIGN
    for d, dt in ((96, BF16), (256, BF16), (132, F32), (6, F32)):
        strides = [8 * 256, 8 * 256, 256, 1]
        q = T([3, 1, 8, d], dt, strides=strides)
        c = T([40, 16, 2, d], dt, strides=[16 * 512, 512, 256, 1])
        assert decode(lib, q=q, kc=c, vc=c, out=q) == UNSUP


def test_python_refuses_tensors_off_the_gpu():
    torch = pytest.importorskip("torch")
    import blockwise_exact_attention_gb300 as bea
    q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    pos = torch.zeros(2, 2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        bea.rope_axes(q, None, pos, (16, 16))
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        bea.paged_write(q, q, i, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        bea.paged_plan(i, i, i[:, None], i, i[:1], 16, 4)
    with pytest.raises(ValueError, match="CUDA"):
        bea.paged_decode(q[:, :1], q, q, i[:2, None], i[:2], workspace=q)


@pytest.mark.parametrize("sections,base,spectrum", [
    ((16, 15), 1e4, "joint"), ((-1, 33), 1e4, "joint"), ((16.0, 16), 1e4, "joint"), ((16, 16), 0.0, "joint"),
    ((16, 16), math.inf, "joint"), ((16, 16), 1e4, "both"), ((32,), 1e4, "joint"), ((16, 8, 8), 1e4, "axis")])
def test_rope_python_refusals(sections, base, spectrum):
    torch = pytest.importorskip("torch")
    import blockwise_exact_attention_gb300 as bea
    q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bea.rope_axes(q, None, torch.zeros(2, 2, 3, dtype=torch.int32), sections, base, spectrum)
