"""The oracle of the calls on shared pages against what has to hold of it, and
the refusals of their entry points, all without a GPU."""

import ctypes
import random

import numpy as np
import pytest

from oracle import paged as op
from oracle import pages as og
from blockwise_exact_attention_gb300 import _lib

ARG, SHAPE, DTYPE, ALIGN, UNSUP = -1, -2, -3, -4, -5
BF16, F32, I32 = 0, 1, 2
FAKE = 0x7F0000000000  # never dereferenced: the checks fail first


def holds(lens, table, shares, pool, n_free, page, contents=None, cache=None):
    """Every page is on the stack or held, counted right, and rows read what they should."""
    held = og.owners(lens, table, len(shares), page)
    assert sorted(pool[:n_free]) == [p for p, h in enumerate(held) if h == 0]
    assert shares == [max(0, h - 1) for h in held]
    for r, l in enumerate(lens):
        if cache is not None:
            assert [cache[table[r][i // page], i % page] for i in range(l)] == contents[r][:l]


@pytest.mark.parametrize("page", [1, 3, 4])
def test_a_life_of_forks_and_ends(page):
    """Random steps of fork, free, plan and compact: no page is lost, counted wrong or written by two rows."""
    rng = random.Random(page)
    n, width, count = 9, 6, 60
    lens, table = [0] * n, [[-1] * width for _ in range(n)]
    shares, pool, n_free = [0] * count, list(range(count)), count
    cache, contents, token = np.zeros((count, page), dtype=int), [[] for _ in range(n)], 1
    seen = set()
    for _ in range(400):
        what = rng.choice(["fork", "free", "plan", "plan", "compact"])
        seen.add(what)
        if what == "fork":
            live = [r for r in range(n) if lens[r]]
            src = [rng.choice(live) if live and not lens[r] and rng.random() < 0.5 else -1 for r in range(n)]
            tokens = [rng.randint(-1, lens[s]) if s >= 0 else 0 for s in src]
            lens, table, shares, n_free, copies, ok, clean = og.fork(src, tokens, lens, table, shares, pool, n_free, page)
            assert clean and og.copy(copies, cache)
            if ok:
                for r, s in enumerate(src):
                    if s >= 0:
                        contents[r] = contents[s][:lens[r]]
        elif what == "free":
            ends = [-1 if rng.random() < 0.3 else 0 for _ in range(n)]
            lens, shares, pool, n_free, clean = og.free(ends, lens, table, shares, pool, n_free, page)
            assert clean
        elif what == "plan":
            new = [rng.randint(0, 3) if lens[r] else rng.choice([0, 0, 5]) for r in range(n)]
            new = [min(a, width * page - l) for a, l in zip(new, lens)]
            old = list(lens)
            slots, _, cu, _, lens, n_free, table, pool, ok = op.plan(lens, new, table, pool, n_free, page, 99)
            if ok:
                for r in range(n):
                    contents[r] = contents[r][:old[r]]
                    for s in slots[cu[r]:cu[r + 1]]:
                        cache[s // page, s % page] = token
                        contents[r].append(token)
                        token += 1
        else:
            most = rng.choice([0, 2, count])
            table, shares, pool, where, copies, ok = og.compact(lens, table, shares, pool, n_free, page, most)
            assert ok and og.copy(copies, cache)
            if most == count:                            # all of the used pages lie below all free ones
                assert sorted(pool[:n_free]) == list(range(count - n_free, count)) and pool[:n_free] == sorted(pool[:n_free])[::-1]
        holds(lens, table, shares, pool, n_free, page, contents, cache)
    assert len(seen) == 4


def test_fork_refuses_the_whole_step():
    lens, table, shares, pool = [5, 0, 0, 4], [[1, 2], [-1, -1], [-1, -1], [3, -1]], [0] * 6, [0, 4, 5]
    good = og.fork([-1, 0, 0, -1], None, lens, table, shares, pool, 3, 4)
    assert good[5] and good[0] == [5, 5, 5, 4] and good[4][1:3] == [[2, 5, 1], [2, 4, 1]] and good[2][1] == 2
    for src, tokens, height in [([-1, 1, 0, -1], None, 3), ([-1, 2, 0, -1], None, 3), ([-1, 0, 0, 0], None, 3),
                                ([-1, 4, -1, -1], None, 3), ([-2, 0, 0, -1], None, 3), ([-1, 0, 0, -1], [0, 6, 0, 0], 3),
                                ([-1, 0, 0, -1], [0, -2, 0, 0], 3), ([-1, 0, 0, -1], None, 1), ([-1, 0, 0, -1], None, 4)]:
        bad = og.fork(src, tokens, lens, table, shares, pool, height, 4)
        assert not bad[5] and bad[:4] == (lens, table, shares, height) and bad[4] == [[-1] * 3] * 4


# ---- the C entry points ------------------------------------------------------------


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    return _lib.load()


def t(shape, dtype=I32, ptr=FAKE, strides=None):
    if strides is None:
        strides, s = [], 1
        for x in reversed(shape):
            strides.insert(0, s)
            s *= x
    return _lib.describe(ptr, dtype, shape, strides)


def ref(x):
    return None if x is None else ctypes.byref(x)


STATE = dict(lens=t((4,)), table=t((4, 8)), shares=t((20,)), pool=t((20,)), n_free=t((1,)), page=16, lens_out=t((4,)),
             height_out=t((1,)), shares_out=t((20,)))
FORK = STATE | dict(src=t((4,)), tokens=t((4,)), copies=t((4, 3)))
FREE = STATE | dict(ends=t((4,)))
COMPACT = STATE | dict(table_out=t((4, 8)), pool_out=t((20,)), map=t((20,)), copies=t((5, 3)))


def fork(lib, **over):
    a = {k: v if k == "page" else ref(v) for k, v in (FORK | over).items()}
    return lib.bea_paged_fork(a["src"], a["tokens"], a["lens"], a["table"], a["shares"], a["pool"], a["n_free"], a["page"],
                              a["lens_out"], a["height_out"], a["shares_out"], a["copies"], None)


def free(lib, **over):
    a = {k: v if k == "page" else ref(v) for k, v in (FREE | over).items()}
    return lib.bea_paged_free(a["ends"], a["lens"], a["table"], a["shares"], a["pool"], a["n_free"], a["page"],
                              a["lens_out"], a["height_out"], a["shares_out"], None)


def compact(lib, **over):
    a = {k: v if k == "page" else ref(v) for k, v in (COMPACT | over).items()}
    return lib.bea_paged_compact(a["lens"], a["table"], a["shares"], a["pool"], a["n_free"], a["page"], a["table_out"],
                                 a["shares_out"], a["pool_out"], a["map"], a["copies"], None)


EVERY = [
    (dict(lens=None), ARG), (dict(table=None), ARG), (dict(shares=None), ARG), (dict(pool=None), ARG), (dict(n_free=None), ARG),
    (dict(shares_out=None), ARG), (dict(page=0), ARG), (dict(page=2 ** 20 + 1), ARG), (dict(lens=t((4, 1))), SHAPE),
    (dict(table=t((3, 8))), SHAPE), (dict(n_free=t((2,))), SHAPE), (dict(shares_out=t((19,))), SHAPE),
    (dict(lens=t((4,), F32)), DTYPE), (dict(pool=t((20,), BF16)), DTYPE), (dict(lens=t((4,), ptr=FAKE + 2)), ALIGN),
    (dict(shares=t((20,), strides=[2])), ALIGN), (dict(table=t((4, 2 ** 26), strides=[2 ** 26, 1]), table_out=t((4, 2 ** 26))), SHAPE),
    (dict(shares=t((2 ** 30 + 1,)), shares_out=t((2 ** 30 + 1,)), map=t((2 ** 30 + 1,))), SHAPE), (dict(lens=t((4,), ptr=0)), ARG),
]


@pytest.mark.parametrize("over,code", EVERY)
def test_refusals_of_all(lib, over, code):
    assert fork(lib, **{k: v for k, v in over.items() if k in FORK}) == code
    assert free(lib, **{k: v for k, v in over.items() if k in FREE}) == code
    assert compact(lib, **{k: v for k, v in over.items() if k in COMPACT}) == code


def test_refusals_of_one(lib):
    overlapping = t((4, 8), strides=[4, 1])
    for call in (fork, free):
        assert call(lib, lens_out=None) == ARG and call(lib, height_out=None) == ARG
        assert call(lib, lens_out=t((5,))) == SHAPE and call(lib, height_out=t((2,))) == SHAPE
    assert fork(lib, src=None) == ARG and fork(lib, src=t((5,))) == SHAPE and fork(lib, tokens=t((3,))) == SHAPE
    assert fork(lib, copies=None) == ARG and fork(lib, copies=t((4, 2))) == SHAPE and fork(lib, copies=t((3, 3))) == SHAPE
    assert fork(lib, copies=t((4, 3), strides=[4, 1])) == ALIGN and fork(lib, table=overlapping) == ARG
    assert free(lib, ends=None) == ARG and free(lib, ends=t((5,))) == SHAPE and free(lib, ends=t((4,), F32)) == DTYPE
    assert compact(lib, table_out=None) == ARG and compact(lib, pool_out=None) == ARG and compact(lib, map=None) == ARG
    assert compact(lib, copies=None) == ARG and compact(lib, table_out=t((4, 7))) == SHAPE and compact(lib, pool_out=t((19,))) == SHAPE
    assert compact(lib, map=t((21,))) == SHAPE and compact(lib, table_out=overlapping) == ARG
    assert compact(lib, table_out=t((4, 8), strides=[9, 1])) == ARG  # the table itself, by other strides
    many = t((2 ** 20 + 1,))
    assert compact(lib, shares=many, shares_out=many, map=many) == UNSUP


def test_refusals_of_copy(lib):
    def copy(copies=t((5, 3)), caches=((7, 16, 2, 64), (7, 16, 2, 64)), count=None, **kw):
        ts = [c if isinstance(c, _lib.BeaTensor) else t(c, BF16, **kw) for c in caches]
        arr = (_lib.BeaTensor * max(1, len(ts)))(*ts)
        return lib.bea_paged_copy(ref(copies), arr, len(ts) if count is None else count, None)

    assert copy(copies=None) == ARG and copy(count=-1) == ARG and lib.bea_paged_copy(ref(t((5, 3))), None, 2, None) == ARG
    assert copy(copies=t((5, 4))) == SHAPE and copy(copies=t((15,))) == SHAPE and copy(copies=t((5, 3), strides=[6, 2])) == ALIGN
    assert copy(copies=t((5, 3), F32)) == DTYPE and copy(caches=((7, 16, 2, 64), (8, 16, 2, 64))) == SHAPE
    assert copy(caches=((7, 16, 2, 64), t((7, 16, 2, 64), F32))) == DTYPE and copy(caches=((7, 16, 128),)) == SHAPE
    assert copy(caches=((7, 16, 2, 4),)) == ALIGN
    assert copy(caches=(t((7, 16, 1, 4), BF16, strides=[128, 8, 8, 1]),)) == UNSUP
    assert copy(caches=(t((7, 16, 2, 64), BF16, strides=[2048, 0, 64, 1]),)) == ARG
    assert copy(caches=(t((7, 16, 2, 64), BF16, ptr=FAKE + 8),)) == ALIGN
    assert copy(caches=()) == 0 and copy(copies=t((0, 3))) == 0
    # nothing to copy: the caches are looked at all the same
    assert copy(copies=t((0, 3)), caches=(t((7, 16, 1, 4), BF16, strides=[128, 8, 8, 1]),)) == UNSUP


def test_python_refusals():
    torch = pytest.importorskip("torch")
    import blockwise_exact_attention_gb300 as bea
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        bea.paged_fork(i, None, i, i[:, None], i, i, i[:1], 16)
    with pytest.raises(ValueError, match="capacity"):
        bea.paged_compact(i, i[:, None], i, i, i[:1], 16, -1)
    with pytest.raises(TypeError, match="tensor"):
        bea.paged_free(None, i, i[:, None], i, i, i[:1], 16)
    with pytest.raises(ValueError, match="CUDA"):
        bea.paged_copy(i.view(4, 1), [])
    cache = bea.PagedKVCache(4, 2, 1, 64, 2, 4, device="cpu")
    for call in (lambda: cache.fork(i), lambda: cache.free(i), lambda: cache.compact(2)):
        with pytest.raises(ValueError, match="share_pages"):
            call()


def test_refusals_of_shared_decoding(lib):
    good = dict(q=t((5, 1, 8, 64), BF16), k=t((20, 16, 2, 64), BF16), v=t((20, 16, 2, 64), BF16), table=t((5, 9000)), lens=t((5,)),
                rows=t((4,)), shared=t((3,)), out=t((5, 1, 8, 64), BF16), lse=t((5, 8, 1), F32))

    def call(scale=0.1, ws=FAKE, size=1 << 40, **over):
        a = [ref(x) for x in (good | over).values()]
        return lib.bea_paged_decode_shared(*a, scale, ws, size, None)

    need = lib.bea_paged_decode_shared_workspace_size(5, 8, 2, 64, 144000, 3)
    assert need > 0 and call(size=need - 1) == -8 and call(ws=None) == -8 and call(ws=FAKE + 16) == -8
    for name in good:
        assert call(**{name: None}) == ARG
    assert call(rows=t((3,))) == SHAPE and call(shared=t((4,))) == SHAPE and call(rows=t((4, 1))) == SHAPE
    assert call(rows=t((4,), F32)) == DTYPE and call(shared=t((3,), ptr=FAKE + 1)) == ALIGN
    assert call(rows=t((1026,)), shared=t((1025,))) == UNSUP and call(scale=0.0) == ARG
    assert call(**{k: t((5, 1, 8, 64) if k in ("q", "out") else (20, 16, 2, 64), F32) for k in ("q", "k", "v", "out")}) == UNSUP
    assert call(q=t((5, 2, 8, 64), BF16)) == SHAPE and call(k=t((20, 16, 3, 64), BF16)) == SHAPE
    assert call(out=t((5, 1, 8, 64), BF16, strides=[0, 512, 64, 1])) == ARG
    # counts past 31 bits: 2 h n, and units times tiles
    assert call(q=t((2 ** 20, 1, 1024, 64), BF16), out=t((2 ** 20, 1, 1024, 64), BF16), lse=t((2 ** 20, 1024, 1), F32),
                table=t((2 ** 20, 9)), lens=t((2 ** 20,))) == SHAPE
    assert call(q=t((2 ** 14, 1, 2, 64), BF16), out=t((2 ** 14, 1, 2, 64), BF16), lse=t((2 ** 14, 2, 1), F32),
                table=t((2 ** 14, 2 ** 25)), lens=t((2 ** 14,)), rows=t((1025,)), shared=t((1024,))) == SHAPE
    # a table with little room: what single requests need
    assert lib.bea_paged_decode_shared_workspace_size(5, 8, 2, 64, 1600, 3) == lib.bea_paged_decode_workspace_size(8, 2, 64, 1600) < need
    assert lib.bea_paged_decode_shared_workspace_size(5, 8, 2, 64, 160, 3) == 0
    for bad in [(-1, 8, 2, 64, 9, 3), (5, -8, 2, 64, 9, 3), (5, 8, 0, 64, 9, 3), (5, 8, 2, -64, 9, 3), (5, 8, 2, 64, -9, 3),
                (5, 8, 2, 64, 9, -3), (2 ** 31, 8, 2, 64, 9, 3), (5, 8, 2, 2 ** 40, 9, 3), (5, 8, 2, 64, 9, 2 ** 40)]:
        assert lib.bea_paged_decode_shared_workspace_size(*bad) == 0
