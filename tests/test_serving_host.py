"""Checks of the rotary and paged calls' arguments and of their oracle that need no GPU."""

import math
import random

import pytest

from oracle import paged as op


@pytest.fixture
def table():
    pytest.importorskip("torch")
    from blockwise_exact_attention_gb300 import rotary
    rotary._built_table.cache_clear()
    return rotary._table


BAD = [((16, 15), 1e4, "joint", "sections"), ((-1, 33), 1e4, "joint", "sections"), ((16.0, 16), 1e4, "joint", "sections"),
       ((16, 16.0), 1e4, "joint", "sections"), ((32,), 1e4, "jointly", "spectrum"), ((16, 16), 0.0, "joint", "base"),
       ((16, 16), -2.0, "joint", "base"), ((16, 16), math.inf, "joint", "base"), ((16, 16), math.nan, "joint", "base"),
       ((16, 16), 1e4, "both", "spectrum"), ((16, 8, 9), 1e4, "axis", "sections"), ((), 1e4, "axis", "sections"),
       (("16", 16), 1e4, "joint", "sections")]


@pytest.mark.parametrize("sections,base,spectrum,names", BAD)
@pytest.mark.parametrize("earlier", [False, True])
def test_rotation_tables_refuse(table, sections, base, spectrum, names, earlier):
    """For their own reason, and whatever was asked for before."""
    if earlier:
        for good in ((16, 16), (32,), (16, 8, 8)):
            for s in ("joint", "axis"):
                table(good, 1e4, s, 64)
    with pytest.raises(ValueError, match=names):
        table(sections, base, spectrum, 64)


def test_rotation_tables_of_equal_arguments_are_equal(table):
    assert table((16, 16), 10000, "joint", 64) == table((16, 16), 1e4, "joint", 64)
    assert table((True, 31), 1e4, "axis", 64) == table((1, 31), 1e4, "axis", 64)
    axis, freq, axes = table((16, 16), 1e4, "joint", 64)
    assert (len(axis), len(freq), axes) == (4 * 32, 8 * 32, 2)


def test_plan_counts_the_pages_that_it_takes():
    """cu_pages against the pages that leave the stack, row by row."""
    rng = random.Random(5)
    n, width, page, pool_len = 5, 6, 4, 40
    lens, table, pool, free = [0] * n, [[-1] * width for _ in range(n)], list(range(pool_len)), pool_len
    steps = 0
    for _ in range(200):
        new = [rng.choice([0, 1, 1, 3, 9, -1]) for _ in range(n)]
        before, had = [list(r) for r in table], list(lens)
        _, _, cu, cup, lens, after, table, pool, ok = op.plan(lens, new, table, pool, free, page, 24)
        if not ok:
            assert cup == [0] * (n + 1) and after == free and table == before
            lens, free = [0] * n, pool_len
            table, pool = [[-1] * width for _ in range(n)], list(range(pool_len))
            continue
        steps += 1
        back = 0
        for r in range(n):
            had_pages = -(-had[r] // page)
            if new[r] < 0:
                back += had_pages
                took = 0
            else:
                took = -(-lens[r] // page) - had_pages
                assert table[r][:had_pages] == before[r][:had_pages]
            assert cup[r + 1] - cup[r] == took
        assert cup[-1] == free + back - after
        free = after
    assert steps > 50
