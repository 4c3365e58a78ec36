"""paged_fork, paged_free, paged_compact and paged_copy against their
definitions: whole numbers and copied bits, equal."""

import random

import pytest

from oracle import pages as og

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

I32 = torch.int32
PAGES = -9


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def i32(x, cols=None):
    return torch.tensor(x, dtype=I32, device="cuda").reshape(len(x), cols if cols is not None else -1) if cols is not None \
        else torch.tensor(x, dtype=I32, device="cuda")


def state(n, width, page, spare, seed, live=0.7, shared=0):
    """lens, table, shares, pool, n_free: rows in groups that hold the same first pages, and free rows."""
    rng = random.Random(seed)
    lens = [rng.randint(0, width * page) if rng.random() < live else 0 for _ in range(n)]
    groups = [[] for _ in range(max(1, n // 4))]
    total, rows = 0, []
    for r in range(n):
        g = groups[rng.randrange(len(groups))]
        held = og.pages(lens[r], page)
        common = min(held, rng.randint(0, shared)) if shared else 0
        while len(g) < common:
            g.append(total)
            total += 1
        rows.append(g[:common] + list(range(total, total + held - common)))
        total += held - common
    count = total + spare
    ids = list(range(count))
    rng.shuffle(ids)
    table = [[ids[p] for p in row] + [-1] * (width - len(row)) for row in rows]
    held = og.owners(lens, table, count, page)
    free = [p for p in range(count) if held[p] == 0]
    rng.shuffle(free)
    shares = [max(0, h - 1) for h in held]
    return lens, table, shares, free + [-1] * (count - len(free)), len(free)


SIZES = [(1, 1, 1), (4, 3, 16), (33, 40, 8), (257, 70, 16), (1100, 9, 20), (60, 600, 1)]


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("some", [False, True])
@pytest.mark.parametrize("n,width,page", SIZES)
def test_fork(n, width, page, some, alias):
    import blockwise_exact_attention_gb300 as bea
    lens, table, shares, pool, height = state(n, width, page, n + 3, n, live=0.4)
    rng = random.Random(n)
    lens[0] = max(lens[0], 1) if table[0][0] >= 0 else lens[0]
    live = [r for r in range(n) if lens[r]]
    src = [rng.choice(live) if live and not lens[r] and rng.random() < 0.8 else -1 for r in range(n)]
    tokens = [rng.randint(-1, lens[s]) if s >= 0 else 99 for s in src] if some else None
    want = og.fork(src, tokens, lens, table, shares, pool, height, page)
    assert want[5] and want[6]
    L, T, S, P, H = i32(lens), i32(table, width), i32(shares), i32(pool), i32([height])
    out = bea.PagedFork(L, H, S, torch.full((n, 3), 7, dtype=I32, device="cuda")) if alias else None
    got = bea.paged_fork(i32(src), None if tokens is None else i32(tokens), L, T, S, P, H, page, out)
    assert got.lens.tolist() == want[0] and T.tolist() == want[1] and got.shares.tolist() == want[2]
    assert got.n_free.tolist() == [want[3]] and got.copies.tolist() == want[4] and P.tolist() == pool
    if not alias:
        assert L.tolist() == lens and S.tolist() == shares and H.tolist() == [height]
    assert bea.device_status() == 0


def test_fork_refused_as_a_whole():
    import blockwise_exact_attention_gb300 as bea
    lens, table, shares, pool = [5, 0, 0, 4], [[1, 2], [-1, -1], [-1, -1], [3, -1]], [0] * 6, [0, 4, 5, -1, -1, -1]
    none, big = [-1] * 4, 2 ** 31 - 1
    for src, tokens, l, height in [([-1, 1, 0, -1], none, lens, 3), ([-1, 2, 0, -1], none, lens, 3), ([-1, 0, 0, 0], none, lens, 3),
                                   ([-1, 4, -1, -1], none, lens, 3), ([-2, 0, 0, -1], none, lens, 3), ([-1, big, -1, -1], none, lens, 3),
                                   ([-1, 0, 0, -1], [0, 6, 0, 0], lens, 3), ([-1, 0, 0, -1], [0, -2, 0, 0], lens, 3),
                                   ([-1, 0, 0, -1], none, lens, 1), ([-1, 0, 0, -1], none, lens, 7), ([-1, 0, 0, -1], none, lens, -1),
                                   ([-1, 0, -1, -1], none, [9, 0, 0, 4], 3), ([-1, 0, -1, -1], none, [-3, 0, 0, 4], 3),
                                   ([-1, 0, -1, -1], none, [5, -1, 0, 4], 3)]:
        T = i32(table, 2)
        got = bea.paged_fork(i32(src), i32(tokens), i32(l), T, i32(shares), i32(pool), i32([height]), 4)
        assert got.lens.tolist() == l and T.tolist() == table and got.shares.tolist() == shares
        assert got.n_free.tolist() == [height] and got.copies.tolist() == [[-1] * 3] * 4
        assert bea.device_status() == PAGES
    # pages outside: handed on uncounted, not copied
    for bad in (-1, 6, big):
        T = i32([[1, bad, 2, -1], [-1] * 4, [-1] * 4], 4)
        got = bea.paged_fork(i32([-1, 0, 0]), i32([0, 9, 6]), i32([9, 0, 0]), T, i32(shares), i32(pool), i32([3]), 4)
        assert T.tolist()[1] == [1, bad, 5, -1] and T.tolist()[2] == [1, 4, -1, -1]
        assert got.shares.tolist() == [0, 2, 0, 0, 0, 0] and got.copies.tolist() == [[-1] * 3, [2, 5, 1], [-1, -1, 0]]
        assert bea.device_status() == PAGES


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("rate", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("n,width,page", SIZES)
def test_free(n, width, page, rate, alias):
    import blockwise_exact_attention_gb300 as bea
    lens, table, shares, pool, height = state(n, width, page, 5, n, shared=width // 2)
    rng = random.Random(n)
    ends = [rng.choice([-1, -7]) if rng.random() < rate else rng.choice([0, 3]) for _ in range(n)]
    want = og.free(ends, lens, table, shares, pool, height, page)
    assert want[4]
    L, T, S, P, H = i32(lens), i32(table, width), i32(shares), i32(pool), i32([height])
    got = bea.paged_free(i32(ends), L, T, S, P, H, page, bea.PagedFreed(L, H, S) if alias else None)
    assert got.lens.tolist() == want[0] and got.shares.tolist() == want[1] and P.tolist() == want[2]
    assert got.n_free.tolist() == [want[3]] and T.tolist() == table
    if not alias:
        assert L.tolist() == lens and S.tolist() == shares and H.tolist() == [height]
    assert bea.device_status() == 0


@pytest.mark.parametrize("n,width,pages", [(3, 5000, 14000), (70, 2000, 131072), (150, 2100, 300000)])
def test_free_of_many_pages(n, width, pages):
    """Caches of which a warp takes several words, and of more than one turn."""
    import blockwise_exact_attention_gb300 as bea
    rng = random.Random(pages)
    ids = rng.sample(range(pages), pages)
    held, rest = ids[:pages * 2 // 3], ids[pages * 2 // 3:]
    counts, table, lens = [0] * pages, [], []
    for _ in range(n):
        m = rng.randint(0, width)
        row = rng.sample(held, m)
        for p in row:
            counts[p] += 1
        table.append(row + [-1] * (width - m))
        lens.append(2 * m - (rng.random() < 0.5 and m > 0))
    shares = [max(c - 1, 0) for c in counts]
    pool = rest + [-1] * (pages - len(rest))
    ends = [rng.choice([-1, 0]) for _ in range(n)]
    want = og.free(ends, lens, table, shares, pool, len(rest), 2)
    P = i32(pool)
    got = bea.paged_free(i32(ends), i32(lens), i32(table, width), i32(shares), P, i32([len(rest)]), 2)
    assert want[4] and got.lens.tolist() == want[0] and got.shares.tolist() == want[1] and P.tolist() == want[2]
    assert got.n_free.tolist() == [want[3]] and bea.device_status() == 0


def test_free_of_wrong_states():
    import blockwise_exact_attention_gb300 as bea
    table = [[1, 2], [1, 9], [-1, 3], [0, 5]]
    shares, pool, page = [0, 1, 0, 0, 0, 0], [4, -1, -1, -1, -1, -1], 4
    for ends, lens, s, p, height in [
            ([-1] * 4, [5, 8, 8, 9], shares, pool, 1),           # a page outside twice, a length past the table
            ([-1] * 4, [5, 4, 0, -2], shares, pool, 1),          # a negative length
            ([-1, -1, 0, 0], [5, 4, 0, 0], [0] * 6, pool, 1),    # given back twice, held once
            ([-1] * 4, [5, 4, 0, 8], shares, pool[:3], 1),       # a stack that is too short
            ([-1] * 4, [5, 4, 0, 8], shares, pool, 7), ([-1] * 4, [5, 4, 0, 8], shares, pool, -1)]:
        want = og.free(ends, lens, table, s, p, height, page)
        assert not want[4]
        P = i32(p)
        got = bea.paged_free(i32(ends), i32(lens), i32(table, 2), i32(s), P, i32([height]), page)
        assert got.lens.tolist() == want[0] and got.shares.tolist() == want[1] and P.tolist() == want[2]
        assert got.n_free.tolist() == [want[3]] and bea.device_status() == PAGES


@pytest.mark.parametrize("n,width,page", [(1, 3000, 8), (2, 8000, 3), (3, 30000, 2), (100, 129, 16), (5, 65, 1)])
def test_few_long_rows(n, width, page):
    """Rows whose entries several warps, or several blocks, take."""
    import blockwise_exact_attention_gb300 as bea
    lens, table, shares, pool, height = state(n, width, page, 2 * n + 9, n, live=0.9, shared=width // 3)
    lens, table = lens + [0] * n, table + [[-1] * width] * n
    src = [-1] * n + [r if lens[r] else -1 for r in range(n)]
    T, S, P, H = i32(table, width), i32(shares), i32(pool), i32([height])
    want = og.fork(src, [-1] * 2 * n, lens, table, shares, pool, height, page)
    got = bea.paged_fork(i32(src), None, i32(lens), T, S, P, H, page)
    assert got.lens.tolist() == want[0] and T.tolist() == want[1] and got.shares.tolist() == want[2]
    assert got.n_free.tolist() == [want[3]] and got.copies.tolist() == want[4]
    lens, table, shares, height = want[0], want[1], want[2], want[3]
    want = og.compact(lens, table, shares, pool, height, page, 50)
    moved = bea.paged_compact(got.lens, T, got.shares, P, got.n_free, page, 50)
    assert all(a.tolist() == b for a, b in zip(moved, want))
    ends = [-1 if r % 3 != 1 else 0 for r in range(2 * n)]
    want = og.free(ends, lens, want[0], want[1], want[2], height, page)
    freed = bea.paged_free(i32(ends), got.lens, moved.block_table, moved.shares, moved.free_pages, got.n_free, page)
    assert freed.lens.tolist() == want[0] and freed.shares.tolist() == want[1] and moved.free_pages.tolist() == want[2]
    assert freed.n_free.tolist() == [want[3]] and bea.device_status() == 0


@pytest.mark.parametrize("most", [0, 3, 10 ** 4])
@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("n,width,page", SIZES)
def test_compact(n, width, page, alias, most):
    import blockwise_exact_attention_gb300 as bea
    lens, table, shares, pool, height = state(n, width, page, n * width // 3 + 1, n, live=0.5, shared=width // 3)
    want = og.compact(lens, table, shares, pool, height, page, most)
    assert want[5]
    L, T, S, P, H = i32(lens), i32(table, width), i32(shares), i32(pool), i32([height])
    out = bea.PagedCompaction(T, S, P, torch.empty_like(S), torch.empty(most, 3, dtype=I32, device="cuda")) if alias else None
    got = bea.paged_compact(L, T, S, P, H, page, most, out)
    for a, b in zip(got, want):
        assert a.tolist() == b
    if not alias:
        assert T.tolist() == table and S.tolist() == shares and P.tolist() == pool
    assert L.tolist() == lens and H.tolist() == [height] and bea.device_status() == 0


def test_compact_of_many_pages():
    """More pages than a thread's word, up to the most that are allowed; past them the call is refused."""
    import blockwise_exact_attention_gb300 as bea
    for count in (31, 32, 33, 32767, 32768, 100001, 2 ** 20):
        g = torch.Generator(device="cuda")
        g.manual_seed(count)
        ids = torch.randperm(count, device="cuda", generator=g).to(I32)
        height = count // 3
        table = ids[height:].reshape(1, -1).contiguous()
        pool = torch.full((count,), -1, dtype=I32, device="cuda")
        pool[:height] = ids[:height]
        got = bea.paged_compact(i32([count - height]), table, torch.zeros_like(pool), pool, i32([height]), 1, count // 2)
        used = count - height
        assert torch.equal(got.free_pages[:height], torch.arange(count - 1, used - 1, -1, dtype=I32, device="cuda"))
        assert (got.free_pages[height:] == -1).all()
        assert torch.equal(got.block_table[0].sort().values, torch.arange(used, dtype=I32, device="cuda"))
        assert torch.equal(got.block_table[0], got.page_map[table[0].long()])
        moved = got.copies[got.copies[:, 0] >= 0]
        assert len(moved) == int((ids[:height] < used).sum()) and torch.equal(got.page_map[moved[:, 0].long()], moved[:, 1])
        low = ids[:height][ids[:height] < used].sort().values
        assert torch.equal(moved[:, 1], low) and (moved[:, 0].diff() < 0).all() and (moved[:, 2] == 1).all()
        assert bea.device_status() == 0
    many = torch.zeros(2 ** 20 + 1, dtype=I32, device="cuda")
    with pytest.raises(bea._lib.BeaError, match="UNSUPPORTED"):
        bea.paged_compact(i32([0]), i32([0], 1), many, many, i32([0]), 1, 4)


def test_compact_of_wrong_states():
    import blockwise_exact_attention_gb300 as bea
    lens, table, shares = [7, 3], [[5, 2], [4, -1]], [0] * 6
    for pool, height in [([0, 1, 0, -1, -1, -1], 3), ([0, 1, 6, -1, -1, -1], 3), ([0, -1, 3, -1, -1, -1], 3),
                         ([0, 1, 3, -1, -1, -1], 7), ([0, 1, 3, -1, -1, -1], -1)]:
        want = og.compact(lens, table, shares, pool, height, 4, 3)
        got = bea.paged_compact(i32(lens), i32(table, 2), i32(shares), i32(pool), i32([height]), 4, 3)
        assert not want[5] and [a.tolist() for a in got] == list(want[:5]) and bea.device_status() == PAGES
    for lens, table in [([7, 3], [[5, 6], [4, -1]]), ([7, 3], [[5, -1], [4, -1]]), ([9, -4], [[5, 2], [4, -1]])]:
        want = og.compact(lens, table, shares, [0, 1, 3, -1, -1, -1], 3, 4, 3)
        got = bea.paged_compact(i32(lens), i32(table, 2), i32(shares), i32([0, 1, 3, -1, -1, -1]), i32([3]), 4, 3)
        assert not want[5] and [a.tolist() for a in got] == list(want[:5]) and bea.device_status() == PAGES


# ---- copy ------------------------------------------------------------------------


def cache_like(how, pages, page, h_kv, d, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if how == "dense":
        c = torch.empty(pages, page, h_kv, d, dtype=dtype, device="cuda")
    elif how == "heads first":
        c = torch.empty(pages, h_kv, page, d, dtype=dtype, device="cuda").transpose(1, 2)
    else:  # keys and values of a token side by side, and something else behind
        c = torch.empty(pages, page, h_kv + 1, 2 * d, dtype=dtype, device="cuda")[:, :, :h_kv, d:]
    return c.copy_(torch.randn(pages, page, h_kv, d, device="cuda", generator=g))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pages,page,h_kv,d", [(40, 16, 8, 128), (9, 1, 1, 64), (33, 20, 3, 80), (12, 300, 2, 64), (300, 3, 1, 8)])
def test_copy(pages, page, h_kv, d, dtype):
    import blockwise_exact_attention_gb300 as bea
    rng = random.Random(pages)
    ids = rng.sample(range(pages), pages)
    copies = [[-1, -1, -1] if rng.random() < 0.3 else [ids[rng.randrange(pages // 2)], new, rng.choice([0, 1, page // 2, page, page])]
              for new in ids[pages // 2:]]
    hows = ["dense", "heads first", "beside", "dense"]
    caches = [cache_like(h, pages, page, h_kv, d, dtype, 1 + i) for i, h in enumerate(hows)]
    want = [c.clone() for c in caches]
    assert all(og.copy(copies, c) for c in want)
    versions = [c._version for c in caches]
    assert bea.paged_copy(i32(copies, 3), caches) is caches
    assert all(torch.equal(a, b) for a, b in zip(caches, want)) and all(c._version > v for c, v in zip(caches, versions))
    assert bea.device_status() == 0


def test_copy_of_many_caches_and_of_nothing():
    import blockwise_exact_attention_gb300 as bea
    caches = [cache_like("dense", 5, 4, 2, 64, torch.bfloat16, i) for i in range(130)]
    want = [c.clone() for c in caches]
    bea.launches_since_reset(True)
    bea.paged_copy(i32([[0, 3, 4], [1, 4, 2]], 3), tuple(caches))
    assert bea.launches_since_reset() == 3
    for a, b in zip(caches, want):
        og.copy([[0, 3, 4], [1, 4, 2]], b)
        assert torch.equal(a, b)
    bea.paged_copy(i32([[0, 3, 4]], 3), [])
    bea.paged_copy(torch.empty(0, 3, dtype=I32, device="cuda"), caches)
    assert all(torch.equal(a, b) for a, b in zip(caches, want)) and bea.device_status() == 0


def test_a_step_is_refused_before_it_changes_the_cache_when_its_copies_would_be():
    import blockwise_exact_attention_gb300 as bea
    cache = bea.PagedKVCache(8, 16, 2, 64, 3, 64, share_pages=True)
    cache.plan(i32([20, 0, 0]), 20)
    names = "block_table", "lens", "shares", "free_pages", "n_free"
    before = [getattr(cache, x).clone() for x in names]
    other_pages = torch.empty(8, 8, 2, 64, dtype=torch.bfloat16, device="cuda")
    short_rows = torch.empty(8, 16, 2, 4, dtype=torch.float16, device="cuda")
    for bad, error in (([cache.k, other_pages], ValueError), ([cache.k, cache.k.float()], bea._lib.BeaError), ([short_rows], TypeError),
                       ([cache.k[..., 4:]], bea._lib.BeaError), ([cache.k, cache.k.cpu()], ValueError)):
        for step in (lambda: cache.fork(i32([-1, 0, -1]), caches=bad), lambda: cache.compact(4, caches=bad)):
            with pytest.raises(error):
                step()
            assert all(torch.equal(getattr(cache, x), b) for x, b in zip(names, before))
    step = cache.fork(i32([-1, 0, -1]), caches=(cache.v, cache.k))
    assert step.lens.tolist() == [20, 20, 0] and bea.device_status() == 0


def test_copy_leaves_out_what_does_not_fit():
    import blockwise_exact_attention_gb300 as bea
    big = 2 ** 31 - 1
    for bad in ([-1, 2, 1], [7, 2, 1], [0, 7, 1], [0, -5, 3], [3, 3, 2], [0, 2, 5], [0, 2, big], [big, 2, 4], [-2 ** 31, 2, 4]):
        cache = cache_like("dense", 7, 4, 2, 64, torch.float32, 1)
        want = cache.clone()
        want[4][:2] = want[1][:2]
        bea.paged_copy(i32([bad, [1, 4, 2]], 3), [cache])
        assert torch.equal(cache, want) and bea.device_status() == PAGES


def test_copy_past_32_bit_offsets():
    import blockwise_exact_attention_gb300 as bea
    cache = torch.empty(70000, 64, 8, 128, dtype=torch.bfloat16, device="cuda")  # 9.2 GB
    cache[69999].normal_()
    cache[3].zero_()
    bea.paged_copy(i32([[69999, 3, 64], [69999, 40000, 63]], 3), [cache])
    assert torch.equal(cache[3], cache[69999]) and torch.equal(cache[40000][:63], cache[69999][:63])


# ---- as they are used --------------------------------------------------------------


def test_a_life_of_a_cache_in_captured_steps():
    """Steps of a cache whose rows share pages, captured once and replayed with new numbers, against the definitions."""
    import blockwise_exact_attention_gb300 as bea
    from oracle import paged as op
    rng = random.Random(3)
    n, width, page, count, h_kv, d = 7, 5, 4, 40, 1, 64
    cache = bea.PagedKVCache(count, page, h_kv, d, n, width * page, share_pages=True)
    lens, table, shares = [0] * n, [[-1] * width for _ in range(n)], [0] * count
    pool, height = cache.free_pages.tolist(), count
    keys = torch.zeros(count, page, dtype=torch.float64)
    cache.k.zero_(), cache.v.zero_()
    src, tokens, new = (torch.zeros(n, dtype=I32, device="cuda") for _ in range(3))
    k = torch.zeros(1, 24, h_kv, d, dtype=torch.bfloat16, device="cuda")

    def fork():
        cache.fork(src, tokens)

    def step():
        cache.write(k, k, cache.plan(new, 24).slot_map)

    def compact():
        cache.compact(6)

    graphs = {}
    src.fill_(-1)
    new.zero_()
    for f in (fork, step, compact):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            f()
        torch.cuda.current_stream().wait_stream(side)
        graphs[f] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[f]):
            f()
    token = 1
    for _ in range(60):
        f = rng.choice([fork, step, step, compact])
        if f is fork:
            live = [r for r in range(n) if lens[r]]
            s = [rng.choice(live) if live and not lens[r] else -1 for r in range(n)]
            t = [rng.randint(-1, lens[x]) if x >= 0 else -1 for x in s]
            src.copy_(i32(s)), tokens.copy_(i32(t))
            lens, table, shares, height, copies, _, _ = og.fork(s, t, lens, table, shares, pool, height, page)
            og.copy(copies, keys)
        elif f is step:
            a = [-1 if lens[r] and rng.random() < 0.25 else min(rng.randint(0, 3), width * page - lens[r]) for r in range(n)]
            new.copy_(i32(a))
            lens, shares, pool, height, _ = og.free(a, lens, table, shares, pool, height, page)
            slots, _, _, _, lens, height, table, pool, _ = op.plan(lens, a, table, pool, height, page, 24)
            for i, slot in enumerate(slots):
                k[0, i] = (token + i) % 251
                if slot >= 0:
                    keys[slot // page, slot % page] = (token + i) % 251
            token += 24
        else:
            table, shares, pool, _, copies, _ = og.compact(lens, table, shares, pool, height, page, 6)
            og.copy(copies, keys)
        graphs[f].replay()
        assert cache.lens.tolist() == lens and cache.shares.tolist() == shares and cache.n_free.tolist() == [height]
        assert cache.free_pages.tolist()[:height] == pool[:height]
        got = cache.block_table.tolist()
        for r, l in enumerate(lens):
            assert got[r][:og.pages(l, page)] == table[r][:og.pages(l, page)]
        assert torch.equal(cache.k[:, :, 0, 0].double().cpu(), keys) and torch.equal(cache.v[:, :, 0, 63].double().cpu(), keys)
        assert bea.device_status() == 0


def test_on_another_stream_behind_its_writer():
    import blockwise_exact_attention_gb300 as bea
    lens, table, shares, pool, height = state(40, 30, 8, 50, 1, live=0.5)
    src = [next(r for r in range(40) if lens[r]) if not l else -1 for l in lens]
    want = og.fork(src, None, lens, table, shares, pool, height, 8)
    side = torch.cuda.Stream()
    for _ in range(20):
        T, P, H, S = i32(table, 30), i32(pool), i32([height]), i32(shares)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            L = i32(lens) + 0
            got = bea.paged_fork(i32(src), None, L, T, S, P, H, 8)
        torch.cuda.current_stream().wait_stream(side)
        assert T.tolist() == want[1] and got.copies.tolist() == want[4] and got.shares.tolist() == want[2]
