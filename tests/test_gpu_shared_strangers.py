"""Rows of a group whose tables name other pages than the first row's among the shared keys: they get their own keys.
Where a row ended and another prompt's took its place, a range of rows still spans it."""

import numpy as np
import pytest

from test_gpu_paged_shared import BF16, F32, check, i32, make, run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def spare(x, row, at, seed):
    """Entry `at` of a row goes to a new page, with values of its own. -> the inputs with it"""
    q, k, v, table, lens = x
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    page = torch.randn((2, 1, *k.shape[1:]), device="cuda", generator=g).to(BF16)
    table = table.clone()
    table[row, at] = k.shape[0]
    return q, torch.cat([k, page[0]]), torch.cat([v, page[1]]), table, lens


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [1, 7, 16, 100, 128, 300])
def test_one_other_page(page, d):
    """The first, one inside, the last of the whole tiles, and the one behind them, of any row, the first among them."""
    import blockwise_exact_attention_gb300 as bea
    keys = 1000 // page * page + page
    x, g = make([(keys, [0, 5, None, 130, page])], 4, 2, d, page, seed=page + d)
    last = keys // 128 * 128 // page                     # the page that the next tile begins in, or that a tile ends in
    for n, (row, at) in enumerate([(1, 0), (3, last // 2), (4, max(last - 1, 0)), (3, min(last, keys // page - 1)), (0, 1),
                                   (0, 0)]):
        y = spare(x, row, at, n)
        for dtype in (BF16, F32):
            check(*run(y, g, 0.2, out_dtype=dtype), *y, 0.2)
        assert bea.device_status() == 0


def test_other_prompts_among_the_rows():
    """Many strangers, with lengths of their own, in groups of many rows and of few, and in all rows."""
    import blockwise_exact_attention_gb300 as bea
    rng = np.random.default_rng(3)
    x, g = make([(1200, [int(a) for a in rng.integers(0, 300, 90)]), (640, [3, 9, 40]), (256, [1] * 12)], 8, 2, 64, 16, seed=5)
    for n, rows in enumerate([[5], [0, 44, 45, 89], [91], list(range(0, 105, 3)), list(range(105))]):
        y = x
        k, v, table = x[1], x[2], x[3].clone()
        for r in rows:                                   # all of its pages are another request's of the same table
            other = (r + 95) % 105 if r < 90 else r - 60
            pages = min(int(x[4][r]), int(x[4][other])) // 16
            table[r, :pages] = x[3][other, :pages]
        y = (x[0], k, v, table, x[4])
        check(*run(y, g, 0.1), *y, 0.1)
        assert bea.device_status() == 0


@pytest.mark.parametrize("n", [300, 1100])
def test_many_rows_of_a_group(n):
    import blockwise_exact_attention_gb300 as bea
    x, g = make([(384, [i % 9 for i in range(n)])], 2, 2, 64, 16, seed=n)
    y = x
    for z, (r, at) in enumerate([(n - 1, 23), (n // 2, 0), (151, 7), (152, 8), (153, 9), (n - 2, 24 - 1)]):
        y = spare(y, r, at, z)
    check(*run(y, g, 0.1), *y, 0.1)
    assert bea.device_status() == 0


def test_a_row_that_took_the_place_of_one_that_ended():
    """Through a cache: forks of a prompt, one of which ends, and another prompt in its row."""
    import blockwise_exact_attention_gb300 as bea
    n, h, h_kv, d, page = 6, 8, 2, 128, 16
    cache = bea.PagedKVCache(400, page, h_kv, d, n, 24000, share_pages=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    cache.k.normal_(generator=gen), cache.v.normal_(generator=gen)
    cache.plan(i32([1500] + [0] * 5), 1500)
    cache.fork(i32([-1, 0, 0, 0, 0, 0]))
    cache.plan(i32([1, 1, -1, 1, 1, -1]), 4)
    cache.plan(i32([1, 1, 1400, 1, 1, 0]), 1404)
    q = torch.randn((n, 1, h, d), device="cuda", generator=gen).to(BF16)
    out, lse = cache.decode_shared(q, i32([0, 6]), i32([1500]), 0.1)
    check(out, lse, q, cache.k, cache.v, cache.block_table, cache.lens, 0.1)
    assert bea.device_status() == 0


@pytest.mark.parametrize("page,prompt,shared", [(16, 1541, 1536), (100, 1540, 1408), (100, 1500, 1408), (256, 1000, 768), (7, 1540, 1536),
                                                (300, 1537, 1408), (1000, 1999, 896)])
def test_forks_that_name_the_prompt_as_shared(page, prompt, shared):
    """The page that a prompt ends in is a copy in each fork: what stands before it stays shared. (A workspace begins with
    the number of shared keys that each row leaves to its group.)"""
    import blockwise_exact_attention_gb300 as bea
    n, h, h_kv, d = 9, 4, 2, 64
    cache = bea.PagedKVCache(12 * (prompt // page + 3), page, h_kv, d, n, 40000, share_pages=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(page)
    cache.k.normal_(generator=gen), cache.v.normal_(generator=gen)
    cache.plan(i32([prompt] + [0] * (n - 1)), prompt)
    cache.fork(i32([-1] + [0] * (n - 2) + [-1]))
    cache.plan(i32([1] * (n - 1) + [prompt]), n - 1 + prompt)       # and one row of another prompt
    q = torch.randn((n, 1, h, d), device="cuda", generator=gen).to(BF16)
    g = i32([0, n]), i32([prompt])
    ws = torch.zeros(bea.paged_decode_shared_workspace_bytes(q, cache.k, cache.block_table, g[1]), dtype=torch.uint8, device="cuda")
    out, lse = cache.decode_shared(q, *g, 0.1, workspace=ws)
    check(out, lse, q, cache.k, cache.v, cache.block_table, cache.lens, 0.1)
    assert ws[:4 * n].view(torch.int32).tolist() == [shared] * (n - 1) + [0] and bea.device_status() == 0
