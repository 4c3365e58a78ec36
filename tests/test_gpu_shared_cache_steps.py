"""Steps of a PagedKVCache that are refused leave it as it was, also where the step is several calls."""

import pytest

from test_gpu_paged_shared import BF16, i32

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def state(cache):
    return [t.clone() for t in (cache.block_table, cache.lens, cache.free_pages, cache.n_free, cache.shares)]


def unchanged(cache, before):
    import blockwise_exact_attention_gb300 as bea
    return all(torch.equal(a, b) for a, b in zip(state(cache), before)) and bea.device_status() == 0


def test_pages_that_cannot_be_copied():
    """Heads of 4 bf16 elements, whose rows are not of 16 bytes; and caches that were put in the place of the first ones."""
    import blockwise_exact_attention_gb300 as bea
    cache = bea.PagedKVCache(12, 4, 1, 4, 4, 16, share_pages=True)
    cache.plan(i32([5, 9, 0, 0]), 14)
    cache.plan(i32([-1, 0, 0, 0]), 0)                    # pages 0 and 1 are holes now
    before = state(cache)
    with pytest.raises(bea._lib.BeaError, match="UNSUPPORTED|ALIGN"):
        cache.fork(i32([-1, -1, 1, -1]))
    assert unchanged(cache, before)
    with pytest.raises(bea._lib.BeaError, match="UNSUPPORTED|ALIGN"):
        cache.compact(3)
    assert unchanged(cache, before)
    cache = bea.PagedKVCache(12, 4, 1, 64, 4, 16, share_pages=True)
    cache.plan(i32([5, 9, 0, 0]), 14)
    cache.plan(i32([-1, 0, 0, 0]), 0)
    before = state(cache)
    cache.v = cache.v[:1].expand(12, 4, 1, 64)
    for step in (lambda: cache.fork(i32([-1, -1, 1, -1])), lambda: cache.compact(3)):
        with pytest.raises(bea._lib.BeaError, match="ARG"):
            step()
        assert unchanged(cache, before)


def test_a_capacity_that_is_none():
    """The rows that end are not freed by a plan that raises."""
    import blockwise_exact_attention_gb300 as bea
    cache = bea.PagedKVCache(12, 4, 1, 64, 4, 16, share_pages=True)
    cache.plan(i32([5, 9, 0, 0]), 14)
    before = state(cache)
    for capacity in (-1, -100, 2.5, None, "many", 2 ** 62):
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            cache.plan(i32([-1, 1, 0, 0]), capacity)
        assert unchanged(cache, before), capacity
    plan = cache.plan(i32([-1, 1, 0, 0]), 1)
    assert plan.lens.tolist() == [0, 10, 0, 0] and cache.n_free.item() == 9
