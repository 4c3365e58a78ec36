"""A paged K/V cache: from request lengths to the attention of one new token.

A serving step is ``paged_plan`` (which pages and slots the new tokens get),
``paged_write`` (their keys and values into the cache) and ``paged_decode``
(each request's newest token against its pages). The calls take the caller's
tensors and keep nothing; ``PagedKVCache`` holds a cache's tensors and passes
them on. All of it runs on the GPU: a step needs no lengths on the host, so it
can be captured into a CUDA graph and replayed.

Requests may share pages: ``paged_fork`` lets rows begin as other rows' copies,
``paged_free`` ends rows and gives back the pages that nobody holds any more,
``paged_compact`` moves the used pages to the lower end of the cache, and
``paged_copy`` carries out the copies that the first and the last list.
``paged_decode_shared`` reads the keys that a group of rows shares once for all.
"""

from __future__ import annotations

import math
from typing import NamedTuple

import torch

from . import _lib


class PagedPlan(NamedTuple):
    slot_map: torch.Tensor   # [capacity] i32, -1 behind the last added token
    positions: torch.Tensor  # [capacity] i32, 0 behind the last
    cu_new: torch.Tensor     # [n + 1] i32, added tokens before each request
    cu_pages: torch.Tensor   # [n + 1] i32, new pages before each request
    lens: torch.Tensor       # [n] i32, the new lengths
    n_free: torch.Tensor     # [1] i32, free pages left


def paged_plan(lens, new_lens, block_table, free_pages, n_free, page_size, capacity, out=None) -> PagedPlan:
    """One scheduling step from request lengths (all int32, on the GPU).

    Request r holds ``lens[r]`` tokens and adds ``new_lens[r]`` (-1: it ends and
    its pages go back). ``block_table`` [n, max_pages] and the stack
    ``free_pages`` (height ``n_free`` [1]) are updated in place; ``lens`` and
    ``n_free`` are not, unless ``out`` (a PagedPlan) holds them as its own.
    ``capacity``: places for added tokens. A step that cannot be done in full
    changes nothing and is reported by ``device_status``. Every page is taken to
    be owned by one row: all pages of a row that ends go on the stack, also those
    that another row shares for reading, which the caller has to prevent."""
    return PagedPlan._make(_lib.bind().paged_plan(lens, new_lens, block_table, free_pages, n_free, page_size, capacity, out))


def paged_write(k, v, slot_map, k_cache, v_cache):
    """Write k, v [n, l, h_kv, d] to the slots ``slot_map`` [n * l] (int32, -1:
    not written) of the caches [num_pages, page_size, h_kv, d], in place."""
    return _lib.bind().paged_write(k, v, slot_map, k_cache, v_cache)


def paged_decode_workspace_bytes(q, k_cache, block_table) -> int:
    return int(_lib.load().bea_paged_decode_workspace_size(q.shape[2], k_cache.shape[2], q.shape[3],
                                                           block_table.shape[1] * k_cache.shape[1]))


def paged_decode(q, k_cache, v_cache, block_table, lens, softmax_scale=None, window_left=-1, out=None, lse=None,
                 out_dtype=None, workspace=None):
    """Attention of one new token per request: q [n, 1, h, d] against the keys
    and values of request r's first ``lens[r]`` slots (the new token's own among
    them) -> (out [n, 1, h, d], lse [n, h, 1] fp32). ``window_left`` >= 0 lets
    the token see only that many keys before its own. No gradient."""
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(q.shape[-1])
    if out_dtype is not None and out_dtype not in (q.dtype, torch.float32):
        raise TypeError(f"out_dtype {out_dtype}: {q.dtype} or float32")
    return _lib.bind().paged_decode(q, k_cache, v_cache, block_table, lens, softmax_scale, window_left, out, lse,
                                    out_dtype is torch.float32, workspace)


def paged_decode_shared_workspace_bytes(q, k_cache, block_table, shared_lens) -> int:
    return int(_lib.load().bea_paged_decode_shared_workspace_size(q.shape[0], q.shape[2], k_cache.shape[2], q.shape[3],
                                                                  block_table.shape[1] * k_cache.shape[1],
                                                                  shared_lens.shape[0]))


def paged_decode_shared(q, k_cache, v_cache, block_table, lens, group_rows, shared_lens, softmax_scale=None, out=None,
                        lse=None, out_dtype=None, workspace=None):
    """``paged_decode`` (bf16, no window) where groups of requests have their first
    keys in common, which are then read once for the group. Group g is the rows
    ``group_rows[g]`` .. ``group_rows[g + 1] - 1`` ([groups + 1] int32, ascending);
    their tables name the same pages for the first ``shared_lens[g]`` keys
    ([groups] int32), as those of forked rows do. Rows of length 0 take no part, and a
    row that names other pages than the group's first reads its keys for itself. The
    page that a forked prompt ends in may be counted in or not: it is not shared.

    The table's width decides whether groups are looked at: only where (n - 1) rows of
    it have room for 96 MB of keys and values, which sharing could save. A table much
    wider than its lengths takes the slower way for few requests; narrow it
    (``block_table[:, :pages]``) where the longest length is known.

    In the product with the values weights of shared keys have 16 bits, where
    ``paged_decode``'s have 24: a bf16 output is as exact, a float32 one is within
    2**-14 of sum(p |v|)."""
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(q.shape[-1])
    if out_dtype is not None and out_dtype not in (q.dtype, torch.float32):
        raise TypeError(f"out_dtype {out_dtype}: {q.dtype} or float32")
    return _lib.bind().paged_decode_shared(q, k_cache, v_cache, block_table, lens, group_rows, shared_lens, softmax_scale,
                                           out, lse, out_dtype is torch.float32, workspace)


class PagedFork(NamedTuple):
    lens: torch.Tensor    # [n] i32, the new lengths
    n_free: torch.Tensor  # [1] i32, free pages left
    shares: torch.Tensor  # [num_pages] i32, owners of a page beyond the first
    copies: torch.Tensor  # [n, 3] i32, (page, new page, tokens); tokens 0: none, -1: not a fork


class PagedFreed(NamedTuple):
    lens: torch.Tensor    # [n] i32, 0 for the rows that ended
    n_free: torch.Tensor  # [1] i32
    shares: torch.Tensor  # [num_pages] i32


class PagedCompaction(NamedTuple):
    block_table: torch.Tensor  # [n, max_pages] i32
    shares: torch.Tensor       # [num_pages] i32
    free_pages: torch.Tensor   # [F] i32, the lowest page on top, -1 behind the last
    page_map: torch.Tensor     # [num_pages] i32, where each page went
    copies: torch.Tensor       # [capacity, 3] i32, (page, new page, page_size) of every move, then -1


def paged_fork(src, tokens, lens, block_table, shares, free_pages, n_free, page_size, out=None) -> PagedFork:
    """Rows begin as copies of other rows, on their pages (all int32, on the GPU).

    ``src`` [n]: the row that row r forks from, -1 for rows that take no part; row
    r has to be free, and its source may not fork itself. ``tokens`` [n] (or None):
    how many of the source's first tokens it takes, -1 for all. ``shares``
    [num_pages] counts a page's owners beyond the first. Full pages are shared; a
    page that a fork ends in is copied to one of its own (``copies``, for
    ``paged_copy``). ``block_table`` is updated in place; ``lens``, ``n_free`` and
    ``shares`` are not, unless ``out`` (a PagedFork) holds them as its own. A step
    that cannot be done in full changes nothing and is reported by
    ``device_status``."""
    return PagedFork._make(_lib.bind().paged_fork(src, tokens, lens, block_table, shares, free_pages, n_free, page_size,
                                                  *(out or (None,) * 4)))


def paged_free(ends, lens, block_table, shares, free_pages, n_free, page_size, out=None) -> PagedFreed:
    """Rows r with ``ends[r]`` < 0 end; their pages that no other row holds go on the
    stack ``free_pages``, in place, in ascending order. For tables with shared
    pages, before ``paged_plan``, whose ``new_lens`` can be passed as ``ends``.
    ``lens``, ``n_free`` and ``shares`` are not changed, unless ``out`` (a
    PagedFreed) holds them as its own."""
    return PagedFreed._make(_lib.bind().paged_free(ends, lens, block_table, shares, free_pages, n_free, page_size,
                                                   *(out or (None,) * 3)))


def paged_compact(lens, block_table, shares, free_pages, n_free, page_size, capacity, out=None) -> PagedCompaction:
    """Moves used pages into lower free ones, at most ``capacity`` of them: the
    lowest free page takes the highest used one's place, and so on. Pages that are
    not on the stack count as used. Nothing is changed in place, unless ``out`` (a
    PagedCompaction) holds the tensors as its own. The contents follow by
    ``paged_copy`` with ``copies``, before anything else writes the cache."""
    return PagedCompaction._make(_lib.bind().paged_compact(lens, block_table, shares, free_pages, n_free, page_size,
                                                           capacity, *(out or (None,) * 5)))


def paged_copy(copies, caches):
    """Copy pages within every one of ``caches`` (a list of [num_pages, page_size,
    h_kv, d] tensors of one shape: keys and values of all layers), in place.
    ``copies`` [m, 3] int32: (page, new page, how many of its first tokens), tokens
    <= 0: no copy. Returns the caches."""
    _lib.bind().paged_copy(copies, caches)
    return caches


class PagedKVCache:
    """The tensors of one paged cache and its requests.

    ``num_pages`` pages of ``page_size`` tokens, up to ``max_requests`` requests
    (rows) of at most ``max_len`` tokens. A row is free while its length is 0.
    ``share_pages``: rows may share pages (``fork``, ``compact``); their owners are
    counted in ``shares``, and requests end through ``paged_free``."""

    def __init__(self, num_pages, page_size, h_kv, d, max_requests, max_len, dtype=torch.bfloat16, device="cuda",
                 share_pages=False):
        i32 = dict(dtype=torch.int32, device=device)
        self.page_size = page_size
        self.k = torch.empty(num_pages, page_size, h_kv, d, dtype=dtype, device=device)
        self.v = torch.empty_like(self.k)
        self.block_table = torch.full((max_requests, -(-max_len // page_size)), -1, **i32)
        self.lens = torch.zeros(max_requests, **i32)
        self.free_pages = torch.arange(num_pages - 1, -1, -1, **i32)  # page 0 is handed out first
        self.n_free = torch.full((1,), num_pages, **i32)
        self.shares = torch.zeros(num_pages, **i32) if share_pages else None

    def plan(self, new_lens, capacity) -> PagedPlan:
        """``paged_plan`` on this cache, its lengths and stack updated in place.
        Where pages are shared, the rows that end (-1) are freed first, also if the
        plan then refuses the rest."""
        if not 0 <= capacity < 2**31:
            raise ValueError(f"capacity {capacity}")
        n, dev = self.lens.shape[0], self.lens.device
        slots, positions, cu_new, cu_pages = torch.empty(2 * (capacity + n + 1), dtype=torch.int32, device=dev).split(
            (capacity, capacity, n + 1, n + 1))
        if self.shares is not None:
            self.free(new_lens)
        return paged_plan(self.lens, new_lens, self.block_table, self.free_pages, self.n_free, self.page_size, capacity,
                          PagedPlan(slots, positions, cu_new, cu_pages, self.lens, self.n_free))

    def _counted(self):
        if self.shares is None:
            raise ValueError("this cache does not count its pages' owners: PagedKVCache(..., share_pages=True)")

    def _caches(self, caches, copies):
        """What a step copies in, refused before the step where ``paged_copy`` would refuse it behind it."""
        if caches is None:
            return paged_copy(copies[:0], [self.k, self.v])
        for c in caches:
            if c.shape[:2] != self.k.shape[:2]:
                raise ValueError(f"a cache of shape {tuple(c.shape)} beside one of {self.k.shape[0]} pages of {self.page_size} "
                                 "tokens")
        return paged_copy(copies[:0], caches)

    def free(self, ends):
        """``paged_free`` on this cache, in place."""
        self._counted()
        return paged_free(ends, self.lens, self.block_table, self.shares, self.free_pages, self.n_free, self.page_size,
                          PagedFreed(self.lens, self.n_free, self.shares))

    def fork(self, src, tokens=None, caches=None):
        """``paged_fork`` on this cache, in place, and its copies in ``caches`` (default: this cache's own two)."""
        self._counted()
        copies = torch.empty(len(self.lens), 3, dtype=torch.int32, device=self.lens.device)
        caches = self._caches(caches, copies)
        step = paged_fork(src, tokens, self.lens, self.block_table, self.shares, self.free_pages, self.n_free,
                          self.page_size, PagedFork(self.lens, self.n_free, self.shares, copies))
        paged_copy(step.copies, caches)
        return step

    def compact(self, capacity, caches=None) -> PagedCompaction:
        """``paged_compact`` on this cache, in place, and its copies in ``caches`` (default: this cache's own two)."""
        self._counted()
        i32 = dict(dtype=torch.int32, device=self.lens.device)
        copies = torch.empty(capacity, 3, **i32)
        caches = self._caches(caches, copies)
        step = paged_compact(self.lens, self.block_table, self.shares, self.free_pages, self.n_free, self.page_size, capacity,
                             PagedCompaction(self.block_table, self.shares, self.free_pages,
                                             torch.empty(len(self.shares), **i32), copies))
        paged_copy(step.copies, caches)
        return step

    def write(self, k, v, slot_map):
        paged_write(k, v, slot_map, self.k, self.v)

    def decode(self, q, softmax_scale=None, window_left=-1, **kw):
        """``paged_decode`` of one new token per row: q [max_requests, 1, h, d]."""
        return paged_decode(q, self.k, self.v, self.block_table, self.lens, softmax_scale, window_left, **kw)

    def decode_shared(self, q, group_rows, shared_lens, softmax_scale=None, **kw):
        """``paged_decode_shared`` of one new token per row. The table is ``max_len`` wide: few rows that are much shorter are
        decoded faster by ``decode``."""
        return paged_decode_shared(q, self.k, self.v, self.block_table, self.lens, group_rows, shared_lens, softmax_scale, **kw)
