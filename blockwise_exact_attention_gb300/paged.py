"""A paged K/V cache: from request lengths to the attention of one new token.

A serving step is ``paged_plan`` (which pages and slots the new tokens get),
``paged_write`` (their keys and values into the cache) and ``paged_decode``
(each request's newest token against its pages). The calls take the caller's
tensors and keep nothing; ``PagedKVCache`` holds a cache's tensors and passes
them on. All of it runs on the GPU: a step needs no lengths on the host, so it
can be captured into a CUDA graph and replayed.
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


class PagedKVCache:
    """The tensors of one paged cache and its requests.

    ``num_pages`` pages of ``page_size`` tokens, up to ``max_requests`` requests
    (rows) of at most ``max_len`` tokens. A row is free while its length is 0."""

    def __init__(self, num_pages, page_size, h_kv, d, max_requests, max_len, dtype=torch.bfloat16, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self.page_size = page_size
        self.k = torch.empty(num_pages, page_size, h_kv, d, dtype=dtype, device=device)
        self.v = torch.empty_like(self.k)
        self.block_table = torch.full((max_requests, -(-max_len // page_size)), -1, **i32)
        self.lens = torch.zeros(max_requests, **i32)
        self.free_pages = torch.arange(num_pages - 1, -1, -1, **i32)  # page 0 is handed out first
        self.n_free = torch.full((1,), num_pages, **i32)

    def plan(self, new_lens, capacity) -> PagedPlan:
        """``paged_plan`` on this cache, its lengths and stack updated in place."""
        n, dev = self.lens.shape[0], self.lens.device
        slots, positions, cu_new, cu_pages = torch.empty(2 * (capacity + n + 1), dtype=torch.int32, device=dev).split(
            (capacity, capacity, n + 1, n + 1))
        return paged_plan(self.lens, new_lens, self.block_table, self.free_pages, self.n_free, self.page_size, capacity,
                          PagedPlan(slots, positions, cu_new, cu_pages, self.lens, self.n_free))

    def write(self, k, v, slot_map):
        paged_write(k, v, slot_map, self.k, self.v)

    def decode(self, q, softmax_scale=None, window_left=-1, **kw):
        """``paged_decode`` of one new token per row: q [max_requests, 1, h, d]."""
        return paged_decode(q, self.k, self.v, self.block_table, self.lens, softmax_scale, window_left, **kw)
