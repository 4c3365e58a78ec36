"""The paged cache's and the rotary embedding's oracle: the definitions in
plain Python and fp64 numpy, token by token, sharing no code with the kernels."""

from __future__ import annotations

import math

import numpy as np


def rope_axes(x, positions, sections, base=10000.0, spectrum="joint", inverse=False):
    """x [n, l, h, d], positions [axes, n, l] -> x turned pair by pair, fp64."""
    x = np.asarray(x, dtype=np.float64)
    half = x.shape[-1] // 2
    y = np.empty_like(x)
    p = 0
    for a, pairs in enumerate(sections):
        for j in range(pairs):
            f = base ** -(2.0 * p / x.shape[-1]) if spectrum == "joint" else base ** -(j / pairs)
            ang = np.asarray(positions[a], dtype=np.float64)[:, :, None] * f
            if inverse:
                ang = -ang
            c, s = np.cos(ang), np.sin(ang)
            u, v = x[..., p], x[..., p + half]
            y[..., p] = u * c - v * s
            y[..., p + half] = v * c + u * s
            p += 1
    return y


def plan(lens, new_lens, table, pool, n_free, page, capacity):
    """One step on lists: (slot_map, positions, cu_new, cu_pages, lens, n_free,
    table, pool, ok); the inputs are left as they are."""
    lens, table, pool = list(lens), [list(r) for r in table], list(pool)
    n, width = len(lens), len(table[0]) if table else 0

    def pages(t):
        return -(-t // page)

    ok = 0 <= n_free <= len(pool)
    for l, a in zip(lens, new_lens):
        ok = ok and l >= 0 and a >= -1 and l + max(a, 0) <= width * page
    if ok:
        back = sum(pages(l) for l, a in zip(lens, new_lens) if a < 0)
        need = sum(pages(l + a) - pages(l) for l, a in zip(lens, new_lens) if a >= 0)
        ok = n_free + back <= len(pool) and need <= n_free + back and sum(max(a, 0) for a in new_lens) <= capacity
    slots, pos, cu, cup = [], [], [0], [0]
    if ok:
        for r in range(n):
            if new_lens[r] < 0:
                for j in range(pages(lens[r])):
                    pool[n_free] = table[r][j]
                    n_free += 1
                lens[r] = 0
        for r in range(n):
            taken = 0
            for i in range(max(new_lens[r], 0)):
                at = lens[r] + i
                if at % page == 0:
                    n_free -= 1
                    taken += 1
                    table[r][at // page] = pool[n_free]
                slots.append(table[r][at // page] * page + at % page)
                pos.append(at)
            cu.append(len(slots))
            cup.append(cup[-1] + taken)
        lens = [l + max(a, 0) for l, a in zip(lens, new_lens)]
    else:
        cu, cup = [0] * (n + 1), [0] * (n + 1)
    slots += [-1] * (capacity - len(slots))
    pos += [0] * (capacity - len(pos))
    return slots, pos, cu, cup, lens, n_free, table, pool, ok


def decode(q, k_cache, v_cache, table, lens, scale, left=-1):
    """q [n, 1, h, d], caches [pages, page, h_kv, d] -> (out, lse, A, S): fp64
    output and log-sum-exp, and per row A = sum_j p_j |v_j| and S = the largest
    scale * sum_i |q_i k_i|, which scale the rounding bounds. Keys in pages
    outside the cache are masked."""
    n, _, h, d = q.shape
    page, h_kv = k_cache.shape[1], k_cache.shape[2]
    width = table.shape[1] * page
    out, a = np.zeros((n, 1, h, d)), np.zeros((n, 1, h, d))
    lse, big = np.full((n, h, 1), -np.inf), np.zeros((n, h, 1))
    for r in range(n):
        length = min(max(int(lens[r]), 0), width)
        first = 0 if left < 0 else max(0, length - 1 - left)
        at = [(int(table[r, j // page]), j % page) for j in range(first, length)]
        at = [(i, o) for i, o in at if 0 <= i < k_cache.shape[0]]
        if not at:
            continue
        ids, offs = np.array(at).T
        k = k_cache[ids, offs].astype(np.float64)
        v = v_cache[ids, offs].astype(np.float64)
        for i in range(h):
            kv = i // (h // h_kv)
            x = q[r, 0, i].astype(np.float64)
            s = scale * (k[:, kv] @ x)
            m = s.max()
            if m == -np.inf:
                continue
            e = np.exp(s - m)
            lse[r, i, 0] = m + math.log(e.sum())
            p = e / e.sum()
            out[r, 0, i] = p @ v[:, kv]
            a[r, 0, i] = p @ np.abs(v[:, kv])
            big[r, i, 0] = scale * (np.abs(k[:, kv]) @ np.abs(x)).max()
    return out, lse, a, big
