"""The oracle of the calls on shared pages: the definitions on Python lists, page
by page, sharing no code with the kernels. Inputs are left as they are."""

from __future__ import annotations


def pages(tokens, page):
    return -(-tokens // page)


def fork(src, tokens, lens, table, shares, pool, n_free, page):
    """(lens, table, shares, n_free, copies, ok, all pages in range)."""
    n, width = len(lens), len(table[0]) if table else 0
    lens, table, shares = list(lens), [list(r) for r in table], list(shares)
    tokens = [-1] * n if tokens is None else tokens
    ok, takes = 0 <= n_free <= len(pool), {}
    for r, s in enumerate(src):
        if s == -1:
            continue
        if not 0 <= s < n or src[s] != -1 or lens[r] != 0 or not 0 <= lens[s] <= width * page or not -1 <= tokens[r] <= lens[s]:
            ok = False
            break
        takes[r] = lens[s] if tokens[r] < 0 else tokens[r]
    if ok:
        ok = sum(t % page != 0 for t in takes.values()) <= n_free
    copies, clean = [[-1, -1, -1] for _ in range(n)], True
    if not ok:
        return lens, table, shares, n_free, copies, False, True
    old = [list(r) for r in table]
    for r, t in takes.items():
        for j in range(t // page):
            table[r][j] = old[src[r]][j]
            if 0 <= table[r][j] < len(shares):
                shares[table[r][j]] += 1
            else:
                clean = False
        copies[r] = [-1, -1, 0]
        if t % page:
            n_free -= 1
            table[r][t // page] = new = pool[n_free]
            last = old[src[r]][t // page]
            if 0 <= new < len(shares) and 0 <= last < len(shares):
                copies[r] = [last, new, t % page]
            else:
                clean = False
        lens[r] = t
    return lens, table, shares, n_free, copies, True, clean


def free(ends, lens, table, shares, pool, n_free, page):
    """(lens, shares, pool, n_free, clean)."""
    lens, shares, pool = list(lens), list(shares), list(pool)
    width = len(table[0]) if table else 0
    if not 0 <= n_free <= len(pool):
        return lens, shares, pool, n_free, False
    clean = True
    for r, e in enumerate(ends):
        if e >= 0:
            continue
        if not 0 <= lens[r] <= width * page:
            clean = False
            continue
        for j in range(pages(lens[r], page)):
            if 0 <= table[r][j] < len(shares):
                shares[table[r][j]] -= 1
            else:
                clean = False
        lens[r] = 0
    for p, s in enumerate(shares):
        if s < 0:
            clean = clean and s == -1 and n_free < len(pool)
            shares[p] = 0
            if n_free < len(pool):
                pool[n_free] = p
                n_free += 1
    return lens, shares, pool, n_free, clean


def compact(lens, table, shares, pool, n_free, page, capacity):
    """(table, shares, pool, page map, copies, ok)."""
    table, shares, pool = [list(r) for r in table], list(shares), list(pool)
    width, count = len(table[0]) if table else 0, len(shares)
    stack = pool[:n_free] if 0 <= n_free <= len(pool) else [-1]
    where = list(range(count))
    if len(set(stack)) != len(stack) or not all(0 <= p < count for p in stack):
        return table, shares, pool, where, [[-1] * 3 for _ in range(capacity)], False
    holes, moves, clean = set(stack), [], True
    while len(moves) < capacity and holes:
        low, high = min(holes), max((p for p in range(count) if p not in holes), default=-1)
        if high < low:
            break
        holes.remove(low)
        holes.add(high)
        moves.append([high, low, page])
        where[high] = low
        shares[low], shares[high] = shares[high], 0
    for r, l in enumerate(lens):
        if not 0 <= l <= width * page:
            clean, l = False, 0 if l < 0 else width * page
        for j in range(pages(l, page)):
            if 0 <= table[r][j] < count:
                table[r][j] = where[table[r][j]]
            else:
                clean = False
    pool = sorted(holes, reverse=True) + [-1] * (len(pool) - n_free)
    return table, shares, pool, where, moves + [[-1] * 3 for _ in range(capacity - len(moves))], clean


def copy(copies, cache):
    """In place: cache[new][:tokens] = cache[old][:tokens] for (old, new, tokens) that fit; whether all did."""
    clean, before = True, cache.copy() if hasattr(cache, "copy") else cache.clone()
    for old, new, t in copies:
        if t <= 0:
            continue
        if not (0 <= old < len(cache) and 0 <= new < len(cache)) or old == new or t > cache.shape[1]:
            clean = False
            continue
        cache[new][:t] = before[old][:t]
    return clean


def owners(lens, table, count, page):
    """How many rows hold each page."""
    held = [0] * count
    for r, l in enumerate(lens):
        for j in range(pages(l, page)):
            held[table[r][j]] += 1
    return held
