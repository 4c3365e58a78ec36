"""What the operators of requests that share pages, and of normed and laid-out
rotary positions, are measured on.

``paged_decode_shared`` (attention of one new token per request, a group's
common first keys read once for all its requests), ``paged_fork`` /
``paged_free`` / ``paged_compact`` with ``paged_copy`` (the pages of a cache
whose requests share them), ``norm_rope_axes`` (RMS norm of every head of q and
k and the rotation in one pass, forward and gradient) and ``rope_axes`` with
interleaved pairs, a part of the head and scaled frequencies. ``run`` computes
a case in its plain form, elementary torch operations in 32 bits (angles in
64), or, where ``own`` is set, by the calls a program makes of this package.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ---- the cases -----------------------------------------------------------------


def listed():
    return [
        # four answers to one prompt, shortly after it: the smallest call, where latency counts
        dict(name="shared_few", op="shared", n=4, groups=1, shared=2000, tail=64, h=32, h_kv=8, d=128, page=16,
             lens_seed=1),
        # a serving batch behind one long document, each request with its own question and answer so far
        dict(name="shared_document", op="shared", n=64, groups=1, shared=32768, tail=1024, h=32, h_kv=8, d=128, page=16,
             lens_seed=2),
        # three system prompts served side by side, one query head per K/V head, pages that divide no tile
        dict(name="shared_three_prompts", op="shared", n=96, groups=3, shared=6000, tail=3000, h=16, h_kv=16, d=64,
             page=24, lens_seed=3),
        # many samples of one long prompt: the shared keys meet 1024 queries a K/V head, products count
        dict(name="shared_samples", op="shared", n=256, groups=1, shared=16384, tail=600, h=32, h_kv=8, d=128, page=64,
             lens_seed=4),
        # a small beam search step: six rows start anew from two others
        dict(name="fork_beams", op="fork", n=8, sources=2, forks=6, max_len=700, page=16, layers=2, h_kv=8, d=128,
             dtype="bf16", lens_seed=5),
        # 200 samples forked from eight prompts, their last pages copied in every layer
        dict(name="fork_samples", op="fork", n=256, sources=8, forks=200, max_len=8192, page=32, layers=4, h_kv=8,
             d=128, dtype="bf16", lens_seed=6),
        # requests of a large batch end, some of whose pages others still hold
        dict(name="free_step", op="free", n=512, groups=7, max_len=8192, ends=0.15, page=16, lens_seed=7),
        # a cache left with holes, its upper pages moved down
        dict(name="compact_cache", op="compact", n=64, max_len=2048, holes=0.4, page=16, layers=2, h_kv=8, d=128,
             dtype="bf16", lens_seed=8),
        # q and k of 256 new tokens
        dict(name="norm_rope_decode_step", op="rope", n=256, l=1, h=32, h_kv=8, d=128, rotary=128, dtype="bf16",
             norm=True, interleaved=False, scaling="none", train=False),
        # a training step on a long sequence: forward, gradients of q, k and both weights
        dict(name="norm_rope_train", op="rope", n=1, l=32768, h=32, h_kv=8, d=128, rotary=128, dtype="bf16", norm=True,
             interleaved=False, scaling="none", train=True),
        # fp32 training on a few short odd sequences, half of the head turned, pairs interleaved, scaled for length
        dict(name="norm_rope_partial_f32_train", op="rope", n=3, l=1369, h=12, h_kv=12, d=64, rotary=32, dtype="f32",
             norm=True, interleaved=True, scaling="yarn", train=True),
        # a prompt far past the trained length: interleaved pairs without norms, frequencies scaled by parts
        dict(name="rope_interleaved_prompt", op="rope", n=2, l=16384, h=32, h_kv=8, d=128, rotary=64, dtype="bf16",
             norm=False, interleaved=True, scaling="yarn", train=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "shared", "fork", "free", "compact", "rope", "rope", "rope"])
    seed = rng.randrange(1 << 30)
    if op == "shared":
        h_kv = rng.choice([1, 2, 3, 4, 8, 16])
        h = h_kv * rng.choice([1, 2, 3, 4, 5, 8, 16] if h_kv <= 4 else [1, 2, 4])
        d = rng.choice([64, 128])
        n = _log(rng, 2, 256)
        # at most 2^27 (query head, shared key) pairs and 2^20 own keys
        most = max(128, min(65536, 2**27 // (n * h)))
        return dict(op="shared", n=n, groups=min(n, rng.choice([1, 1, 1, 2, 5])), shared=_log(rng, 64, most),
                    tail=_log(rng, 1, min(4096, 2**20 // n)), h=h, h_kv=h_kv, d=d,
                    page=rng.choice([1, 8, 16, 16, 20, 32, 64, 100, 128]), lens_seed=seed)
    if op in ("fork", "compact"):
        page = rng.choice([1, 8, 16, 20, 32, 64])
        layers, h_kv, d = rng.choice([1, 2, 4, 7]), rng.choice([1, 2, 3, 8]), rng.choice([64, 128])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        row = layers * 2 * h_kv * d * (2 if dtype == "bf16" else 4)
        if op == "compact":
            n = _log(rng, 1, 300)
            max_len = _log(rng, 16, max(32, min(8192, 2**30 // (row * n), 2**16 * page // n)))
            return dict(op="compact", n=n, max_len=max_len, holes=rng.choice([0.05, 0.3, 0.6]), page=page,
                        layers=layers, h_kv=h_kv, d=d, dtype=dtype, lens_seed=seed)
        sources = _log(rng, 1, 40)
        forks = _log(rng, 1, 400)
        max_len = _log(rng, 16, max(32, min(16384, 2**29 // (row * (sources + 8)), 2**16 * page // (sources + 8))))
        return dict(op="fork", n=sources + forks + rng.randrange(0, 20), sources=sources, forks=forks, max_len=max_len,
                    page=page, layers=layers, h_kv=h_kv, d=d, dtype=dtype, lens_seed=seed)
    if op == "free":
        n = _log(rng, 1, 1200)
        page = rng.choice([1, 8, 16, 20, 32, 64])
        return dict(op="free", n=n, groups=rng.randint(1, min(n, 20)), max_len=_log(rng, 16, max(32, min(16384, 2**19 * page // n))),
                    ends=rng.choice([0.02, 0.2, 0.7]), page=page, lens_seed=seed)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([32, 64, 80, 96, 128, 256])
    h_kv = rng.choice([1, 2, 3, 8, 12])
    h = h_kv * rng.choice([1, 2, 4])
    n = _log(rng, 1, 300)
    l = _log(rng, 1, max(1, min(20000, 2**27 // (n * (h + h_kv) * d))))
    norm = rng.random() < 0.7
    return dict(op="rope", n=n, l=l, h=h, h_kv=h_kv, d=d, rotary=rng.choice([d, d, d // 32 * 16]), dtype=dtype, norm=norm,
                interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                train=rng.random() < 0.5)


def _pages(tokens, page):
    return -(-tokens // page)


def _esize(case):
    return 2 if case["dtype"] == "bf16" else 4


def _shared(case):
    """(first row of every group and the end, shared tokens of every group, lengths of all rows)."""
    rng = random.Random(case["lens_seed"])
    n, groups, page = case["n"], case["groups"], case["page"]
    cuts = [n * g // groups for g in range(groups + 1)]
    shared, lens = [], [0] * n
    for g in range(groups):
        s = case["shared"] if groups == 1 else rng.randint(case["shared"] // 2, case["shared"])
        shared.append(s // page * page)
        for r in range(cuts[g], cuts[g + 1]):
            lens[r] = shared[g] + _log(rng, 1, case["tail"])
    if n > 40:
        lens[n // 3] = 0  # a row without a request
    return cuts, shared, lens


def _fork(case):
    """(src, tokens, lens): sources first, then rows that fork, then rows that have nothing to do with it."""
    rng = random.Random(case["lens_seed"])
    n, s, f = case["n"], case["sources"], case["forks"]
    lens = [rng.randint(max(1, case["max_len"] // 2), case["max_len"]) for _ in range(s)] + [0] * (n - s)
    src, tokens = [-1] * n, [-1] * n
    for r in range(s, s + f):
        src[r] = rng.randrange(s)
        if rng.random() < 0.25:
            tokens[r] = rng.randint(0, lens[src[r]])
    for r in range(s + f, n):
        lens[r] = rng.randint(1, case["page"] * 2)
    return src, tokens, lens


def _free(case):
    """(group of every row, shared pages of every group, lens, ends)."""
    rng = random.Random(case["lens_seed"])
    n, groups = case["n"], case["groups"]
    top = max(1, case["max_len"] // case["page"])
    pages = [rng.randint(0, top // 2) for _ in range(groups)]
    group, lens, ends = [], [], []
    for r in range(n):
        g = rng.randrange(groups)
        group.append(g)
        lens.append(min(case["max_len"], pages[g] * case["page"] + rng.randint(1, max(1, case["max_len"] // 2))))
        ends.append(-1 if rng.random() < case["ends"] else rng.choice([0, 1]))
    ends[0] = -1
    if n > 3:
        lens[n // 2] = 0
    return group, pages, lens, ends


def _compact(case):
    rng = random.Random(case["lens_seed"])
    lens = [_log(rng, 1, case["max_len"]) for _ in range(case["n"])]
    used = sum(_pages(l, case["page"]) for l in lens)
    pages = max(used + 1, int(used / (1 - case["holes"])))
    # which pages are used: any, by the case alone, so that its work is too
    ids = rng.sample(range(pages), pages)
    return lens, used, pages, ids


def _moves(ids, used):
    taken, holes = sorted(ids[:used], reverse=True), sorted(ids[used:])
    return sum(1 for a, b in zip(taken, holes) if b < a)


def work(case):
    op = case["op"]
    if op == "shared":
        cuts, shared, lens = _shared(case)
        h, h_kv, d, n, page = case["h"], case["h_kv"], case["d"], case["n"], case["page"]
        keys = pages = 0
        for g, s in enumerate(shared):
            live = [l for l in lens[cuts[g]:cuts[g + 1]] if l > 0]
            keys += (s if live else 0) + sum(l - s for l in live)
            pages += s // page + sum(_pages(l - s, page) for l in live)
        return {"bytes": keys * h_kv * d * 2 * 2 + 4 * (pages + n) + 2 * n * h * d * 2 + n * h * 4,
                "flops": 4 * sum(lens) * h * d}
    if op == "fork":
        src, tokens, lens = _fork(case)
        took = [lens[s] if t < 0 else t for s, t in zip(src, tokens) if s >= 0]
        page, n = case["page"], case["n"]
        row = case["layers"] * 2 * case["h_kv"] * case["d"] * _esize(case)
        entries = sum(_pages(t, page) for t in took)
        return {"bytes": 2 * row * sum(t % page for t in took) + 8 * entries + 4 * (7 * n + 2), "flops": 0}
    if op == "free":
        _, _, lens, ends = _free(case)
        entries = sum(_pages(l, case["page"]) for l, e in zip(lens, ends) if e < 0)
        return {"bytes": 8 * entries + 4 * (3 * case["n"] + 2), "flops": 0}
    if op == "compact":
        lens, used, pages, ids = _compact(case)
        moves = _moves(ids, used)
        row = case["layers"] * 2 * case["page"] * case["h_kv"] * case["d"] * _esize(case)
        return {"bytes": 2 * row * moves + 8 * used + 8 * (pages - used) + 12 * pages + 12 * moves, "flops": 0}
    rows = case["n"] * case["l"] * (case["h"] + case["h_kv"])
    elems, e, pos = rows * case["d"], _esize(case), 4 * case["n"] * case["l"]
    each = (3 if case["rotary"] else 0) + (4 if case["norm"] else 0)
    if not case["train"]:
        return {"bytes": 2 * elems * e + pos, "flops": each * elems}
    # the gradient reads the input once more where the norm's needs it
    back = 3 if case["norm"] else 2
    return {"bytes": (2 + back) * elems * e + 2 * pos, "flops": (each + each * 2) * elems}


# ---- inputs --------------------------------------------------------------------


def _i32(x, dev="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _caches(case, pages, g):
    shape = (pages, case["page"], case["h_kv"], case["d"])
    return [torch.randn(shape, dtype=DTYPES[case["dtype"]], device="cuda", generator=g)
            for _ in range(2 * case["layers"])]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    host = random.Random(int(seed))
    dev = torch.device("cuda")
    s = dict(case)
    op = case["op"]

    def normal(*shape, dtype):
        return torch.randn(*shape, dtype=dtype, device=dev, generator=g)

    if op == "shared":
        cuts, shared, lens = _shared(case)
        n, page = case["n"], case["page"]
        width = max(1, _pages(max(lens), page))
        rows, total = [], 0
        for gr, sh in enumerate(shared):
            first, total = list(range(total, total + sh // page)), total + sh // page
            for l in lens[cuts[gr]:cuts[gr + 1]]:
                mine = max(0, _pages(l, page) - len(first))
                rows.append((first + list(range(total, total + mine)) if l > 0 else []))
                total += mine
        ids = list(range(total + 3))
        host.shuffle(ids)
        table = torch.full((n, width), -1, dtype=torch.int32)
        order = torch.tensor(ids, dtype=torch.int32)
        for r, row in enumerate(rows):
            if row:
                table[r, :len(row)] = order[torch.tensor(row)]
        cache = (total + 3, page, case["h_kv"], case["d"])
        bf = torch.bfloat16
        s |= {"q": normal(n, 1, case["h"], case["d"], dtype=bf), "k_cache": normal(*cache, dtype=bf),
              "v_cache": normal(*cache, dtype=bf), "block_table": table.to(dev), "lens": _i32(lens),
              "group_rows": _i32(cuts), "shared_lens": _i32(shared), "cuts": cuts, "prefix": shared,
              "scale": 1.0 / math.sqrt(case["d"])}
    elif op == "fork":
        src, tokens, lens = _fork(case)
        n, page = case["n"], case["page"]
        width = _pages(case["max_len"], page) + 2
        counts = [_pages(l, page) for l in lens]
        used = sum(counts)
        pages = used + case["forks"] + 5
        ids = list(range(pages))
        host.shuffle(ids)
        table = torch.full((n, width), -1, dtype=torch.int32)
        at = 0
        for r, c in enumerate(counts):
            table[r, :c] = torch.tensor(ids[at:at + c], dtype=torch.int32)
            at += c
        free = ids[used:] + [-1] * used
        s |= {"src": _i32(src), "tokens": _i32(tokens), "lens": _i32(lens), "block_table": table.to(dev),
              "shares": torch.zeros(pages, dtype=torch.int32, device=dev), "free_pages": _i32(free),
              "n_free": _i32([pages - used]), "caches": _caches(case, pages, g)}
    elif op == "free":
        group, first, lens, ends = _free(case)
        n, page = case["n"], case["page"]
        width = _pages(case["max_len"], page)
        starts, total = [], 0
        for c in first:
            starts.append(total)
            total += c
        rows = []
        for gr, l in zip(group, lens):
            c = _pages(l, page)
            common = min(c, first[gr])
            rows.append(list(range(starts[gr], starts[gr] + common)) + list(range(total, total + c - common)))
            total += c - common
        owners = torch.zeros(total, dtype=torch.int32)
        for row in rows:
            owners[torch.tensor(row, dtype=torch.long)] += 1
        pages = total + 9
        ids = list(range(pages))
        host.shuffle(ids)
        order = torch.tensor(ids, dtype=torch.int32)
        table = torch.full((n, width), -1, dtype=torch.int32)
        for r, row in enumerate(rows):
            table[r, :len(row)] = order[torch.tensor(row, dtype=torch.long)]
        shares = torch.zeros(pages, dtype=torch.int32)
        shares[order[:total].long()] = (owners - 1).clamp(min=0)
        # pages that no row holds any more (a group without a row) are free
        none = [ids[p] for p in range(total) if int(owners[p]) == 0]
        pool = ids[total:] + none
        free = pool + [-1] * (pages - len(pool))
        s |= {"ends": _i32(ends), "lens": _i32(lens), "block_table": table.to(dev), "shares": shares.to(dev),
              "free_pages": _i32(free), "n_free": _i32([len(pool)])}
    elif op == "compact":
        lens, used, pages, ids = _compact(case)
        n, page = case["n"], case["page"]
        width = _pages(case["max_len"], page)
        mine = ids[:used]
        host.shuffle(mine)
        table = torch.full((n, width), -1, dtype=torch.int32)
        at = 0
        for r, l in enumerate(lens):
            c = _pages(l, page)
            table[r, :c] = torch.tensor(mine[at:at + c], dtype=torch.int32)
            at += c
        pool = ids[used:]
        host.shuffle(pool)
        s |= {"lens": _i32(lens), "block_table": table.to(dev), "free_pages": _i32(pool + [-1] * used),
              "shares": torch.zeros(pages, dtype=torch.int32, device=dev), "n_free": _i32([pages - used]),
              "capacity": pages // 2, "caches": _caches(case, pages, g)}
    else:
        dt = DTYPES[case["dtype"]]
        n, l, d = case["n"], case["l"], case["d"]
        q, k = (n, l, case["h"], d), (n, l, case["h_kv"], d)
        start = torch.randint(0, 100000, (n, 1), device=dev, generator=g)
        pos = torch.arange(l, device=dev)[None, :] + start
        s |= {"q": normal(*q, dtype=dt).requires_grad_(case["train"]),
              "k": normal(*k, dtype=dt).requires_grad_(case["train"]),
              "positions": pos[None].to(torch.int32).contiguous()}
        if case["norm"]:
            s |= {"q_weight": (1 + 0.1 * normal(d, dtype=torch.float32)).to(dt).requires_grad_(case["train"]),
                  "k_weight": (1 + 0.1 * normal(d, dtype=torch.float32)).to(dt).requires_grad_(case["train"])}
        if case["train"]:
            s |= {"dq": normal(*q, dtype=dt), "dk": normal(*k, dtype=dt)}
    return s


# ---- one pass ------------------------------------------------------------------


def run(s):
    return _own(s) if own else _plain(s)


SCALING = {"linear": dict(kind="linear", factor=4.0), "ntk": dict(kind="ntk", factor=4.0),
           "yarn": dict(kind="yarn", factor=8.0, original_max=4096)}


def _own(s):
    import blockwise_exact_attention_gb300 as bea

    op = s["op"]
    if op == "shared":
        return bea.paged_decode_shared(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["lens"],
                                       s["group_rows"], s["shared_lens"], s["scale"])
    if op == "fork":
        f = bea.paged_fork(s["src"], s["tokens"], s["lens"], s["block_table"], s["shares"], s["free_pages"],
                           s["n_free"], s["page"])
        caches = bea.paged_copy(f.copies, s["caches"])
        return (f.lens, f.shares, f.n_free, f.copies, s["block_table"], *caches)
    if op == "free":
        f = bea.paged_free(s["ends"], s["lens"], s["block_table"], s["shares"], s["free_pages"], s["n_free"], s["page"])
        return f.lens, f.shares, f.n_free, s["free_pages"]
    if op == "compact":
        c = bea.paged_compact(s["lens"], s["block_table"], s["shares"], s["free_pages"], s["n_free"], s["page"],
                              s["capacity"])
        caches = bea.paged_copy(c.copies, s["caches"])
        return (c.block_table, c.shares, c.free_pages, c.page_map, c.copies, *caches)
    scaling = None if s["scaling"] == "none" else bea.RopeScaling(**SCALING[s["scaling"]])
    how = dict(sections=(s["rotary"] // 2,), rotary_dim=s["rotary"], layout="interleaved" if s["interleaved"] else "half",
               scaling=scaling)
    q, k, pos = s["q"], s["k"], s["positions"]
    if not s["train"]:
        if s["norm"]:
            return bea.norm_rope_axes(q, k, pos, q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, **how)
        return bea.rope_axes(q, k, pos, **how)
    if s["norm"]:
        qo, ko = bea.norm_rotary_axes(q, k, pos, q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, **how)
        leaves = (q, k, s["q_weight"], s["k_weight"])
    else:
        qo, ko = bea.rotary_axes(q, k, pos, **how)
        leaves = (q, k)
    return (qo.detach(), ko.detach(), *torch.autograd.grad((qo, ko), leaves, (s["dq"], s["dk"])))


def _plain(s):
    return {"shared": _plain_shared, "fork": _plain_fork, "free": _plain_free, "compact": _plain_compact,
            "rope": _plain_rope}[s["op"]](s)


def _plain_shared(s):
    q, lens, table, page = s["q"], s["lens"].long(), s["block_table"].long(), s["page"]
    n, _, h, d = q.shape
    h_kv = s["k_cache"].shape[2]
    qg = q.reshape(n, h_kv, h // h_kv, d).float()
    outs, lses = [], []
    for r0, r1, shared in zip(s["cuts"], s["cuts"][1:], s["prefix"]):
        rows, cols = r1 - r0, shared // page
        owner = r0 + (lens[r0:r1] > 0).to(torch.int32).argmax()
        first = table[owner, :cols].clamp(min=0)
        kp = s["k_cache"][first].reshape(shared, h_kv, d).float()
        vp = s["v_cache"][first].reshape(shared, h_kv, d).float()
        rest = table[r0:r1, cols:].clamp(min=0)
        kr = s["k_cache"][rest].reshape(rows, -1, h_kv, d).float()
        vr = s["v_cache"][rest].reshape(rows, -1, h_kv, d).float()
        key = torch.arange(shared + kr.shape[1], device=q.device)
        seen = key[None, :] < lens[r0:r1, None]
        # all of the group's queries against the shared keys in one product a head, each row's own keys apart
        x = qg[r0:r1].permute(1, 0, 2, 3)  # [h_kv, rows, g, d]
        grp = h // h_kv
        sp = torch.matmul(x.reshape(h_kv, rows * grp, d), kp.permute(1, 2, 0)).reshape(h_kv, rows, grp, shared)
        sr = torch.matmul(qg[r0:r1], kr.permute(0, 2, 3, 1)).permute(1, 0, 2, 3)
        score = torch.where(seen[None, :, None, :], torch.cat([sp, sr], -1) * s["scale"], -math.inf)
        top = score.max(-1, keepdim=True).values
        p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
        total = p.sum(-1, keepdim=True)
        vr = torch.where(seen[:, shared:, None, None], vr, 0.0)
        o = torch.matmul(p[..., :shared].reshape(h_kv, rows * grp, shared), vp.permute(1, 0, 2)).reshape(x.shape)
        o = o + torch.matmul(p[..., shared:].permute(1, 0, 2, 3), vr.permute(0, 2, 1, 3)).permute(1, 0, 2, 3)
        o = o / torch.where(total == 0, 1.0, total)
        lse = torch.where(total == 0, -math.inf, top + torch.log(total))
        outs.append(o.permute(1, 0, 2, 3).reshape(rows, 1, h, d))
        lses.append(lse.permute(1, 0, 2, 3).reshape(rows, h, 1))
    return torch.cat(outs).to(q.dtype), torch.cat(lses)


def _plain_copy(copies, caches, page):
    frm, to, tokens = copies.long().unbind(1)
    r, c = torch.nonzero(torch.arange(page, device=copies.device)[None, :] < tokens[:, None], as_tuple=True)
    for cache in caches:
        cache[to[r], c] = cache[frm[r], c]
    return caches


def _plain_fork(s):
    i32 = torch.int32
    src, lens, ps = s["src"].long(), s["lens"].long(), s["page"]
    table, free = s["block_table"].long().clone(), s["free_pages"].long()
    forked, frm = src >= 0, src.clamp(min=0)
    took = torch.where(forked, torch.where(s["tokens"] < 0, lens[frm], s["tokens"].long()), 0)
    full, part = took // ps, took % ps
    need = (part > 0).long()
    new = free[(s["n_free"].long() - 1 - (need.cumsum(0) - need)).clamp(min=0)]
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    old = table[frm]
    shared = col < full[:, None]
    shares = s["shares"].long().index_add(0, old[shared], torch.ones_like(old[shared]))
    table = torch.where(shared, old, table)
    table = torch.where((col == full[:, None]) & (need > 0)[:, None], new[:, None], table)
    last = old.gather(1, full[:, None].clamp(max=table.shape[1] - 1))[:, 0]
    copies = torch.where((need > 0)[:, None], torch.stack([last, new, part], 1), -1)
    copies[:, 2] = torch.where(forked & (need == 0), 0, copies[:, 2])
    lens = torch.where(forked, took, lens)
    caches = _plain_copy(copies, s["caches"], ps)
    return (lens.to(i32), shares.to(i32), (s["n_free"].long() - need.sum()).to(i32), copies.to(i32), table.to(i32),
            *caches)


def _plain_free(s):
    i32 = torch.int32
    lens, ps, table = s["lens"].long(), s["page"], s["block_table"].long()
    ended = s["ends"] < 0
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    given = table[ended[:, None] & (col < ((lens + ps - 1) // ps)[:, None])]
    left = s["shares"].long().index_add(0, given, -torch.ones_like(given))
    back = torch.nonzero(left < 0)[:, 0]
    free = s["free_pages"].clone()
    at = s["n_free"].long() + torch.arange(back.numel(), device=table.device)
    free[at] = back.to(i32)
    return (torch.where(ended, 0, lens).to(i32), left.clamp(min=0).to(i32), (s["n_free"] + back.numel()).to(i32), free)


def _plain_compact(s):
    i32 = torch.int32
    table, n_free = s["block_table"].long(), int(s["n_free"])
    pages = s["shares"].numel()
    dev = table.device
    is_free = torch.zeros(pages, dtype=torch.bool, device=dev)
    is_free[s["free_pages"].long()[:n_free]] = True
    holes = torch.nonzero(is_free)[:, 0]
    taken = torch.nonzero(~is_free)[:, 0].flip(0)
    m = min(holes.numel(), taken.numel())
    move = holes[:m] < taken[:m]
    move[s["capacity"]:] = False
    frm, to = taken[:m][move], holes[:m][move]
    page_map = torch.arange(pages, device=dev)
    page_map[frm] = to
    shares = s["shares"].clone()
    shares[to] = s["shares"][frm]
    shares[frm] = 0
    is_free[frm], is_free[to] = True, False
    free = torch.full_like(s["free_pages"], -1)
    free[:n_free] = torch.nonzero(is_free)[:, 0].flip(0).to(i32)
    ps = s["page"]
    col = torch.arange(table.shape[1], device=dev)[None, :]
    live = col < ((s["lens"].long() + ps - 1) // ps)[:, None]
    new_table = torch.where(live, page_map[table.clamp(min=0)], table)
    copies = torch.full((s["capacity"], 3), -1, dtype=torch.long, device=dev)
    copies[:frm.numel()] = torch.stack([frm, to, torch.full_like(frm, ps)], 1)
    caches = _plain_copy(copies, s["caches"], ps)
    return new_table.to(i32), shares, free, page_map.to(i32), copies.to(i32), *caches


def _turned(x, cos, sin, rotary, interleaved):
    a, b = (x[..., :rotary:2], x[..., 1:rotary:2]) if interleaved else (x[..., : rotary // 2], x[..., rotary // 2:rotary])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([y, x[..., rotary:]], -1)


def _plain_rope(s):
    dev, rotary, inter = s["q"].device, s["rotary"], s["interleaved"]
    half = rotary // 2
    pair = torch.arange(half, dtype=torch.float64, device=dev)
    base, amplitude = 10000.0, 1.0
    if s["scaling"] == "ntk" and half > 1:
        base = base * SCALING["ntk"]["factor"] ** (half / (half - 1))
    freq = torch.pow(base, -pair / half)
    if s["scaling"] == "linear":
        freq = freq / SCALING["linear"]["factor"]
    if s["scaling"] == "yarn":
        f, length = SCALING["yarn"]["factor"], SCALING["yarn"]["original_max"]
        keep = ((freq * length / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        freq = freq / f * (1 - keep) + freq * keep
        amplitude = 0.1 * math.log(f) + 1.0
    angle = s["positions"][0].double()[..., None] * freq
    cos = (angle.cos() * amplitude).float()[:, :, None]
    sin = (angle.sin() * amplitude).float()[:, :, None]
    outs, grads, wgrads = [], [], []
    for x, w, g in (("q", "q_weight", "dq"), ("k", "k_weight", "dk")):
        dt = s[x].dtype
        x = s[x].detach().float()
        if s["norm"]:
            wf = s[w].detach().float()
            rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            y = x * rstd
        outs.append(_turned(y * wf if s["norm"] else x, cos, sin, rotary, inter).to(dt))
        if not s["train"]:
            continue
        gz = _turned(s[g].float(), cos, -sin, rotary, inter)
        if s["norm"]:
            # a long sum: in 64 bits
            wgrads.append((gz * y).double().sum((0, 1, 2)).to(s[w].dtype))
            gy = gz * wf
            gz = rstd * (gy - y * (gy * y).mean(-1, keepdim=True))
        grads.append(gz.to(dt))
    return (*outs, *grads, *wgrads)


# ---- the definition in 64 bits --------------------------------------------------


def exact(case, seed):
    """The definition, row by row in float64. None where the outputs are copied or whole numbers."""
    if case["op"] in ("fork", "free", "compact"):
        return None
    s = prepare(case, seed)
    n, h, d, h_kv = case["n"], case["h"], case["d"], case["h_kv"]
    f64 = torch.float64
    if case["op"] == "shared":
        _, _, lens = _shared(case)
        out = torch.zeros(n, 1, h, d, dtype=f64, device="cuda")
        lse = torch.full((n, h, 1), -math.inf, dtype=f64, device="cuda")
        for r, length in enumerate(lens):
            if length == 0:
                continue
            ids = s["block_table"][r, : _pages(length, case["page"])].long()
            keys = s["k_cache"][ids].flatten(0, 1)[:length].double().transpose(0, 1)
            vals = s["v_cache"][ids].flatten(0, 1)[:length].double().transpose(0, 1)
            z = torch.bmm(s["q"][r, 0].double().view(h_kv, h // h_kv, d), keys.transpose(1, 2)) / math.sqrt(d)
            lse[r, :, 0] = torch.logsumexp(z, -1).flatten()
            out[r, 0] = torch.bmm(torch.softmax(z, -1), vals).reshape(h, d)
        return out, lse
    pairs = case["rotary"] // 2
    freq, size = [], 1.0
    for i in range(pairs):
        w = 10000.0 ** (-i / pairs)
        if case["scaling"] == "linear":
            w /= 4.0
        elif case["scaling"] == "ntk":
            w *= 4.0 ** (-i / (pairs - 1)) if pairs > 1 else 1.0
        elif case["scaling"] == "yarn":
            size = 1.0 + 0.1 * math.log(8.0)
            turns = 4096 * w / (2 * math.pi)
            share = min(1.0, max(0.0, (turns - 1.0) / 31.0))
            w = share * w + (1 - share) * w / 8.0
        freq.append(w)
    angle = s["positions"][0].double()[:, :, None, None] * torch.tensor(freq, dtype=f64, device="cuda")
    turn = torch.polar(torch.full_like(angle, size), angle)
    at = torch.arange(pairs, device="cuda")
    re, im = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + pairs)

    def turned(x, by):
        y = x.clone()
        z = torch.complex(x[..., re], x[..., im]) * by
        y[..., re], y[..., im] = z.real, z.imag
        return y

    outs, grads, wgrads = [], [], []
    for x, w, g in (("q", "q_weight", "dq"), ("k", "k_weight", "dk")):
        x = s[x].detach().double()
        if case["norm"]:
            scale = s[w].detach().double()
            size_of = torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS)
        outs.append(turned(x / size_of * scale if case["norm"] else x, turn))
        if case["train"]:
            back = turned(s[g].double(), turn.conj())
            if case["norm"]:
                wgrads.append((back * x / size_of).sum((0, 1, 2)))
                back = back * scale / size_of
                back = back - x * (back * x).sum(-1, keepdim=True) / (d * size_of.square())
            grads.append(back)
    return (*outs, *grads, *wgrads)
