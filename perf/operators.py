"""What the serving and position operators are measured on.

Four operators that work together: ``rope_axes`` (rotary positions with one or
several axes, forward and gradient), ``paged_plan`` (block tables, slot map and
positions from request lengths), ``paged_write`` (new keys and values into a
paged cache) and ``paged_decode`` (attention of one new token per request over
that cache). ``run`` computes a case in its plain form, elementary torch
operations in 32 bits (angles in 64), or, where ``own`` is set, by the calls a
program makes of this package.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases -----------------------------------------------------------------


def listed():
    return [
        # one chat request shortly after its prompt: the smallest call, where only latency counts
        dict(name="decode_one_request", op="decode", n=1, h=32, h_kv=8, d=128, dtype="bf16", page=16, max_len=512,
             min_len=129, full=False, window=-1, lens_seed=1),
        # a serving batch in mid-flight: ragged lengths over three decades, one row without a request
        dict(name="decode_ragged_batch", op="decode", n=64, h=32, h_kv=8, d=128, dtype="bf16", page=16, max_len=8192,
             min_len=0, full=False, window=-1, lens_seed=2),
        # one document-length context: all of the card works on one row, split over its length
        dict(name="decode_long_context", op="decode", n=1, h=32, h_kv=8, d=128, dtype="bf16", page=64,
             max_len=131072, min_len=130001, full=True, window=-1, lens_seed=3),
        # the largest: a full batch of long contexts, several GB of cache in one pass
        dict(name="decode_large_batch", op="decode", n=48, h=32, h_kv=8, d=128, dtype="bf16", page=16,
             max_len=32768, min_len=16384, full=True, window=-1, lens_seed=4),
        # sliding window over long fp32 rows, one query head per K/V head, pages that divide nothing
        dict(name="decode_window_f32", op="decode", n=33, h=16, h_kv=16, d=64, dtype="f32", page=24, max_len=12288,
             min_len=0, full=False, window=1024, lens_seed=5),
        # a decode step of 256 requests: one token each, a few requests end
        dict(name="plan_decode_step", op="plan", n=256, page=16, max_len=8192, prefill=0, capacity=256, lens_seed=6),
        # continuous batching with chunked prefill: most rows add one token, some thousands
        dict(name="plan_prefill_mix", op="plan", n=1024, page=16, max_len=16384, prefill=8192, capacity=524288,
             lens_seed=7),
        # the new keys and values of that decode step
        dict(name="write_decode_step", op="write", n=256, h_kv=8, d=128, dtype="bf16", page=16, pages=4096, used=251),
        # and of a prefill of 64k tokens, the tail of the buffer unused
        dict(name="write_prefill", op="write", n=65536, h_kv=8, d=128, dtype="bf16", page=64, pages=2048, used=64999),
        # q and k of 256 new tokens with time, height and width positions
        dict(name="rope_decode_step", op="rope", n=256, l=1, h=32, h_kv=8, d=128, dtype="bf16", axes=3, joint=True,
             train=False),
        # a training step on a long video: forward and gradient
        dict(name="rope_video_train", op="rope", n=1, l=32768, h=32, h_kv=8, d=128, dtype="bf16", axes=3, joint=True,
             train=True),
        # image patches in fp32, 37 x 37 of them, each axis with its own frequencies, forward and gradient
        dict(name="rope_image_f32_train", op="rope", n=3, l=1369, h=12, h_kv=12, d=64, dtype="f32", axes=2,
             joint=False, train=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "plan", "write", "rope", "rope"])
    if op == "decode":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        d = rng.choice([64, 128]) if dtype == "bf16" else rng.choice([32, 48, 64, 80, 96, 128])
        h_kv = rng.choice([1, 2, 3, 4, 5, 8, 16, 32])
        h = h_kv * rng.choice([1, 2, 3, 4, 6, 8] if h_kv > 2 else [1, 3, 4, 7, 8, 12, 16, 20])
        row = h_kv * d * (2 if dtype == "bf16" else 4) * 2
        # at most 1.5 GB of visible cache and 2^27 (query head, key) pairs
        n = _log(rng, 1, 400)
        most = max(64, min(150000, 1_500_000_000 // (row * n), 2**27 // (n * h)))
        max_len = _log(rng, 17, most)
        full = rng.random() < 0.4
        return dict(op="decode", n=n, h=h, h_kv=h_kv, d=d, dtype=dtype, page=rng.choice([1, 8, 16, 16, 20, 32, 64, 100, 256]),
                    max_len=max_len, min_len=rng.choice([0, 1, max_len // 2]) if n > 1 else max(1, max_len // 2),
                    full=full, window=rng.choice([-1, -1, _log(rng, 1, max(2, max_len))]), lens_seed=rng.randrange(1 << 30))
    if op == "plan":
        n = _log(rng, 1, 1500)
        max_len = _log(rng, 64, 16384)
        prefill = rng.choice([0, _log(rng, 2, max_len)])
        return dict(op="plan", n=n, page=rng.choice([1, 8, 16, 20, 32, 64, 128]), max_len=max_len, prefill=prefill,
                    capacity=max(n, min(524288, n * max(1, prefill // 8))), lens_seed=rng.randrange(1 << 30))
    if op == "write":
        n = _log(rng, 1, 60000)
        page = rng.choice([1, 8, 16, 20, 32, 64])
        return dict(op="write", n=n, h_kv=rng.choice([1, 2, 3, 8, 16]), d=rng.choice([64, 128]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), page=page, pages=(n + page - 1) // page + rng.randrange(1, 999),
                    used=max(1, n - rng.randrange(0, 1 + n // 4)))
    n = _log(rng, 1, 300)
    h_kv = rng.choice([1, 2, 3, 8, 12])
    return dict(op="rope", n=n, l=_log(rng, 1, max(1, 20000 // n)), h=h_kv * rng.choice([1, 2, 4]), h_kv=h_kv,
                d=rng.choice([32, 64, 80, 96, 128, 256]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                axes=rng.choice([1, 2, 3, 4]), joint=rng.random() < 0.5, train=rng.random() < 0.5)


def _lens(case):
    """Request lengths of a decode case: given by the case alone, so that its work is too."""
    rng = random.Random(case["lens_seed"])
    lo, hi = case["min_len"], case["max_len"]
    if case["full"]:
        lens = [rng.randint(min(max(1, lo), hi), hi) for _ in range(case["n"])]
    else:
        lens = [_log(rng, min(max(1, lo), hi), hi) for _ in range(case["n"])]
    if lo == 0 and case["n"] > 2:
        lens[case["n"] // 2] = 0
    return lens


def _plan_lens(case):
    """(lens, new_lens) of a plan case: a few rows are free, a few end, some add a prompt's chunk."""
    rng = random.Random(case["lens_seed"])
    left = case["capacity"]
    lens, new = [], []
    for _ in range(case["n"]):
        l = rng.randrange(0, case["max_len"])
        what = rng.random()
        if what < 0.05:
            l, a = 0, 0
        elif what < 0.10:
            a = -1
        elif case["prefill"] and what < 0.30:
            a = rng.randint(1, case["prefill"])
        else:
            a = 1
        a = min(a, case["max_len"] - l, left)
        left -= max(a, 0)
        lens.append(l)
        new.append(a)
    return lens, new


def _sections(case):
    """Pairs per axis: uneven, all of the head dim."""
    half, axes = case["d"] // 2, case["axes"]
    if axes == 1:
        return (half,)
    first = max(1, half // (axes + 1))
    rest = half - first
    cuts = [rest * i // (axes - 1) for i in range(axes)]
    return (first,) + tuple(b - a for a, b in zip(cuts, cuts[1:]))


def _esize(case):
    return 2 if case["dtype"] == "bf16" else 4


def _pages(tokens, page):
    return -(-tokens // page)


def work(case):
    op = case["op"]
    if op == "decode":
        left = case["window"]
        seen = [l if left < 0 else min(l, left + 1) for l in _lens(case)]
        n, h, d, e = case["n"], case["h"], case["d"], _esize(case)
        kv = sum(seen) * case["h_kv"] * d * e * 2
        tables = sum(_pages(s, case["page"]) for s in seen) * 4 + n * 4
        return {"bytes": kv + tables + 2 * n * h * d * e + n * h * 4, "flops": 4 * sum(seen) * h * d}
    if op == "plan":
        lens, new = _plan_lens(case)
        ps, n = case["page"], case["n"]
        ended = sum(_pages(l, ps) for l, a in zip(lens, new) if a < 0)
        added = sum(_pages(l + a, ps) - _pages(l, ps) for l, a in zip(lens, new) if a >= 0)
        # lens and new_lens read, three rows of n written; pages that change hands read and written; two
        # numbers for each place of the token buffers
        return {"bytes": 4 * (5 * n + 4) + 8 * (ended + added) + 8 * case["capacity"], "flops": 0}
    if op == "write":
        row = case["h_kv"] * case["d"] * _esize(case) * 2
        return {"bytes": 2 * row * case["used"] + 4 * case["n"], "flops": 0}
    rows = case["n"] * case["l"] * (case["h"] + case["h_kv"])
    passes = 2 if case["train"] else 1
    return {"bytes": passes * (2 * rows * case["d"] * _esize(case) + 4 * case["axes"] * case["n"] * case["l"]),
            "flops": passes * 3 * rows * case["d"]}


# ---- inputs --------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dev = torch.device("cuda")

    def normal(*shape, dtype):
        return torch.randn(*shape, dtype=dtype, device=dev, generator=g)

    s = dict(case)
    op = case["op"]
    if op == "decode":
        dt = DTYPES[case["dtype"]]
        lens, page = _lens(case), case["page"]
        width = _pages(case["max_len"], page)
        counts = torch.tensor([_pages(l, page) for l in lens], device=dev)
        total = int(counts.sum())
        pages = total + 3  # a few pages that nobody owns
        perm = torch.randperm(pages, device=dev, generator=g).to(torch.int32)
        place = torch.arange(width, device=dev)
        start = counts.cumsum(0) - counts
        at = start[:, None] + place[None, :]
        table = torch.where(place[None, :] < counts[:, None], perm[at.clamp(max=pages - 1)], -1).to(torch.int32)
        cache = (pages, page, case["h_kv"], case["d"])
        s |= {"q": normal(case["n"], 1, case["h"], case["d"], dtype=dt), "k_cache": normal(*cache, dtype=dt),
              "v_cache": normal(*cache, dtype=dt), "block_table": table.contiguous(),
              "lens": torch.tensor(lens, dtype=torch.int32, device=dev), "scale": 1.0 / math.sqrt(case["d"])}
    elif op == "plan":
        lens, new = _plan_lens(case)
        ps, n = case["page"], case["n"]
        width = _pages(case["max_len"], ps)
        counts = torch.tensor([_pages(l, ps) for l in lens], device=dev)
        used = int(counts.sum())
        added = sum(_pages(l + a, ps) - _pages(l, ps) for l, a in zip(lens, new) if a >= 0)
        pages = used + added + 17
        perm = torch.randperm(pages, device=dev, generator=g).to(torch.int32)
        place = torch.arange(width, device=dev)
        start = counts.cumsum(0) - counts
        at = start[:, None] + place[None, :]
        table = torch.where(place[None, :] < counts[:, None], perm[at.clamp(max=pages - 1)], -1).to(torch.int32)
        free = torch.full((pages,), -1, dtype=torch.int32, device=dev)
        free[: pages - used] = perm[used:]
        s |= {"lens": torch.tensor(lens, dtype=torch.int32, device=dev),
              "new_lens": torch.tensor(new, dtype=torch.int32, device=dev), "block_table": table.contiguous(),
              "free_pages": free, "n_free": torch.tensor([pages - used], dtype=torch.int32, device=dev)}
    elif op == "write":
        dt = DTYPES[case["dtype"]]
        cache = (case["pages"], case["page"], case["h_kv"], case["d"])
        slots = torch.randperm(case["pages"] * case["page"], device=dev, generator=g)[: case["n"]].to(torch.int32)
        slots[case["used"]:] = -1
        new = (1, case["n"], case["h_kv"], case["d"])
        s |= {"k": normal(*new, dtype=dt), "v": normal(*new, dtype=dt), "slot_map": slots,
              "k_cache": torch.zeros(cache, dtype=dt, device=dev), "v_cache": torch.zeros(cache, dtype=dt, device=dev)}
    else:
        dt = DTYPES[case["dtype"]]
        n, l, axes = case["n"], case["l"], case["axes"]
        q, k = (n, l, case["h"], case["d"]), (n, l, case["h_kv"], case["d"])
        # time runs on from a far start, the other axes are grid coordinates
        time = torch.arange(l, device=dev)[None, :] + torch.randint(0, 100000, (n, 1), device=dev, generator=g)
        grid = torch.randint(0, 256, (axes - 1, n, l), device=dev, generator=g)
        s |= {"q": normal(*q, dtype=dt).requires_grad_(case["train"]),
              "k": normal(*k, dtype=dt).requires_grad_(case["train"]),
              "positions": torch.cat([time[None], grid]).to(torch.int32).contiguous(), "sections": _sections(case)}
        if case["train"]:
            s |= {"dq": normal(*q, dtype=dt), "dk": normal(*k, dtype=dt)}
    return s


# ---- one pass ------------------------------------------------------------------


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import blockwise_exact_attention_gb300 as bea

    op = s["op"]
    if op == "decode":
        return bea.paged_decode(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["lens"], s["scale"],
                                window_left=s["window"])
    if op == "plan":
        p = bea.paged_plan(s["lens"], s["new_lens"], s["block_table"], s["free_pages"], s["n_free"], s["page"],
                           s["capacity"])
        return (p.slot_map, p.positions, p.cu_new, p.lens, p.n_free, s["block_table"], s["free_pages"])
    if op == "write":
        return bea.paged_write(s["k"], s["v"], s["slot_map"], s["k_cache"], s["v_cache"])
    spectrum = "joint" if s["joint"] else "axis"
    if not s["train"]:
        return bea.rope_axes(s["q"], s["k"], s["positions"], s["sections"], spectrum=spectrum)
    qo, ko = bea.rotary_axes(s["q"], s["k"], s["positions"], s["sections"], spectrum=spectrum)
    dq, dk = torch.autograd.grad((qo, ko), (s["q"], s["k"]), (s["dq"], s["dk"]))
    return qo.detach(), ko.detach(), dq, dk


def _plain(s):
    return {"decode": _plain_decode, "plan": _plain_plan, "write": _plain_write, "rope": _plain_rope}[s["op"]](s)


def _plain_decode(s):
    q, lens, table, page = s["q"], s["lens"].long(), s["block_table"].long(), s["page"]
    n, _, h, d = q.shape
    h_kv = s["k_cache"].shape[2]
    rows = table.clamp(min=0)
    k = s["k_cache"][rows].reshape(n, -1, h_kv, d).float()
    v = s["v_cache"][rows].reshape(n, -1, h_kv, d).float()
    key = torch.arange(k.shape[1], device=q.device)[None, :]
    seen = key < lens[:, None]
    if s["window"] >= 0:
        seen = seen & (key >= lens[:, None] - 1 - s["window"])
    qg = q.reshape(n, h_kv, h // h_kv, d).float()
    score = torch.matmul(qg, k.permute(0, 2, 3, 1)) * s["scale"]
    score = torch.where(seen[:, None, None, :], score, -math.inf)
    top = score.max(-1, keepdim=True).values
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    v = torch.where(seen[:, :, None, None], v, 0.0)
    out = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total == 0, 1.0, total)
    lse = torch.where(total == 0, -math.inf, top + torch.log(total))
    return out.reshape(n, 1, h, d).to(q.dtype), lse.reshape(n, h, 1)


def _plain_plan(s):
    lens, new, ps, cap = s["lens"].long(), s["new_lens"].long(), s["page"], s["capacity"]
    table, free = s["block_table"].clone(), s["free_pages"].clone()
    ended = new < 0
    add = new.clamp(min=0)
    had = (lens + ps - 1) // ps
    after = torch.where(ended, 0, lens + add)
    has = torch.where(ended, 0, (after + ps - 1) // ps)
    back = torch.where(ended, had, 0)
    need = torch.where(ended, 0, has - had)
    back_at = s["n_free"].long() + back.cumsum(0) - back
    need_at = need.cumsum(0) - need
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    gives = ended[:, None] & (col < had[:, None])
    free[(back_at[:, None] + col)[gives]] = table[gives]
    top = s["n_free"].long() + back.sum()
    takes = ~ended[:, None] & (col >= had[:, None]) & (col < has[:, None])
    table[takes] = free[(top - 1 - (need_at[:, None] + col - had[:, None]))[takes]]
    cu = torch.cat([torch.zeros_like(add[:1]), add.cumsum(0)])
    i = torch.arange(cap, device=table.device)
    row = torch.searchsorted(cu[1:].contiguous(), i, right=True).clamp(max=lens.numel() - 1)
    used = i < cu[-1]
    pos = torch.where(used, lens[row] + i - cu[row], 0)
    slot = torch.where(used, table[row, (pos // ps).clamp(max=table.shape[1] - 1)].long() * ps + pos % ps, -1)
    i32 = torch.int32
    return slot.to(i32), pos.to(i32), cu.to(i32), after.to(i32), (top - need.sum()).to(i32), table, free


def _plain_write(s):
    slot = s["slot_map"].long()
    used = slot >= 0
    for cache, new in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])):
        flat = cache.view(-1, *cache.shape[2:])
        flat[slot[used]] = new.reshape(-1, *cache.shape[2:])[used]
    return s["k_cache"], s["v_cache"]


def _turn(x, cos, sin):
    a, b = x.float().chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(x.dtype)


def _plain_rope(s):
    dev, half = s["q"].device, s["d"] // 2
    sections = torch.tensor(s["sections"], device=dev)
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device=dev), sections, output_size=half)
    pair = torch.arange(half, dtype=torch.float64, device=dev)
    if s["joint"]:
        exponent = pair / half
    else:
        exponent = (pair - (sections.cumsum(0) - sections)[axis]) / sections[axis]
    freq = torch.pow(10000.0, -exponent)
    angle = s["positions"][axis].permute(1, 2, 0).double() * freq  # [n, l, d/2]
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    qo, ko = _turn(s["q"].detach(), cos, sin), _turn(s["k"].detach(), cos, sin)
    if not s["train"]:
        return qo, ko
    return qo, ko, _turn(s["dq"], cos, -sin), _turn(s["dk"], cos, -sin)


# ---- the definition in 64 bits --------------------------------------------------


def exact(case, seed):
    """The definition, row by row in float64. None where the outputs are copied or whole numbers."""
    if case["op"] in ("plan", "write"):
        return None
    s = prepare(case, seed)
    if case["op"] == "decode":
        n, h, d, h_kv, ps = case["n"], case["h"], case["d"], case["h_kv"], case["page"]
        out = torch.zeros(n, 1, h, d, dtype=torch.float64, device="cuda")
        lse = torch.full((n, h, 1), -math.inf, dtype=torch.float64, device="cuda")
        for r, length in enumerate(_lens(case)):
            lo = 0 if case["window"] < 0 else max(0, length - 1 - case["window"])
            if length <= lo:
                continue
            ids = s["block_table"][r, : _pages(length, ps)].long()
            keys = s["k_cache"][ids].flatten(0, 1)[lo:length].double()
            vals = s["v_cache"][ids].flatten(0, 1)[lo:length].double()
            for kv in range(h_kv):
                heads = slice(kv * (h // h_kv), (kv + 1) * (h // h_kv))
                z = (s["q"][r, 0, heads].double() @ keys[:, kv].T) / math.sqrt(d)
                lse[r, heads, 0] = torch.logsumexp(z, -1)
                out[r, 0, heads] = torch.softmax(z, -1) @ vals[:, kv]
        return out, lse
    half = case["d"] // 2
    place, freq = [], []
    for a, pairs in enumerate(_sections(case)):
        for j in range(pairs):
            e = len(freq) / half if case["joint"] else j / pairs
            place.append(a)
            freq.append(10000.0 ** -e)
    angle = s["positions"].double()[place] * torch.tensor(freq, dtype=torch.float64, device="cuda")[:, None, None]
    turn = torch.polar(torch.ones_like(angle), angle).permute(1, 2, 0)[:, :, None]

    def turned(x, by):
        z = torch.complex(x.detach()[..., :half].double(), x.detach()[..., half:].double()) * by
        return torch.cat([z.real, z.imag], -1)

    outs = [turned(s["q"], turn), turned(s["k"], turn)]
    if case["train"]:
        outs += [turned(s["dq"], turn.conj()), turned(s["dk"], turn.conj())]
    return tuple(outs)
