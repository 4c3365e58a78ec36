"""paged_plan, paged_write and paged_decode against their definitions.

Bounds of paged_decode against fp64. With u = 2^-23 (a unit in the last place,
which also covers sums that truncate) a score, a sum of d products of exact
inputs in fp32, is within (d + 2) u S of the true one, S = scale * sum |q_i k_i|
at its largest; the exponential adds 2^-21 relative, and weights that are split
into two bf16 terms 2^-15 (the first is cut to 8 bits and leaves at most 2^-7, of
which rounding the second to 8 bits leaves at most 2^-8).
So every weight is within e = (d + 2) u S + 2^-21 + 2^-15 of the true one,
relative, numerator and denominator alike, and a sum over L keys adds L u: the
output is within (2 e + 2 L u) A, A = sum_j p_j |v_j|, the log-sum-exp within e +
L u + u |lse|. A bf16 output adds half a step, 2^-8 of its value."""

import math

import numpy as np
import pytest

from oracle import paged as op

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
PAGES = -9


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def draw(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (scale * torch.randn(shape, device="cuda", generator=g)).to(dtype)


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


# ---- decode ----------------------------------------------------------------------


def make(lens, h, h_kv, d, page, dtype, seed=0, extra_pages=3, extra_cols=2, poison=True, qscale=1.0):
    """q, caches and a shuffled table for requests of these lengths. What no
    request owns, and the rest of a request's last page, holds NaN and infinity."""
    n = len(lens)
    counts = [-(-l // page) for l in lens]
    pages = sum(counts) + extra_pages
    rng = np.random.default_rng(seed)
    perm = rng.permutation(pages)
    width = max(counts, default=0) + extra_cols
    table = np.full((n, width), -1, dtype=np.int32)
    at = 0
    for r, c in enumerate(counts):
        table[r, :c] = perm[at:at + c]
        at += c
    k, v = draw((pages, page, h_kv, d), dtype, seed + 1), draw((pages, page, h_kv, d), dtype, seed + 2)
    if poison:
        own = np.zeros((pages, page), dtype=bool)
        for r, l in enumerate(lens):
            for j in range(l):
                own[table[r, j // page], j % page] = True
        rest = torch.from_numpy(~own).cuda()
        k[rest], v[rest] = math.nan, math.inf
    q = draw((n, 1, h, d), dtype, seed + 3, qscale)
    return q, k, v, i32(table), i32(lens)


def check(out, lse, q, k, v, table, lens, scale, left=-1):
    ref_o, ref_l, a, s = op.decode(f64(q), f64(k), f64(v), table.cpu().numpy(), lens.cpu().numpy(), scale, left)
    u = 2.0 ** -23
    keys = max(int(lens.max()), 0)
    e = (q.shape[3] + 2) * u * s + 2 ** -21 + 2 ** -15
    o, l = f64(out), f64(lse)
    empty = np.isneginf(ref_l)
    assert np.array_equal(np.isneginf(l), empty)
    fin = ~empty
    le = np.abs(np.where(fin, l, 0) - np.where(fin, ref_l, 0))
    lt = e + keys * u + u * np.abs(np.where(fin, ref_l, 0))
    assert (le <= lt).all(), (le / lt).max()
    tol = (2 * e + 2 * keys * u)[:, None, :, :] .reshape(a.shape[0], 1, a.shape[2], 1) * a + 1e-38
    if out.dtype == BF16:
        tol = tol + 2 ** -8 * (np.abs(ref_o) + tol)
    err = np.abs(o - ref_o)
    assert (err <= tol).all(), (err / tol).max()
    assert not o[np.broadcast_to(empty.reshape(a.shape[0], 1, a.shape[2], 1), o.shape)].any()


RAGGED = [1, 0, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 300, 511, 512, 513, 700, 5, 1025]
HEADS = [(1, 1), (2, 1), (4, 4), (8, 2), (7, 1), (16, 1), (17, 1), (34, 2), (15, 5)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,h_kv", HEADS)
def test_decode_bf16_heads(h, h_kv, d):
    import blockwise_exact_attention_gb300 as bea
    x = make(RAGGED, h, h_kv, d, 16, BF16, seed=h + d)
    scale = 1.0 / math.sqrt(d)
    out, lse = bea.paged_decode(*x, scale)
    assert out.dtype == BF16 and out.shape == x[0].shape
    check(out, lse, *x, scale)
    out32, lse32 = bea.paged_decode(*x, scale, out_dtype=F32)
    check(out32, lse32, *x, scale)
    assert torch.equal(out32.to(BF16), out) and torch.equal(lse, lse32)
    assert bea.device_status() == 0


@pytest.mark.parametrize("d", [4, 12, 32, 64, 80, 100, 128])
@pytest.mark.parametrize("h,h_kv", [(1, 1), (6, 2), (9, 1), (20, 1)])
def test_decode_f32(h, h_kv, d):
    import blockwise_exact_attention_gb300 as bea
    x = make(RAGGED, h, h_kv, d, 24, F32, seed=h + d)
    out, lse = bea.paged_decode(*x)
    check(out, lse, *x, 1.0 / math.sqrt(d))
    assert bea.device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [1, 3, 8, 16, 20, 48, 64, 1000])
@pytest.mark.parametrize("left", [-1, 0, 1, 15, 100])
def test_decode_pages_and_windows(page, left, dtype):
    import blockwise_exact_attention_gb300 as bea
    x = make([1, 0, 40, 16, 101, 117, 999, 640], 4, 2, 64, page, dtype, seed=page)
    out, lse = bea.paged_decode(*x, 0.2, window_left=left)
    check(out, lse, *x, 0.2, left)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 96)])
@pytest.mark.parametrize("lens", [[9001], [5000, 3], [2049, 4097, 1, 0, 2048], [700] * 40, [1] * 300, [4000] * 9])
def test_decode_split_lengths(lens, dtype, d):
    import blockwise_exact_attention_gb300 as bea
    x = make(lens, 8, 2, d, 16, dtype, seed=len(lens), qscale=3.0)
    out, lse = bea.paged_decode(*x, 0.125)
    check(out, lse, *x, 0.125)
    again = bea.paged_decode(*x, 0.125)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])      # no order left to chance
    out, lse = bea.paged_decode(*x, 0.125, window_left=1500)
    check(out, lse, *x, 0.125, 1500)


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (F32, 32)])
@pytest.mark.parametrize("h,h_kv", [(40, 1), (66, 2), (300, 1), (150, 1)])
def test_decode_wide_groups(h, h_kv, dtype, d):
    """Query heads of a K/V head dealt to neighbouring CTAs, and past 16 such blocks to further launches."""
    import blockwise_exact_attention_gb300 as bea
    x = make([2500, 0, 3, 700], h, h_kv, d, 16, dtype, seed=h)
    out, lse = bea.paged_decode(*x, 0.15)
    check(out, lse, *x, 0.15)
    assert bea.device_status() == 0


def test_decode_more_requests_than_one_pass_takes():
    import blockwise_exact_attention_gb300 as bea
    n = 5003
    lens = [int(l) for l in np.random.default_rng(1).integers(0, 40, n)]
    x = make(lens, 2, 1, 64, 16, BF16, poison=False)
    out, lse = bea.paged_decode(*x, 0.125)
    check(out, lse, *x, 0.125)


def test_decode_layouts():
    """A cache with heads before tokens, K and V as halves of one tensor, q and out
    as slices, a table with a row stride, pages shared between requests."""
    import blockwise_exact_attention_gb300 as bea
    q, k, v, table, lens = make([700, 33, 400], 8, 2, 128, 16, BF16, seed=5, poison=False)
    table[1, :2] = table[0, :2]
    scale = 0.09
    want, want_lse = bea.paged_decode(q, k, v, table, lens, scale)
    check(want, want_lse, q, k, v, table, lens, scale)
    khd, vhd = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
    both = torch.stack([k, v], 1)                          # [pages, 2, page, h_kv, d]
    fused = torch.zeros((3, 1, 12, 128), dtype=BF16, device="cuda")
    fused[:, :, :8] = q
    wide = torch.full((3, table.shape[1] + 5), 10 ** 6, dtype=I32, device="cuda")
    wide[:, :table.shape[1]] = table
    big = torch.full((3, 1, 8, 256), 7.0, dtype=BF16, device="cuda")
    for qq, kk, vv, tt, oo in [(q, khd, vhd, table, None), (q, both[:, 0], both[:, 1], table, None), (q, k, vhd, table, None),
                               (fused[:, :, :8], k, v, wide[:, :table.shape[1]], big[..., :128])]:
        out, lse = bea.paged_decode(qq, kk, vv, tt, lens, scale, out=oo)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert (big[..., 128:] == 7).all()
    assert bea.device_status() == 0


def test_decode_merges_with_other_keys():
    """(out, lse) of two halves of a cache, folded by ring_merge, is the whole's."""
    import blockwise_exact_attention_gb300 as bea
    q, k, v, table, lens = make([1000, 500], 4, 2, 64, 20, BF16, seed=6, poison=False)
    left = i32([600, 500])
    a, la = bea.paged_decode(q, k, v, table, left, 0.125, out_dtype=F32)
    rest = i32([400, 0])
    b, lb = bea.paged_decode(q, k, v, table[:, 30:].contiguous(), rest, 0.125, out_dtype=F32)
    bea.ring_merge(a, la, b, lb)
    check(a, la, q, k, v, table, lens, 0.125)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 64)])
def test_decode_bad_pages_and_lengths(dtype, d):
    import blockwise_exact_attention_gb300 as bea
    q, k, v, table, lens = make([100, 100, 100, 40, 100], 4, 2, d, 16, dtype, seed=7, poison=False, extra_cols=0)
    assert bea.device_status() == 0
    for bad in (-1, k.shape[0], 2 ** 31 - 1, -(2 ** 31)):
        t = table.clone()
        t[0, 2], t[4, 0], t[4, 6] = bad, bad, bad
        t[3, 2:] = bad
        out, lse = bea.paged_decode(q, k, v, t, lens, 0.1)
        assert bea.device_status() == PAGES and bea.device_status() == 0
        check(out, lse, q, k, v, t, lens, 0.1)
        t[:] = bad                                          # nothing left to see
        out, lse = bea.paged_decode(q, k, v, t, lens, 0.1)
        assert bea.device_status() == PAGES
        assert not out.any() and torch.isneginf(lse).all()
    over = i32([100, 113, -5, 2 ** 31 - 1, -(2 ** 31)])       # 7 pages of 16: 112 keys
    table[1, 6] = table[0, 6]
    table[3] = table[0]
    out, lse = bea.paged_decode(q, k, v, table, over, 0.1)
    assert bea.device_status() == PAGES
    check(out, lse, q, k, v, table, over, 0.1)


def test_decode_infinities_and_nan_in_visible_places():
    import blockwise_exact_attention_gb300 as bea
    q, k, v, table, lens = make([90, 90, 90, 90], 2, 1, 64, 16, BF16, seed=8, poison=False)
    v[table[0, 1], 3] = math.inf                            # weight > 0 on an infinite value
    k[table[1, 4], 2] = math.nan
    lowest = torch.finfo(BF16).min
    q[2], k[table[2, 0], 0] = lowest, lowest                # a score past the largest number: NaN by the definition
    q[3] = 0
    k[table[3, 2], 1] = lowest
    out, lse = bea.paged_decode(q, k, v, table, lens, 0.125)
    assert torch.isposinf(out[0]).all() and torch.isfinite(lse[0]).all()
    assert out[1].isnan().all() and lse[1].isnan().all()
    assert out[2].isnan().all()
    check(out[3:], lse[3:], q[3:], k, v, table[3:], lens[3:], 0.125)


def test_decode_scores_of_the_lowest_value():
    """Keys so far below the largest that their weight is 0, and rows whose scores
    are all of that size."""
    import blockwise_exact_attention_gb300 as bea
    q, k, v, table, lens = make([600, 600], 2, 1, 64, 16, F32, seed=9, poison=False)
    q[:] = 1e15
    k[table[0].long()] = -1e15
    k[table[0, 3], 5] = 1.0
    k[table[1].long()] = -1e15
    out, lse = bea.paged_decode(q, k, v, table, lens, 0.125)
    assert torch.equal(out[0, 0, 0], v[table[0, 3], 5, 0])
    ref = v[table[1, :38].long()].reshape(-1, 64)[:600].double().mean(0)
    assert (out[1, 0, 0].double() - ref).abs().max() <= 600 * 2 ** -22
    assert torch.isfinite(lse).all()


def test_decode_offsets_past_32_bits():
    import blockwise_exact_attention_gb300 as bea
    pages, page, h_kv, d = 34000, 64, 8, 128                 # 2.2e9 elements a cache
    k = torch.empty((pages, page, h_kv, d), dtype=BF16, device="cuda")
    v = torch.empty_like(k)
    ids = [33999, 0, 33001, 17000, 32999]
    for i, p in enumerate(ids):
        k[p], v[p] = draw((page, h_kv, d), BF16, 30 + i), draw((page, h_kv, d), BF16, 40 + i)
    q, table, lens = draw((1, 1, 16, d), BF16, 50), i32([ids]), i32([300])
    out, lse = bea.paged_decode(q, k, v, table, lens, 0.1)
    small = torch.stack([k[p] for p in ids]), torch.stack([v[p] for p in ids])
    check(out, lse, q, *small, i32([list(range(5))]), lens, 0.1)


def test_decode_empty_batch_and_empty_cache():
    import blockwise_exact_attention_gb300 as bea
    q, k, v, table, lens = make([30, 20], 4, 2, 64, 16, BF16, seed=10)
    out, lse = bea.paged_decode(q[:0], k, v, table[:0], lens[:0], 0.1)
    assert out.shape == (0, 1, 4, 64) and lse.shape == (0, 4, 1)
    out, lse = bea.paged_decode(q, k, v, table[:, :0], i32([0, 0]), 0.1)
    assert not out.any() and torch.isneginf(lse).all()
    out, lse = bea.paged_decode(q, k[:0], v[:0], table, i32([0, 0]), 0.1)
    assert not out.any() and torch.isneginf(lse).all()
    assert bea.device_status() == 0


def test_decode_in_two_graphs_and_on_two_streams():
    """Captured once, replayed on new lengths, tables and values; a second graph and
    an eager call on another stream run with workspaces of their own."""
    import blockwise_exact_attention_gb300 as bea
    sets = [make(l, 8, 2, 128, 16, BF16, seed=s, extra_pages=400 - sum(-(-x // 16) for x in l), extra_cols=200 - max(-(-x // 16) for x in l))
            for s, l in ((60, [3000, 17, 0, 900]), (70, [1, 2500, 64, 100]), (80, [0, 0, 0, 3100]))]
    static = [t.clone() for t in sets[0]]
    outs, graphs = [], []
    for _ in range(2):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            bea.paged_decode(*static, 0.1)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(bea.paged_decode(*static, 0.1))
        graphs.append(g)
    for x in sets:
        for t, new in zip(static, x):
            t.copy_(new)
        side.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
            eager = bea.paged_decode(*static, 0.1)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        check(*outs[0], *x, 0.1)
        for a, b in ((outs[1], outs[0]), (eager, outs[0])):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_behind_other_nodes():
    """The calls' launches behind a memset, a copy and a fork of the captured stream."""
    import blockwise_exact_attention_gb300 as bea
    x = make([3000, 70], 8, 2, 128, 16, BF16, seed=90)
    q, k, v, table, lens = x
    bea.paged_decode(*x, 0.1)
    junk, q2 = torch.ones(1000, device="cuda"), torch.empty_like(q)
    slots = i32([5, -1])
    new = draw((2, 1, 2, 128), BF16, 91)
    kc, vc = torch.zeros_like(k), torch.zeros_like(v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        junk.zero_()
        a = bea.paged_decode(*x, 0.1)
        q2.copy_(q)
        b = bea.paged_decode(q2, k, v, table, lens, 0.1)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            bea.paged_write(new, new, slots, kc, vc)
            c = bea.paged_decode(q2, k, v, table, lens, 0.1)
        d = bea.paged_decode(q2, k, v, table, lens, 0.1)
        torch.cuda.current_stream().wait_stream(side)
        e = bea.paged_decode(q2, k, v, table, lens, 0.1)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    check(*a, *x, 0.1)
    for y in (b, c, d, e):
        assert torch.equal(a[0], y[0]) and torch.equal(a[1], y[1])
    assert torch.equal(kc.view(-1, 2, 128)[5], new[0, 0])


def test_first_call_inside_a_capture():
    """A process whose first calls are captured ones (no warm-up)."""
    import subprocess
    import sys
    code = """
import torch, blockwise_exact_attention_gb300 as bea
q = torch.randn(2, 1, 4, 64, device="cuda").bfloat16()
k, v = torch.randn(2, 9, 16, 2, 64, device="cuda").bfloat16().unbind(0)
table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
lens = torch.tensor([60, 3], dtype=torch.int32, device="cuda")
pos = lens.view(1, 2, 1)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    turned, _ = bea.rope_axes(q, None, pos, (32,))
    out, lse = bea.paged_decode(turned, k, v, table, lens, 0.1)
g.replay()
ref, ref_lse = bea.paged_decode(bea.rope_axes(q, None, pos, (32,))[0], k, v, table, lens, 0.1)
assert torch.equal(out, ref) and torch.equal(lse, ref_lse) and bea.device_status() == 0
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert r.stdout.strip() == "captured", r.stderr[-2000:]


def test_written_tensors_are_known_to_autograd():
    import blockwise_exact_attention_gb300 as bea
    x = make([30, 20], 4, 2, 64, 16, BF16, seed=92)
    q, k, v, table, lens = x
    new = draw((2, 1, 2, 64), BF16, 93)
    leaf = k.clone().requires_grad_()
    with pytest.raises(ValueError, match="requires grad"):
        bea.paged_write(new, new, lens, leaf, v)
    w = torch.ones_like(k, requires_grad=True)
    y = (w * k).sum()
    bea.paged_write(new, new, lens, k, v)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with pytest.raises(ValueError, match="requires grad"):
        bea.paged_decode(*x, out=torch.zeros_like(q, requires_grad=True))


def test_decode_workspace_is_checked():
    import blockwise_exact_attention_gb300 as bea
    x = make([5000], 8, 2, 128, 16, BF16, seed=11)
    need = bea.paged_decode_workspace_bytes(x[0], x[1], x[3])
    if need:
        ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
        out, lse = bea.paged_decode(*x, 0.1, workspace=ws[:need])
        assert (ws[need:] == 255).all()
        check(out, lse, *x, 0.1)
        for bad in (ws[:need - 1], ws[16:]):
            with pytest.raises(RuntimeError, match="WORKSPACE"):
                bea.paged_decode(*x, 0.1, workspace=bad)


# ---- write -----------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,l,h_kv,d,page", [(1, 1, 1, 64, 16), (5, 1, 2, 128, 16), (2, 37, 3, 8, 5), (1, 700, 8, 128, 64),
                                             (3, 11, 1, 264, 1)])
def test_write(n, l, h_kv, d, page, dtype):
    import blockwise_exact_attention_gb300 as bea
    pages = (n * l) // page + 9
    rng = np.random.default_rng(0)
    slots = rng.permutation(pages * page)[:n * l].astype(np.int32)
    slots[rng.random(n * l) < 0.2] = -1
    k, v = draw((n, l, h_kv, d), dtype, 1), draw((n, l, h_kv, d), dtype, 2)
    kc, vc = draw((pages, page, h_kv, d), dtype, 3), draw((pages, page, h_kv, d), dtype, 4)
    want = [kc.clone(), vc.clone()]
    for w, new in zip(want, (k, v)):
        flat, src = w.view(-1, h_kv, d), new.reshape(-1, h_kv, d)
        for t, s in enumerate(slots):
            if s >= 0:
                flat[int(s)] = src[t]
    bea.paged_write(k, v, i32(slots), kc, vc)
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    assert bea.device_status() == 0


def test_write_layouts_and_bad_slots():
    import blockwise_exact_attention_gb300 as bea
    n, h_kv, d, page, pages = 40, 2, 64, 16, 6
    qkv = draw((n, 1, 8, d), BF16, 5)
    k, v = qkv[:, :, 4:6], qkv[:, :, 6:8]                   # slices of a fused projection
    slots = torch.randperm(pages * page, device="cuda")[:n].to(I32)
    want_k, want_v = (torch.zeros((pages, page, h_kv, d), dtype=BF16, device="cuda") for _ in range(2))
    bea.paged_write(k.contiguous(), v.contiguous(), slots, want_k, want_v)
    hd = torch.zeros((pages, h_kv, page, d), dtype=BF16, device="cuda").transpose(1, 2)
    both = torch.zeros((pages, 2, page, h_kv, d), dtype=BF16, device="cuda")
    bea.paged_write(k, v, slots, hd, both[:, 1])
    assert torch.equal(hd, want_k) and torch.equal(both[:, 1], want_v) and not both[:, 0].any()
    one = k[:1].expand(n, 1, h_kv, d)                       # the same row for every token
    bea.paged_write(one, one, slots, hd, both[:, 0])
    assert (hd.reshape(-1, h_kv, d)[slots.long()] == k[0]).all()
    assert bea.device_status() == 0
    before = want_k.clone()
    bad = slots.clone()
    bad[3], bad[7], bad[9], bad[11] = -2, pages * page, 2 ** 31 - 1, -(2 ** 31)
    keep = torch.ones(n, dtype=torch.bool)
    keep[[3, 7, 9, 11]] = False
    bea.paged_write(v, k, bad, want_k, want_v)
    assert bea.device_status() == PAGES
    flat = before.view(-1, h_kv, d)
    flat[slots.long()[keep.cuda()]] = v.reshape(-1, h_kv, d)[keep.cuda()]
    assert torch.equal(want_k, before)


def test_write_offsets_past_32_bits():
    import blockwise_exact_attention_gb300 as bea
    pages, page, h_kv, d = 34000, 64, 8, 128
    kc = torch.zeros((pages, page, h_kv, d), dtype=BF16, device="cuda")
    vc = torch.zeros_like(kc)
    slots = i32([pages * page - 1, 0, 33000 * 64 + 5])
    k, v = draw((3, 1, h_kv, d), BF16, 6), draw((3, 1, h_kv, d), BF16, 7)
    bea.paged_write(k, v, slots, kc, vc)
    for i, s in enumerate(slots.tolist()):
        assert torch.equal(kc[s // page, s % page], k[i, 0]) and torch.equal(vc[s // page, s % page], v[i, 0])
    assert int(kc.count_nonzero()) == int(k.count_nonzero())


# ---- plan ------------------------------------------------------------------------


def run_plan(lens, new, table, pool, n_free, page, capacity, in_place=False):
    import blockwise_exact_attention_gb300 as bea
    t, f = i32(table).reshape(len(lens), -1), i32(pool)
    L, nf = i32(lens), i32([n_free])
    out = None
    if in_place:
        n = len(lens)
        e = lambda m: torch.full((m,), 12345, dtype=I32, device="cuda")  # noqa: E731
        out = bea.PagedPlan(e(capacity), e(capacity), e(n + 1), e(n + 1), L, nf)
    p = bea.paged_plan(L, i32(new), t, f, nf, page, capacity, out)
    got = [x.tolist() for x in p]
    got[5] = got[5][0]
    if not in_place:
        assert L.tolist() == list(lens) and nf.tolist() == [n_free]
    return (*got, t.tolist(), f.tolist())


def expect(lens, new, table, pool, n_free, page, capacity, status=0):
    import blockwise_exact_attention_gb300 as bea
    *want, ok = op.plan(lens, new, table, pool, n_free, page, capacity)
    assert ok == (status == 0)
    for in_place in (False, True):
        got = run_plan(lens, new, table, pool, n_free, page, capacity, in_place)
        for name, a, b in zip(("slots", "positions", "cu_new", "cu_pages", "lens", "n_free", "table", "pool"), got, want):
            assert a == b, name
        assert bea.device_status() == status
    return want


@pytest.mark.parametrize("n,page,capacity", [(1, 16, 1), (3, 1, 7), (33, 4, 64), (1000, 16, 3000), (1024, 7, 5000), (2500, 16, 9000),
                                             (4, 64, 4097)])
def test_plan_steps(n, page, capacity):
    rng = np.random.default_rng(n)
    width = -(-200 // page)
    total = n * width + 5
    lens, table = [0] * n, [[-1] * width for _ in range(n)]
    pool, free = [int(x) for x in rng.permutation(total)], total
    for step in range(4):
        new = [int(x) for x in rng.choice([0, 1, 1, 2, 9, -1], n)]
        big = int(rng.integers(n))
        new[big] = min(width * page - lens[big], max(0, capacity - sum(max(a, 0) for a in new)))
        left = capacity
        for r in range(n):
            new[r] = min(new[r], left, width * page - lens[r])
            left -= max(new[r], 0)
        *_, lens, free, table, pool = expect(lens, new, table, pool, free, page, capacity)


def test_plan_refuses_whole_steps():
    base = dict(lens=[5, 16, 0], new=[1, 1, 3], table=[[0, -1], [1, -1], [-1, -1]], pool=[2, 3, 4, -1], n_free=3, page=16, capacity=8)
    expect(**base)
    for change in (dict(new=[1, -2, 3]), dict(lens=[5, -1, 0]), dict(lens=[5, 33, 0]), dict(new=[28, 1, 3]), dict(new=[4, 2, 3], capacity=8),
                   dict(n_free=1), dict(n_free=-1), dict(n_free=5), dict(n_free=4, new=[-1, 1, 3], pool=[2, 3, 4, 5]),
                   dict(new=[2 ** 31 - 1, 0, 0]), dict(lens=[2 ** 31 - 1, 16, 0], new=[-1, 0, 0]), dict(new=[0, 0, 2 ** 31 - 1], capacity=5000),
                   dict(new=[1, 1, 3], capacity=0)):
        expect(**{**base, **change}, status=PAGES)


def test_plan_without_requests_or_places():
    import blockwise_exact_attention_gb300 as bea
    none = i32([])
    for capacity in (0, 7, 5000):
        p = bea.paged_plan(none, none, i32([]).reshape(0, 3), i32([4, 5]), i32([2]), 16, capacity)
        assert p.slot_map.tolist() == [-1] * capacity and p.positions.tolist() == [0] * capacity
        assert p.cu_new.tolist() == p.cu_pages.tolist() == [0] and p.lens.tolist() == [] and p.n_free.tolist() == [2]
    expect([20, 0, 3], [0, 0, -1], [[1, 2], [-1, -1], [0, -1]], [7, 8, -1, -1], 2, 16, 0)
    assert bea.device_status() == 0


def test_plan_ends_feed_the_new():
    # nothing is free until row 0 ends; its pages go to rows 1 and 2 in the same step
    expect([40, 16, 0], [-1, 1, 17], [[7, 5, 9, -1], [1, -1, -1, -1], [-1] * 4], [0] * 9, 0, 16, 32)


def test_plan_reports_pages_that_have_no_slot():
    import blockwise_exact_attention_gb300 as bea
    p = bea.paged_plan(i32([0, 0, 4]), i32([2, 1, 1]), i32([[-1], [-1], [2 ** 31 - 1]]), i32([-7, 3]), i32([2]), 16, 5)
    assert p.slot_map.tolist() == [48, 49, -1, -1, -1] and p.n_free.tolist() == [0]
    assert bea.device_status() == PAGES


def test_plan_captured_and_replayed():
    import blockwise_exact_attention_gb300 as bea
    for capacity in (64, 6000):                            # one launch, two launches
        cache = bea.PagedKVCache(500, 16, 1, 64, 8, 1600)
        new = i32([0] * 8)
        cache.plan(new, capacity)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p = cache.plan(new, capacity)
        state = ([0] * 8, cache.block_table.tolist(), cache.free_pages.tolist(), 500)
        for step in ([3, 0, 17, 1, 0, 0, 16, 2], [1] * 8, [-1, 1, 1, -1, 20, 1, 1, 1], [5, 1, 1, 1, -1, 1, 1, 1]):
            new.copy_(i32(step))
            g.replay()
            lens, table, pool, free = state
            *want, lens, free, table, pool, ok = op.plan(lens, step, table, pool, free, 16, capacity)
            state = (lens, table, pool, free)
            assert ok and [x.tolist() for x in p[:4]] == want
            assert cache.lens.tolist() == lens and cache.n_free.tolist() == [free]
            assert cache.block_table.tolist() == table and cache.free_pages.tolist() == pool
        assert bea.device_status() == 0


def test_python_refusals():
    import blockwise_exact_attention_gb300 as bea
    q, k, v, table, lens = make([30, 20], 4, 2, 64, 16, BF16, seed=12)
    with pytest.raises(ValueError):
        bea.paged_decode(q, k.cpu(), v, table, lens)
    with pytest.raises(TypeError):
        bea.paged_decode(q, k, v, table.long(), lens)
    with pytest.raises(TypeError):
        bea.paged_decode(q.half(), k, v, table, lens)
    with pytest.raises(RuntimeError, match="SHAPE"):
        bea.paged_decode(q.expand(2, 3, 4, 64), k, v, table, lens)
    with pytest.raises(RuntimeError, match="DTYPE"):
        bea.paged_write(q, q, lens, k.float(), v.float())
    with pytest.raises(RuntimeError, match="SHAPE"):
        bea.paged_plan(lens, lens, table[:1], lens, lens[:1], 16, 4)
    assert bea.device_status() == 0
