"""paged_decode_shared against the definition of single-token attention.

Bounds against fp64 as for paged_decode: with u = 2^-23 (which covers sums that
are cut off) a score is within (d + 2) u S of the true one, the exponential adds
2^-21, so a weight is within e = (d + 2) u S + 2^-21 relative. In the product with
the values a weight of the requests' own keys has 24 bits; one of the shared keys
has two bf16 terms for an f32 output (the first is cut to 8 bits and leaves at most
2^-7, of which rounding the second to 8 bits leaves at most 2^-9; a last bit that is
set may add 2^-23) and is rounded to one for a bf16 output: w = 2^-15 or 2^-8. A sum
over L keys adds L u, and joining the parts by their maxima and log-sum-exps 2^-20
more each time an exponent of size |lse| goes through fp32: the output is within (2
e + w + 2 L u + 2^-19 + 4 u |lse|) A, A = sum p |v|, the log-sum-exp (whose weights are
not rounded) within e + L u + 2^-20 + 4 u |lse|. A bf16 output adds half a step, 2^-8
of its value."""

import math
import random

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


def draw(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (scale * torch.randn(shape, device="cuda", generator=g)).to(BF16)


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def make(groups, h, h_kv, d, page, seed=0, qscale=1.0, wide=True):
    """groups: (shared keys, own keys of each row; None: a row without a request). What nobody owns holds NaN and
    infinity. `wide`: the table has room for so many keys that sharing may be worth it, whatever the lengths. -> (q, k, v,
    table, lens), (group_rows, shared_lens)"""
    rng = np.random.default_rng(seed)
    lens, rows, cuts, total = [], [], [0], 0
    for shared, own in groups:
        whole = shared // page
        first = list(range(total, total + whole))
        total += whole
        for o in own:
            length = 0 if o is None else shared + o
            mine = max(0, -(-length // page) - whole)
            rows.append(([] if o is None else first + list(range(total, total + mine)), whole))
            total += mine
            lens.append(length)
        cuts.append(len(lens))
    pages = total + 3
    perm = rng.permutation(pages)
    n, width = len(lens), max((len(r) for r, _ in rows), default=0) + 1
    if wide and n > 1:
        width = max(width, 97_000_000 // (h_kv * d * 4 * page * (n - 1)) + 2)
    table = np.full((n, width), -1, dtype=np.int32)
    own_slot = np.zeros((pages, page), dtype=bool)
    for r, (row, _) in enumerate(rows):
        table[r, :len(row)] = perm[row]
        for j in range(lens[r]):
            own_slot[table[r, j // page], j % page] = True
    k, v, q = draw((pages, page, h_kv, d), seed + 1), draw((pages, page, h_kv, d), seed + 2), draw((n, 1, h, d), seed + 3, qscale)
    rest = torch.from_numpy(~own_slot).cuda()
    k[rest], v[rest] = math.nan, math.inf
    # the prefix is shared page by page
    return (q, k, v, i32(table), i32(lens)), (i32(cuts), i32([s // page * page for s, _ in groups]))


def check(out, lse, q, k, v, table, lens, scale):
    ref_o, ref_l, a, s = op.decode(f64(q), f64(k), f64(v), table.cpu().numpy(), lens.cpu().numpy(), scale)
    u = 2.0 ** -23
    keys = max(int(lens.max()), 0)
    e = (q.shape[3] + 2) * u * s + 2 ** -21
    w = 2 ** -8 if out.dtype == BF16 else 2 ** -15
    o, l = f64(out), f64(lse)
    empty = np.isneginf(ref_l)
    assert np.array_equal(np.isneginf(l), empty)
    size = np.abs(np.where(empty, 0, ref_l))
    le = np.abs(np.where(empty, 0, l) - np.where(empty, 0, ref_l))
    lt = e + keys * u + 2 ** -20 + 4 * u * size
    assert (le <= lt).all(), (le / lt).max()
    tol = (2 * e + w + 2 * keys * u + 2 ** -19 + 4 * u * size).reshape(a.shape[0], 1, a.shape[2], 1) * a + 1e-38
    if out.dtype == BF16:
        tol = tol + 2 ** -8 * (np.abs(ref_o) + tol)
    err = np.abs(o - ref_o)
    assert (err <= tol).all(), (err / tol).max()
    assert not o[np.broadcast_to(empty.reshape(a.shape[0], 1, a.shape[2], 1), o.shape)].any()


def run(x, g, scale, **kw):
    import blockwise_exact_attention_gb300 as bea
    return bea.paged_decode_shared(*x, *g, scale, **kw)


HEADS = [(1, 1), (4, 4), (8, 2), (7, 1), (16, 1), (17, 1), (15, 5), (40, 2)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,h_kv", HEADS)
def test_heads(h, h_kv, d):
    import blockwise_exact_attention_gb300 as bea
    x, g = make([(400, [1, 0, 17, None, 300, 31, 2])], h, h_kv, d, 16, seed=h + d)
    scale = 1.0 / math.sqrt(d)
    out, lse = run(x, g, scale)
    assert out.dtype == BF16 and out.shape == x[0].shape and lse.shape == (7, h, 1)
    check(out, lse, *x, scale)
    out32, lse32 = run(x, g, scale, out_dtype=F32)
    check(out32, lse32, *x, scale)
    assert bea.device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,h,h_kv", [(31, 4, 1), (32, 4, 1), (33, 4, 1), (64, 4, 1), (65, 4, 1), (96, 4, 1), (97, 8, 2), (150, 4, 1),
                                      (300, 2, 2)])
def test_rows_around_the_units(n, h, h_kv, d):
    """Query rows that fill a half of a unit, a unit, or several, and end inside one."""
    rng = random.Random(n)
    x, g = make([(640, [rng.randint(0, 40) for _ in range(n)])], h, h_kv, d, 32, seed=n)
    out, lse = run(x, g, 0.1)
    check(out, lse, *x, 0.1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [1, 3, 4, 8, 16, 20, 24, 48, 64, 100, 128, 256, 1000])
def test_pages(page, d):
    x, g = make([(1000 // page * page + page, [0, 5, 130, page])], 4, 2, d, page, seed=page)
    out, lse = run(x, g, 0.2)
    check(out, lse, *x, 0.2)


@pytest.mark.parametrize("page", [2, 5, 7, 12, 30, 31, 50, 63, 65, 96, 126, 127, 129, 160, 192, 200, 513])
def test_pages_in_boxes_of_several_sizes(page):
    """Pages that end inside a tile, their rows in boxes of every power of two."""
    x, g = make([(1300 // page * page + page, [0, 9, 130]), (900 // page * page + page, [1, 70])], 6, 3, 64, page, seed=page)
    out, lse = run(x, g, 0.2)
    check(out, lse, *x, 0.2)


@pytest.mark.parametrize("shared", [0, 1, 127, 128, 129, 255, 256, 384, 385, 512, 1152, 5000])
def test_shared_lengths(shared):
    """None, less than a tile, odd and even numbers of tiles, cut over the CTAs and not."""
    x, g = make([(shared, [3, 0, 200, 1])], 8, 2, 128, 1, seed=shared)
    out, lse = run(x, g, 0.1)
    check(out, lse, *x, 0.1)


@pytest.mark.parametrize("n,h,h_kv", [(1100, 2, 1), (5, 300, 1)])
def test_more_than_one_round_of_the_rest(n, h, h_kv):
    """More requests, or more heads to a K/V head, than the kernel of the requests' own keys takes at once, some of them cut
    between CTAs."""
    rng = random.Random(n)
    own = [rng.choice([0, 1, 9, 700]) for _ in range(n)] if n < 100 else [1500 if i % 300 == 7 else i % 5 for i in range(n)]
    x, g = make([(256, own)], h, h_kv, 64, 16, seed=n)
    out, lse = run(x, g, 0.1)
    check(out, lse, *x, 0.1)
    out, lse = run(x, g, 0.1, out_dtype=F32)
    check(out, lse, *x, 0.1)


def test_a_cache_of_one_page_many_times():
    """An expanded cache, which cannot be copied by box: nothing is shared."""
    import blockwise_exact_attention_gb300 as bea
    k, v, q = draw((1, 16, 2, 64), 1), draw((1, 16, 2, 64), 2), draw((3, 1, 4, 64), 3)
    table, lens = torch.arange(60000, dtype=I32, device="cuda").repeat(3, 1) % 40, i32([600, 620, 630])
    x = (q, k.expand(40, 16, 2, 64), v.expand(40, 16, 2, 64), table, lens)
    got, want = run(x, (i32([0, 3]), i32([600])), 0.1), bea.paged_decode(*x, 0.1)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_small_tables_take_the_kernel_of_single_requests():
    import blockwise_exact_attention_gb300 as bea
    x, g = make([(400, [1, 17, 300])], 8, 2, 64, 16, seed=1, wide=False)
    out, lse = run(x, g, 0.1)
    want = bea.paged_decode(*x, 0.1)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_a_long_prefix_and_large_scores():
    x, g = make([(20000, [1, 700, 90])], 8, 2, 128, 64, seed=1, qscale=20.0)
    out, lse = run(x, g, 0.15)
    check(out, lse, *x, 0.15)
    again, lse2 = run(x, g, 0.15)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d", [64, 128])
def test_groups(d):
    """Several, empty ones, one request alone, nobody alive, rows of no group, and many more than the GPU has CTAs."""
    import blockwise_exact_attention_gb300 as bea
    x, (cuts, shared) = make([(300, [5, 6]), (0, [9]), (512, []), (700, [40, None, 3, 8]), (256, [None, None]), (900, [17]),
                              (128, [0] * 33)], 8, 2, d, 4, seed=d)
    check(*run(x, (cuts, shared), 0.1), *x, 0.1)
    check(*run(x, (cuts[1:6], shared[1:5]), 0.1), *x, 0.1)  # the first and the last rows in no group
    check(*run(x, (cuts[:1], shared[:0]), 0.1), *x, 0.1)    # no groups
    assert bea.device_status() == 0
    rng = random.Random(5)
    x, g = make([(rng.choice([128, 256, 400]), [rng.randint(0, 9) for _ in range(rng.choice([1, 2, 3]))]) for _ in range(400)],
                4, 4, d, 8, seed=6)
    check(*run(x, g, 0.1), *x, 0.1)
    assert bea.device_status() == 0


def test_no_more_is_shared_than_all_have():
    """A shared length past the shortest request's, and past the table."""
    import blockwise_exact_attention_gb300 as bea
    x, (cuts, _) = make([(512, [0, 400, None, 77])], 4, 1, 64, 16, seed=2)
    for shared in (512, 513, 700, 10 ** 6, 2 ** 31 - 1):
        short = x[4].clone()
        short[1] = 300                                   # of the first 512 keys
        y = (*x[:4], short)
        # rows 0, 1 and 3 have the same first 512 keys, whatever more is claimed of those that have no more
        if shared == 512:
            check(*run(y, (cuts, i32([shared])), 0.1), *y, 0.1)
        y = (*x[:4], i32([512, 300, 0, 512]))
        check(*run(y, (cuts, i32([shared])), 0.1), *y, 0.1)
        assert bea.device_status() == 0
    long = (*x[:4], i32([10 ** 6, 0, 0, 512]))           # past the table: counts as all of it, whose last page is none
    got = run(long, (cuts, i32([512])), 0.1)
    want = bea.paged_decode(*long, 0.1)
    assert bea.device_status() == PAGES
    assert (got[0].float() - want[0].float()).abs().max() <= 2 ** -6 and (got[1] - want[1]).abs()[[0, 3]].max() <= 1e-4


def test_wrong_groups_and_pages_are_reported():
    import blockwise_exact_attention_gb300 as bea
    x, (cuts, shared) = make([(400, [5, 6, 9]), (300, [7, 1])], 4, 2, 64, 16, seed=3)
    want = bea.paged_decode(*x, 0.1)
    for bad in ([0, 4, 3], [0, 3, 6], [-1, 3, 5], [5, 3, 0], [0, 2 ** 31 - 1, 5]):
        out, lse = run(x, (i32(bad), shared), 0.1)
        assert bea.device_status() == PAGES
        check(out, lse, *x, 0.1)
        assert torch.equal(out, want[0])                 # nothing shared
    out, lse = run(x, (cuts, i32([-5, 288])), 0.1)
    assert bea.device_status() == PAGES
    check(out, lse, *x, 0.1)
    for where, page in [(0, -1), (7, 10 ** 6), (12, -7), (24, 2 ** 31 - 1)]:
        table = x[3].clone()
        table[:3, where] = page                          # of the shared ones (24: of what is not a whole tile)
        y = (*x[:3], table, x[4])
        out, lse = run(y, (cuts, shared), 0.1)
        assert bea.device_status() == PAGES
        check(out, lse, *y, 0.1)


def test_strides_and_given_outputs():
    import blockwise_exact_attention_gb300 as bea
    (q, k, v, table, lens), g = make([(500, [5, 6, 0]), (300, [7, 100])], 8, 2, 128, 16, seed=4)
    want, wl = run((q, k, v, table, lens), g, 0.1)
    ks = k.transpose(1, 2).contiguous().transpose(1, 2)  # [pages, h_kv, page, d] in memory
    vs = torch.empty(v.shape[0], v.shape[1], 3, 2, 128, dtype=BF16, device="cuda")[:, :, 1].copy_(v)
    qs = torch.empty(5, 1, 12, 128, dtype=BF16, device="cuda")[:, :, 2:10].copy_(q)
    ts = torch.full((5, 2 * table.shape[1]), -1, dtype=I32, device="cuda")[:, :table.shape[1]].copy_(table)
    out = torch.zeros(5, 2, 10, 128, dtype=BF16, device="cuda")
    lse = torch.zeros(5, 8, 3, device="cuda")
    ws = torch.full((bea.paged_decode_shared_workspace_bytes(q, k, table, g[1]),), 255, dtype=torch.uint8, device="cuda")
    got = run((qs, ks, vs, ts, lens), g, 0.1, out=out[:, 1:, 1:9], lse=lse[..., 1:2], workspace=ws)
    assert torch.equal(got[0], want) and torch.equal(got[1], wl)
    assert not out[:, 0].any() and not out[:, 1, 0].any() and not lse[..., 0].any() and not lse[..., 2].any()
    with pytest.raises(bea._lib.BeaError, match="WORKSPACE"):
        run((q, k, v, table, lens), g, 0.1, workspace=ws[:-256])


def test_infinite_and_undefined_values():
    """An infinite value stays infinite in its column; what is no number spreads to its heads' rows only."""
    (q, k, v, table, lens), g = make([(256, [5, 6])], 4, 2, 64, 16, seed=5)
    page = int(table[0, 3])
    v[page, 2, 0, 7] = math.inf
    out, lse = run((q, k, v, table, lens), g, 0.1)
    assert (out[:, 0, :2, 7] == math.inf).all() and lse.isfinite().all()
    assert out[:, 0, 2:].isfinite().all() and out[:, 0, :2, :7].isfinite().all() and out[:, 0, :2, 8:].isfinite().all()
    k[page, 2, 1, 0] = math.nan
    out, lse = run((q, k, v, table, lens), g, 0.1)
    assert out[:, 0, 2:].isnan().all() and lse[:, 2:].isnan().all() and lse[:, :2].isfinite().all()
    k[page, 2, 1, 0] = 0
    k[:, :, 1], q[:, :, 2:] = -math.inf, 1.0              # every score of K/V head 1 is -inf
    out, lse = run((q, k, v, table, lens), g, 0.1)
    assert (lse[:, 2:] == -math.inf).all() and not out[:, 0, 2:].isnan().any()


def test_nothing_to_do():
    import blockwise_exact_attention_gb300 as bea
    (q, k, v, table, lens), g = make([(300, [5, 6])], 4, 2, 64, 16, seed=6)
    for y in [(q, k, v, table, lens * 0), (q, k[:0], v[:0], table, lens), (q, k, v, table[:, :0], lens)]:
        out, lse = run(y, g, 0.1)
        assert not out.any() and (lse == -math.inf).all()
    bea.device_status()
    out, lse = run((q[:0], k, v, table[:0], lens[:0]), (i32([0]), i32([])), 0.1)
    assert out.shape == (0, 1, 4, 64) and bea.device_status() == 0
    with pytest.raises(bea._lib.BeaError, match="UNSUPPORTED"):
        run((q.float(), k.float(), v.float(), table, lens), g, 0.1)
    with pytest.raises(bea._lib.BeaError, match="UNSUPPORTED"):
        run((q, k, v, table, lens), (i32([0] * 1025 + [2]), i32([0] * 1025)), 0.1)
    with pytest.raises(bea._lib.BeaError, match="SHAPE"):
        run((q, k, v, table, lens), (g[0], i32([0, 0])), 0.1)


def test_captured_and_replayed_with_other_lengths():
    import blockwise_exact_attention_gb300 as bea
    x, (cuts, shared) = make([(900, [50, 60, 70, 80, 20]), (700, [31, 600, 2])], 8, 2, 128, 16, seed=7)
    q, k, v, table, lens = x
    k.nan_to_num_(0.5), v.nan_to_num_(0.5, posinf=0.5)
    lens, cuts, shared = lens.clone(), cuts.clone(), shared.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run((q, k, v, table, lens), (cuts, shared), 0.1)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = run((q, k, v, table, lens), (cuts, shared), 0.1)
    start = lens.clone()
    for step in ([0] * 8, [-1, -5, -70, 0, -10, 0, -500, -1], None):
        lens.copy_(start + i32(step) if step else start * i32([1, 0, 1, 0, 0, 0, 1, 1]))
        shared.copy_(i32([896, 688]) if step else i32([500, 100]))
        graph.replay()
        check(out, lse, q, k, v, table, lens, 0.1)
    assert bea.device_status() == 0


def test_two_streams_at_once():
    import blockwise_exact_attention_gb300 as bea
    xs = [make([(3000, [50, 60, 70, 80, 20])], 8, 2, 128, 16, seed=s) for s in (8, 9)]
    want = [run(x, g, 0.1) for x, g in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(10):
        for (x, g), s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(run(x, g, 0.1))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for i, r in enumerate(got) for a, b in zip(r, want[i % 2])) and bea.device_status() == 0


def test_past_32_bit_offsets():
    page, h_kv, d = 64, 8, 128
    k = torch.zeros(40000, page, h_kv, d, dtype=BF16, device="cuda")  # 5.2 GB
    v = torch.zeros_like(k)
    ids = [39999, 5, 39000, 20000, 38000]
    k[ids], v[ids] = draw((5, page, h_kv, d), 1), draw((5, page, h_kv, d), 2)
    q = draw((3, 1, 16, d), 3)
    table = i32([[39999, 5, 39000, 20000] + [-1] * 200, [39999, 5, 39000, 20000] + [-1] * 200, [39999, 5, 39000, 38000] + [-1] * 200])
    lens = i32([256, 200, 230])
    out, lse = run((q, k, v, table, lens), (i32([0, 3]), i32([192])), 0.1)
    small = torch.zeros(40000, dtype=torch.long, device="cuda")
    small[ids] = torch.arange(5, device="cuda")
    check(out, lse, q, k[ids], v[ids], small[table[:, :4].long()].to(I32), lens, 0.1)


def test_forked_rows_decode_together():
    """The calls as they are used: a prompt, forks of it, steps of their own, and attention over what they share."""
    import blockwise_exact_attention_gb300 as bea
    h, h_kv, d, page, n, prompt = 8, 2, 128, 16, 6, 1000
    cache = bea.PagedKVCache(200, page, h_kv, d, n, 20000, share_pages=True)
    cache.k.fill_(math.nan), cache.v.fill_(math.nan)
    weight = [1 + draw((d,), 20 + i, 0.1).float() for i in range(2)]
    seq = [[] for _ in range(n)]

    def step(new, capacity, seed):
        plan = cache.plan(i32(new), capacity)
        q, k, v = draw((1, capacity, h, d), seed), draw((1, capacity, h_kv, d), seed + 1), draw((1, capacity, h_kv, d), seed + 2)
        q, k = bea.norm_rope_axes(q, k, plan.positions.view(1, 1, -1), (64,), *weight)
        cache.write(k, v, plan.slot_map)
        at = 0
        for r, a in enumerate(new):
            seq[r] = [] if a < 0 else seq[r] + [(k[0, at + i], v[0, at + i]) for i in range(a)]
            at += max(a, 0)
        return q

    step([prompt] + [0] * 5, prompt, 1)
    cache.fork(i32([-1, 0, 0, 0, 0, -1]))
    for r in range(1, 5):
        seq[r] = list(seq[0])
    groups, shared = i32([0, 5]), i32([prompt // page * page])
    for s, new in enumerate([[1, 1, 1, 1, 1, 0], [1, 1, -1, 1, 1, 40], [1, 0, 0, 1, 1, 1], [-1, 1, 0, 1, 1, 1]]):
        q = step(new, 64, 10 * s + 30)
        last, at = [], 0
        for a in new:
            at += max(a, 0)
            last.append(max(at - 1, 0))
        out, lse = cache.decode_shared(q[0, last].unsqueeze(1), groups, shared)
        for r in range(n):
            if not seq[r]:
                assert not out[r].any() and (lse[r] == -math.inf).all()
                continue
            k, v = (torch.stack([t[i] for t in seq[r]])[None] for i in (0, 1))
            ref, ref_lse = bea.flash_mha_fwd(q[:, last[r]:last[r] + 1], k.contiguous(), v.contiguous(), out_dtype=F32)
            # the forward's weights are bf16, 2^-9 of each
            assert (out[r].float() - ref[0]).abs().max() <= 2 ** -8 * ref.abs().max() + 2 ** -8 * v.float().abs().max()
            assert (lse[r] - ref_lse[0]).abs().max() <= 1e-3
    assert bea.device_status() == 0
    kept = cache.decode(q[0, last].unsqueeze(1))
    cache.compact(100)
    moved = cache.decode(q[0, last].unsqueeze(1))
    assert torch.equal(kept[0], moved[0]) and torch.equal(kept[1], moved[1]) and bea.device_status() == 0
