"""norm_rope_axes, norm_rotary_axes and the other layouts of rope_axes against
the fp64 definition.

Bounds, u = 2^-24 (half a step of fp32). A sum of d <= 256 squares in chains of
at most 16 products and 5 exchanges is within 21 u of the true one, its mean and
eps add 3 u, the root halves that and adds u: r is within 13 u, and y = x (r w)
within 15 u < 2^-20 of its value. Turned, an element is within e1 = 2^-20.9 + 2 u
(the amplitude) + |position| 2^-51 of a = amplitude (|y_i| + |y_k|), as for the
plain rotation, so the result is within a (2^-19 + |position| 2^-51).
Backward, with G the spread of |g| over the pairs and W the weights: gy = g' w is
within G W (e1 + u), sum(gy x) within S = sum(G W |x|) times (e1 + 21 u), its
factor r^2 / d adds 27 u: dx = r (gy - x c) is within r (G W + |x| r^2 S / d) (2^-18
+ |position| 2^-50). A weight's gradient is within T = sum over rows of G |x| r
times (e1 + 15 u + R u) for R rows. A bf16 result adds half a step, 2^-8 of its
value."""

import math

import numpy as np
import pytest

from oracle import norm_rope as on

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def draw(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (scale * torch.randn(shape, device="cuda", generator=g)).to(dtype)


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def close(got, ref, tol, dtype):
    if dtype == BF16:
        tol = tol + 2 ** -8 * (np.abs(ref) + tol)
    err = np.abs(f64(got) - ref)
    assert got.dtype == dtype and (err <= tol + 1e-37).all(), (err / (tol + 1e-37)).max()


def far(pos):
    return float(np.abs(pos).max(initial=0))


def check_fwd(got, x, w, pos, sections, dtype, norm=True, inverse=False, **how):
    rd, layout = how.get("rotary_dim") or x.shape[-1], how.get("layout", "half")
    if norm:
        ref = on.norm_turn(f64(x), f64(w), EPS, pos, sections, **how)
        y = on.norm_turn(f64(x), f64(w), EPS, pos, (0,), rotary_dim=0)
    else:
        ref = on.turn(f64(x), pos, sections, inverse=inverse, **how)
        y = f64(x)
    a = on.spread(y, rd, layout, how.get("amplitude", 1.0))
    close(got, ref, a * (2 ** -19 + far(pos) * 2.0 ** -51), dtype)


def check_bwd(dx, dw, x, w, g, pos, sections, dtype, **how):
    rd, layout = how.get("rotary_dim") or x.shape[-1], how.get("layout", "half")
    rx, rw = on.norm_turn_bwd(f64(x), f64(w), EPS, f64(g), pos, sections, **how)
    X = np.abs(f64(x))
    W = np.ones(x.shape[-1]) if w is None else np.abs(f64(w))
    G = on.spread(f64(g), rd, layout, how.get("amplitude", 1.0))
    r = 1 / np.sqrt((X ** 2).mean(-1, keepdims=True) + EPS)
    S = (G * W * X).sum(-1, keepdims=True)
    if dx is not None:
        close(dx, rx, r * (G * W + X * r ** 2 * S / x.shape[-1]) * (2 ** -18 + far(pos) * 2.0 ** -50), dtype)
    if dw is not None:
        T = (G * X * r).reshape(-1, x.shape[-1]).sum(0)
        rows = X.size // x.shape[-1]
        close(dw, rw, T * (2 ** -20.9 + 17 * 2 ** -24 + rows * 2 ** -24 + far(pos) * 2.0 ** -51), w.dtype)


def positions(n, l, axes, seed=3, top=5000):
    pos = np.random.default_rng(seed).integers(-100, top, (axes, n, l)).astype(np.int32)
    return pos, torch.from_numpy(pos).cuda()


SCALE = dict(kind="yarn", factor=4.0, original_max=512)
CASES = [
    # n, l, hq, hk, d, sections, how
    (1, 1, 1, 1, 16, (8,), {}),
    (2, 7, 4, 2, 64, (8, 12, 12), {}),
    (3, 33, 5, 1, 128, (32,), dict(rotary_dim=64)),
    (2, 65, 9, 8, 80, (10, 0, 14), dict(rotary_dim=48, spectrum="axis")),
    (2, 5, 3, 3, 256, (128,), dict(layout="interleaved")),
    (65, 1, 17, 0, 32, (1, 6), dict(rotary_dim=14, layout="interleaved")),
    (1, 130, 6, 2, 96, (1,), dict(rotary_dim=2, layout="interleaved")),
    (4, 9, 2, 1, 48, (0,), dict(rotary_dim=0)),
    (2, 40, 8, 2, 128, (64,), dict(scaling=SCALE)),
    (2, 17, 4, 4, 64, (16,), dict(rotary_dim=32, layout="interleaved", scaling=SCALE)),
]


def split(how):
    """(what the package takes, what the oracle takes)."""
    import blockwise_exact_attention_gb300 as bea
    own, ora = dict(how), dict(how)
    if "scaling" in how:
        own["scaling"] = bea.RopeScaling(**how["scaling"])
        ora.pop("scaling")
        ora |= how["scaling"] | dict(amplitude=0.1 * math.log(how["scaling"]["factor"]) + 1)
    return own, ora


@pytest.mark.parametrize("dtype,wtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, None)])
@pytest.mark.parametrize("n,l,hq,hk,d,sections,how", CASES)
def test_norm_and_gradients(n, l, hq, hk, d, sections, how, dtype, wtype):
    import blockwise_exact_attention_gb300 as bea
    own, ora = split(how)
    pos, p = positions(n, l, len(sections))
    x = [draw((n, l, hq, d), dtype, 1, 2.0), draw((n, l, hk, d), dtype, 2, 0.3) if hk else None]
    w = [None if wtype is None or (i and not hk) else (1 + draw((d,), F32, 5 + i, 0.3)).to(wtype) for i in range(2)]
    g = [draw((n, l, hq, d), dtype, 3), draw((n, l, hk, d), dtype, 4) if hk else None]
    out = bea.norm_rope_axes(*x, p, sections, *w, EPS, **own)
    leaves = [t.requires_grad_() for t in (*x, *w) if t is not None]
    traced = bea.norm_rotary_axes(*x, p, sections, *w, EPS, **own)
    for i in range(2):
        if x[i] is None:
            assert out[i] is None and traced[i] is None
            continue
        check_fwd(out[i], x[i], w[i], pos, sections, dtype, **ora)
        assert torch.equal(out[i], traced[i])
    outs = [t for t in traced if t is not None]
    grads = dict(zip(map(id, leaves), torch.autograd.grad(outs, leaves, [t for t in g if t is not None])))
    for i in range(2):
        if x[i] is not None:
            check_bwd(grads[id(x[i])], None if w[i] is None else grads[id(w[i])], x[i], w[i], g[i], pos, sections, dtype, **ora)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("n,l,hq,hk,d,sections,how", CASES[2:])
def test_layouts_without_norm(n, l, hq, hk, d, sections, how, inverse, dtype):
    import blockwise_exact_attention_gb300 as bea
    own, ora = split(how)
    pos, p = positions(n, l, len(sections))
    q, k = draw((n, l, hq, d), dtype, 1), draw((n, l, hk, d), dtype, 2) if hk else None
    qo, ko = bea.rope_axes(q, k, p, sections, inverse=inverse, **own)
    check_fwd(qo, q, None, pos, sections, dtype, norm=False, inverse=inverse, **ora)
    if hk:
        check_fwd(ko, k, None, pos, sections, dtype, norm=False, inverse=inverse, **ora)
    q.requires_grad_()
    g = draw(q.shape, dtype, 5)
    (dq,) = torch.autograd.grad(bea.rotary_axes(q, k, p, sections, **own)[0], q, g)
    check_fwd(dq, g, None, pos, sections, dtype, norm=False, inverse=True, **ora)


def test_many_rows_take_the_wide_kernel_and_the_same_values():
    """More rows than fill the GPU: eight heads a thread, and heads that do not fill a group."""
    import blockwise_exact_attention_gb300 as bea
    n, l, hq, hk, d = 2, 5000, 13, 3, 128
    pos, p = positions(n, l, 1, top=200000)
    q, k, w = draw((n, l, hq, d), BF16, 1), draw((n, l, hk, d), BF16, 2), draw((d,), F32, 3)
    qo, ko = bea.norm_rope_axes(q, k, p, (64,), w, None, EPS)
    rows = [0, 1, 2499, 4999]
    check_fwd(qo[:, rows], q[:, rows], w, pos[:, :, rows], (64,), BF16)
    check_fwd(ko[:, rows], k[:, rows], None, pos[:, :, rows], (64,), BF16)
    few, _ = bea.norm_rope_axes(q[:, :3], None, p[:, :, :3], (64,), w, None, EPS)
    assert torch.equal(few, qo[:, :3])                   # the narrow kernel's bits
    # a long sum for the weights, and the same bits from call to call
    q.requires_grad_(), k.requires_grad_(), w.requires_grad_()
    g = [draw(q.shape, BF16, 4), draw(k.shape, BF16, 5)]
    twice = [torch.autograd.grad(bea.norm_rotary_axes(q, k, p, (64,), w, None, EPS), (q, k, w), g) for _ in range(2)]
    assert all(torch.equal(a, b) for a, b in zip(*twice))
    check_bwd(twice[0][0][:, rows], None, q[:, rows], w, g[0][:, rows], pos[:, :, rows], (64,), BF16)
    check_bwd(None, twice[0][2], q, w, g[0], pos, (64,), BF16)


@pytest.mark.parametrize("d,how", [(64, dict(rotary_dim=32, layout="interleaved")), (80, dict(rotary_dim=48)),
                                   (256, dict(layout="interleaved")), (128, dict(rotary_dim=64)), (96, dict()),
                                   (48, dict(rotary_dim=2, layout="interleaved")), (16, dict(rotary_dim=0))])
def test_many_rows_in_every_layout(d, how):
    """Threads with several chunks, whose rows run ahead through shared memory: the bits of threads with one, in place too,
    and the gradients of rows anywhere."""
    import blockwise_exact_attention_gb300 as bea
    n, l, hq, hk = (2, 11000, 13, 6) if d < 256 else (1, 4001, 13, 6)
    sections = (how.get("rotary_dim", d) // 2,)
    pos, p = positions(n, l, 1, top=200000)
    q, k, w = draw((n, l, hq, d), BF16, 1, 2.0), draw((n, l, hk, d), BF16, 2, 0.3), draw((d,), F32, 3)
    qo, ko = bea.norm_rope_axes(q, k, p, sections, w, None, EPS, **how)
    rows = [0, 1, 2, l // 2, l - 2, l - 1]
    check_fwd(qo[:, rows], q[:, rows], w, pos[:, :, rows], sections, BF16, **how)
    check_fwd(ko[:, rows], k[:, rows], None, pos[:, :, rows], sections, BF16, **how)
    for at in range(0, l, 1000):                         # few enough for threads with one chunk
        part = slice(at, at + 1000)
        few = bea.norm_rope_axes(q[:1, part], k[:1, part], p[:, :1, part], sections, w, None, EPS, **how)
        assert torch.equal(few[0], qo[:1, part]) and torch.equal(few[1], ko[:1, part])
    g = [draw(q.shape, BF16, 4), draw(k.shape, BF16, 5)]
    leaves = [t.clone().requires_grad_() for t in (q, k, w)]
    grads = torch.autograd.grad(bea.norm_rotary_axes(*leaves[:2], p, sections, leaves[2], None, EPS, **how), leaves, g)
    check_bwd(grads[0][:, rows], None, q[:, rows], w, g[0][:, rows], pos[:, :, rows], sections, BF16, **how)
    check_bwd(grads[1][:, rows], None, k[:, rows], None, g[1][:, rows], pos[:, :, rows], sections, BF16, **how)
    small = slice(0, 50)
    dq, dk = (t.detach().clone().requires_grad_() for t in (q[:, small], k[:, small]))
    again = torch.autograd.grad(bea.norm_rotary_axes(dq, dk, p[:, :, small].contiguous(), sections, w, None, EPS, **how), (dq, dk),
                                [t[:, small] for t in g])
    assert torch.equal(again[0], grads[0][:, small]) and torch.equal(again[1], grads[1][:, small])
    bea.norm_rope_axes(q, k, p, sections, w, None, EPS, q_out=q, k_out=k, **how)
    assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_strides_and_in_place(layout):
    import blockwise_exact_attention_gb300 as bea
    n, l, hq, hk, d = 2, 19, 4, 2, 64
    pos, p = positions(n, l, 1)
    fused = draw((n, l, hq + 2 * hk, d), BF16, 1)
    q, k = fused[:, :, :hq], fused[:, :, hq:hq + hk]
    keep = fused.clone()
    how = dict(rotary_dim=32, layout=layout)
    qo, ko = bea.norm_rope_axes(q, k, p, (16,), **how, eps=EPS)
    check_fwd(qo, q, None, pos, (16,), BF16, **how)
    wide = torch.empty(n, l, hq, 2 * d, dtype=BF16, device="cuda").fill_(7)
    bea.norm_rope_axes(q, None, p, (16,), **how, eps=EPS, q_out=wide[..., d:])
    assert torch.equal(wide[..., d:], qo) and (wide[..., :d] == 7).all()
    swapped = q.transpose(1, 2).contiguous().transpose(1, 2)  # [n, h, l, d] in memory
    assert torch.equal(bea.norm_rope_axes(swapped, None, p, (16,), **how, eps=EPS)[0], qo)
    row = p[:, :1].expand(1, n, l)                       # one row of positions for the batch
    both = bea.norm_rope_axes(q[:1].expand(n, l, hq, d), None, row, (16,), **how, eps=EPS)[0]
    assert torch.equal(both[0], qo[0]) and torch.equal(both[1], qo[0])
    got = bea.norm_rope_axes(q, k, p, (16,), **how, eps=EPS, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(fused[:, :, hq + hk:], keep[:, :, hq + hk:])


def test_gradient_of_broadcast_and_strided_inputs():
    import blockwise_exact_attention_gb300 as bea
    n, l, h, d = 3, 11, 4, 64
    pos, p = positions(n, l, 1)
    one, w = draw((1, l, 1, d), F32, 1).requires_grad_(), draw((d,), F32, 2).requires_grad_()
    g = draw((n, l, h, d), F32, 3)
    out, none = bea.norm_rotary_axes(one.expand(n, l, h, d), None, p, (32,), w, eps=EPS)
    d1, dw = torch.autograd.grad(out, (one, w), g)
    rx, rw = on.norm_turn_bwd(f64(one.expand(n, l, h, d)), f64(w), EPS, f64(g), pos, (32,))
    assert none is None and np.allclose(f64(d1), rx.sum((0, 2), keepdims=True), rtol=1e-4, atol=1e-4)
    assert np.allclose(f64(dw), rw, rtol=1e-4, atol=1e-3)
    # gradients that autograd hands over expanded, of another layout, or to be negated
    x = draw((n, l, h, d), F32, 4).requires_grad_()
    (a,) = torch.autograd.grad(bea.norm_rotary_axes(x, None, p, (32,), w, eps=EPS)[0].sum(), x)
    check_bwd(a, None, x, w, torch.ones_like(x), pos, (32,), F32)
    t = torch.view_as_complex(torch.stack([g, g], -1)).conj().imag  # -g, the negation pending
    assert t.is_neg()
    (b,) = torch.autograd.grad(bea.norm_rotary_axes(x, None, p, (32,), w, eps=EPS)[0], x, t)
    check_bwd(b, None, x, w, -g, pos, (32,), F32)


def test_only_the_gradients_that_are_asked_for():
    import blockwise_exact_attention_gb300 as bea
    n, l, hq, hk, d = 2, 9, 4, 2, 64
    pos, p = positions(n, l, 1)
    q, k = draw((n, l, hq, d), BF16, 1), draw((n, l, hk, d), BF16, 2)
    qw, kw = draw((d,), BF16, 3), draw((d,), F32, 4)
    gq, gk = draw(q.shape, BF16, 5), draw(k.shape, BF16, 6)
    want = {}
    for t in (q, k, qw, kw):
        t.requires_grad_()
    out = bea.norm_rotary_axes(q, k, p, (32,), qw, kw, EPS)
    want = torch.autograd.grad(out, (q, k, qw, kw), (gq, gk))
    (only,) = torch.autograd.grad(bea.norm_rotary_axes(q, k, p, (32,), qw, kw, EPS), kw, (gq, gk))
    assert torch.equal(only, want[3])
    dk, dkw = torch.autograd.grad(bea.norm_rotary_axes(q, k, p, (32,), qw, kw, EPS)[1], (k, kw), gk)
    assert torch.equal(dk, want[1]) and torch.equal(dkw, want[3])
    (dq,) = torch.autograd.grad(bea.norm_rotary_axes(q, k.detach(), p, (32,), qw.detach(), kw.detach(), EPS), q, (gq, gk),
                                allow_unused=True)
    assert torch.equal(dq, want[0])
    same = bea.norm_rotary_axes(q, k, p, (32,), qw, qw, EPS)  # one weight for both
    (dw,) = torch.autograd.grad(same, qw, (gq, gk))
    parts = [torch.autograd.grad(bea.norm_rotary_axes(q, k, p, (32,), qw, qw, EPS)[i], qw, g)[0] for i, g in ((0, gq), (1, gk))]
    assert torch.equal(dw, parts[0] + parts[1])
    with torch.no_grad():
        assert not bea.norm_rotary_axes(q, k, p, (32,), qw, kw, EPS)[0].requires_grad
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(bea.norm_rotary_axes(q, k, p, (32,), qw, kw, EPS), q, (gq, gk), create_graph=True)
    y = bea.norm_rotary_axes(q, k, p, (32,), qw, kw, EPS)
    with torch.no_grad():
        q.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        torch.autograd.grad(y, q, (gq, gk))


def test_rows_of_zeros_and_values_that_are_no_numbers():
    import blockwise_exact_attention_gb300 as bea
    _, p = positions(1, 4, 1)
    q = draw((1, 4, 2, 64), F32, 1)
    q[0, 0, 0] = 0
    q[0, 1, 0, 5] = math.nan                             # of the turned half: its row only
    q[0, 2, 1, 40] = math.inf                            # of the rest
    out, _ = bea.norm_rope_axes(q, None, p, (16,), rotary_dim=32)
    assert (out[0, 0, 0] == 0).all()
    assert out[0, 1, 0].isnan().all() and out[0, 1, 1].isfinite().all() and out[0, 3].isfinite().all()
    for layout in ("half", "interleaved"):
        turned, _ = bea.rope_axes(q, None, p, (16,), rotary_dim=32, layout=layout)
        assert turned[0, 2, 1, 40] == math.inf and turned[0, 2].isfinite().sum() == 127
        assert turned[0, 1, 0].isnan().sum() == 2 and torch.equal(turned[..., 32:], q[..., 32:])
    x = q.clone().requires_grad_()
    (dx,) = torch.autograd.grad(bea.norm_rotary_axes(x, None, p, (32,))[0].sum(), x)
    assert dx[0, 0, 0].isfinite().all() and dx[0, 3].isfinite().all()


def test_empty_and_refused():
    import blockwise_exact_attention_gb300 as bea
    _, p = positions(2, 0, 1)
    q, w = torch.empty(2, 0, 4, 64, device="cuda", requires_grad=True), torch.ones(64, device="cuda", requires_grad=True)
    out, _ = bea.norm_rotary_axes(q, None, p, (32,), w)
    dq, dw = torch.autograd.grad(out, (q, w), torch.empty_like(out))
    assert out.shape == q.shape and dq.shape == q.shape and (dw == 0).all()
    _, p = positions(2, 3, 1)
    q = draw((2, 3, 4, 64), BF16, 1)
    with pytest.raises(ValueError, match="sections"):
        bea.norm_rope_axes(q, None, p[:0], (32,))
    with pytest.raises(bea._lib.BeaError, match="UNSUPPORTED"):
        bea.norm_rope_axes(q, None, p, (15,), rotary_dim=30)
    with pytest.raises(bea._lib.BeaError, match="SHAPE"):
        bea.norm_rope_axes(q, None, p, (32,), torch.ones(32, device="cuda"))
    with pytest.raises(bea._lib.BeaError, match="ARG"):
        bea.norm_rope_axes(q, None, p, (32,), None, torch.ones(64, device="cuda"))
    with pytest.raises(ValueError, match="requires grad"):
        bea.norm_rope_axes(q, None, p, (32,), q_out=torch.empty_like(q).requires_grad_())


def test_captured_training_step_and_streams():
    import blockwise_exact_attention_gb300 as bea
    n, l, h, d = 2, 64, 4, 128
    pos, p = positions(n, l, 1)
    x, w, g = draw((n, l, h, d), BF16, 1), draw((d,), F32, 2), draw((n, l, h, d), BF16, 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        xs, ws = x.clone().requires_grad_(), w.clone().requires_grad_()

        def step():
            out, _ = bea.norm_rotary_axes(xs, None, p, (64,), ws, eps=EPS)
            return (out.detach(), *torch.autograd.grad(out, (xs, ws), g))

        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step()
        for seed in (4, 5):
            with torch.no_grad():
                xs.copy_(draw(x.shape, BF16, seed))
            graph.replay()
            side.synchronize()
            check_fwd(got[0], xs, ws, pos, (64,), BF16)
            check_bwd(got[1], got[2], xs, ws, g, pos, (64,), BF16)
    torch.cuda.synchronize()
    y = x.clone().requires_grad_()
    alive = bea.norm_rotary_axes(y, None, p, (64,))[0]   # made on the default stream
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        with pytest.raises(RuntimeError, match="norm_rotary_axes: captured"):
            bea.norm_rotary_axes(y, None, p, (64,))
    del alive


def test_past_32_bit_offsets():
    """Rows behind 2^32 bytes, of a view that skips between its tokens."""
    import blockwise_exact_attention_gb300 as bea
    l, h, d = 33, 2, 64
    gap = torch.empty(l, 2 ** 27, dtype=BF16, device="cuda")  # 8.9 GB, of which little is touched
    x = gap.as_strided((1, l, h, d), (0, 2 ** 27, d, 1))
    x.copy_(draw((1, l, h, d), BF16, 1))
    pos, p = positions(1, l, 1)
    check_fwd(bea.norm_rope_axes(x, None, p, (32,), eps=EPS)[0], x, None, pos, (32,), BF16)
    bea.norm_rope_axes(x, None, p, (32,), eps=EPS, q_out=x)
    x0 = draw((1, l, h, d), BF16, 1)
    check_fwd(x, x0, None, pos, (32,), BF16)
