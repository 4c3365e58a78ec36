"""The angles of rope_axes, and its kernels for many heads and many rows.

u = 1, v = 0 turn to (cos, sin) as the kernel has them. The angle less its nearest quarter turn is at most a quarter of
a half turn, so rounding it to fp32 is off by at most 2^-27 half turns, 2^-25.34 radians, and its 32 bits before that by
2^-31.3 radians; sincospif is good to one unit in the last place, 2^-24 of values below 1; the fixed-point step is off by
2^-65 turns and 2^-52 of itself, which the positions here keep below 2^-36 with the oracle's own rounding: 2^-24 +
2^-25.34 + 2^-31.3 + 2^-36 < 2^-23.5 in all."""

import numpy as np
import pytest

from oracle import paged as op

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def draw(shape, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, dtype=dtype, device="cuda", generator=g)


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("base", [10000.0, 1.0])
def test_cosines_and_sines(base, inverse):
    import blockwise_exact_attention_gb300 as bea
    l, d = 4000, 64
    x = torch.zeros((1, l, 1, d), dtype=F32, device="cuda")
    x[..., :d // 2] = 1
    pos = np.random.default_rng(1).integers(-2 ** 16, 2 ** 16, (1, 1, l)).astype(np.int32)
    pos[0, 0, :4] = 0, 1, -1, 2
    y = bea.rope_axes(x, None, torch.from_numpy(pos).cuda(), (d // 2,), base, inverse=inverse)[0]
    ref = op.rope_axes(x.double().cpu().numpy(), pos, (d // 2,), base, inverse=inverse)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert err.max() <= 2 ** -23.5, err.max() * 2 ** 24
    assert (y[0, 0, 0, :d // 2] == 1).all() and (y[0, 0, 0, d // 2:] == 0).all()     # position 0 turns nothing


def turned(pos, freqs, inverse=0):
    """(cos, sin) of every position (rows) by every frequency, from the C entry point."""
    import ctypes
    import blockwise_exact_attention_gb300 as bea
    from blockwise_exact_attention_gb300 import _lib
    m, half = len(pos), len(freqs)
    x = torch.zeros((1, m, 1, 2 * half), dtype=F32, device="cuda")
    x[..., :half] = 1
    y = torch.empty_like(x)
    p = torch.tensor(pos, dtype=I32, device="cuda")[None, None]
    t = lambda z, code: _lib.describe(z.data_ptr(), code, z.shape, z.stride())  # noqa: E731
    rc = _lib.load().bea_rope_axes(t(x, 1), None, t(p, 2), (ctypes.c_int32 * half)(), (ctypes.c_double * half)(*freqs), inverse,
                                   t(y, 1), None, torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and bea.device_status() == 0
    y = y[0, :, 0].double().cpu().numpy()
    return y[:, :half], y[:, half:]


def test_whole_quarters_are_exact():
    """Steps of an eighth of a turn (pi / 4 as a double is one within 2^-54: its fixed-point step is exact): cosines and
    sines of the quarters without an error."""
    for sign in (1, -1):
        for inverse in (0, 1):
            c, s = turned(range(-8, 9), [sign * np.pi / 4] * 4, inverse)
            for i, p in enumerate(range(-8, 9)):
                if p % 2 == 0:
                    want = [(1, 0), (0, 1), (-1, 0), (0, -1)][p // 2 * sign * (-1) ** inverse % 4]
                    assert (c[i] == want[0]).all() and (s[i] == want[1]).all(), p


def test_small_frequencies_of_either_sign_at_far_positions():
    """At 2^31 the fixed-point step's 2^-65 turns are 2^-31.3 radians, 2^-52 of an angle below 2^21 are 2^-31, and the fp64
    product below is off by 2^-32: with the 2^-23.5 above less than 2^-23.4 in all."""
    freqs = [1e-3, 1e-5, 3e-7, 2.0 ** -40] + [-1e-3, -1e-5, -3e-7, -2.0 ** -40]
    pos = [2 ** 31 - 1, -(2 ** 31), 2 ** 30 + 12345, -123456789, 1, -1, 0]
    ang = np.array(pos, dtype=np.float64)[:, None] * np.array(freqs)
    for inverse in (0, 1):
        c, s = turned(pos, freqs, inverse)
        assert np.abs(c - np.cos(ang)).max() <= 2 ** -23.4
        assert np.abs(s - np.sin(ang) * (-1) ** inverse).max() <= 2 ** -23.4


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 64), (BF16, 80), (F32, 24)])
@pytest.mark.parametrize("inverse", [False, True])
def test_many_rows(dtype, d, inverse):
    """As many rows as the kernel for eight heads a thread takes; the last heads of q and the first of k in one group.
    The same bits as in slices, which the kernel for four heads turns, and the oracle's values where they are asked."""
    import blockwise_exact_attention_gb300 as bea
    hq, hk = 9, 4
    pieces = d // 2 // (4 if dtype == F32 else 8)
    l = 152 * 2048 // (2 * pieces) + 33
    qkv = draw((1, l, hq + 2 * hk, d), dtype, 2)
    q, k, v = qkv.split((hq, hk, hk), 2)
    keep = v.clone()
    half = d // 2
    sections = (half // 4, 0, half - half // 4)
    pos = torch.randint(-5000, 5000, (3, 1, l), dtype=I32, device="cuda")
    qo, ko = bea.rope_axes(q, k, pos, sections, spectrum="axis", inverse=inverse)
    step = l // 5 + 1
    for at in range(0, l, step):
        part = slice(at, min(at + step, l))
        a, b = bea.rope_axes(q[:, part], k[:, part], pos[:, :, part], sections, spectrum="axis", inverse=inverse)
        assert torch.equal(a, qo[:, part]) and torch.equal(b, ko[:, part])
    few = [0, 1, l // 2, l - 2, l - 1]
    u = 2.0 ** -8 if dtype == BF16 else 0.0
    for x, y in ((q, qo), (k, ko)):
        xs = x[:, few].double().cpu().numpy()
        ref = op.rope_axes(xs, pos[:, :, few].cpu().numpy(), sections, spectrum="axis", inverse=inverse)
        r = np.abs(xs)
        r = np.concatenate([r[..., :half] + r[..., half:]] * 2, -1)
        # a cosine and a sine within 2^-23.5, two roundings of 2^-24; then the output's
        tol = r * (2 ** -23.5 + 2 ** -23) + u * np.abs(ref) * (1 + 2 ** -8) + 1e-38
        assert (np.abs(y[:, few].double().cpu().numpy() - ref) <= tol).all()
    bea.rope_axes(q, k, pos, sections, spectrum="axis", inverse=inverse, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, keep)


def test_more_work_than_32_bits_count():
    """2^31 pieces: rows that share one row of memory in, 69 GB out."""
    import blockwise_exact_attention_gb300 as bea
    if torch.cuda.mem_get_info()[0] < 90e9:
        pytest.skip("needs 90 GB")
    d, l = 256, 2 ** 27 + 1001
    q = draw((1, 1, 1, d), BF16, 3).expand(1, l, 1, d)
    pos = torch.arange(l, dtype=I32, device="cuda")[None, None]
    out, _ = bea.rope_axes(q, None, pos, (d // 2,))
    step = 2 ** 22
    for at in range(0, l, step):
        part = slice(at, min(at + step, l))
        assert torch.equal(bea.rope_axes(q[:, part], None, pos[:, :, part], (d // 2,))[0], out[:, part]), at
    del out
    torch.cuda.empty_cache()


def test_write_of_more_pieces_than_32_bits_count():
    import blockwise_exact_attention_gb300 as bea
    h_kv, d, page, pages = 64, 256, 16, 8
    l = 2 ** 20 + 77                                        # of 2^11 pieces each
    k, v = (draw((1, 1, h_kv, d), BF16, s).expand(1, l, h_kv, d) for s in (4, 5))
    slots = torch.full((l,), -1, dtype=I32, device="cuda")
    to = {0: 5, 1: 100, 2 ** 19: 17, 2 ** 20 - 1: 99, 2 ** 20: 3, 2 ** 20 + 1: 127, l - 1: 64}
    for t, s in to.items():
        slots[t] = s
    kc, vc = (torch.zeros((pages, page, h_kv, d), dtype=BF16, device="cuda") for _ in range(2))
    bea.paged_write(k, v, slots, kc, vc)
    for cache, new in ((kc, k), (vc, v)):
        flat = cache.view(-1, h_kv, d)
        hit = torch.zeros(pages * page, dtype=torch.bool, device="cuda")
        hit[list(to.values())] = True
        assert (flat[hit] == new[0, 0]).all() and not flat[~hit].any()
    assert bea.device_status() == 0


def test_a_gradient_with_a_pending_negation():
    """Autograd may hand over a view whose negation is pending (the imaginary part of a conjugate)."""
    import blockwise_exact_attention_gb300 as bea
    q = draw((1, 5, 2, 16), F32, 6).requires_grad_()
    p = torch.arange(5, dtype=I32, device="cuda")[None, None]
    g = draw((1, 5, 2, 16), F32, 7)
    (dq,) = torch.autograd.grad(bea.rotary_axes(q, None, p, (8,))[0], q, torch._neg_view(g))
    assert torch.equal(dq, bea.rope_axes(-g, None, p, (8,), inverse=True)[0])
    k = draw((1, 5, 1, 16), F32, 8).requires_grad_()
    dq, dk = torch.autograd.grad(bea.rotary_axes(q, k, p, (8,)), (q, k), (g, torch._neg_view(g[:, :, :1])))
    assert torch.equal(dk, bea.rope_axes(-g[:, :, :1], None, p, (8,), inverse=True)[0])
