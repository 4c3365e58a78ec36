"""rope_axes and rotary_axes against the fp64 definition.

Bounds. u' = u c - v s in fp32 from a cosine and sine that are within 2^-22 of
the true ones (sincospif is good to 2 units in the last place, 2^-23, of values
at most 1; the angle itself is within 2^-25 half turns, 2^-23.3 radians): with r
= |u| + |v| the fp32 value is within r (2^-22 + 2^-23.3 + 2 * 2^-24) < r 2^-20.9
of the true one, and far positions add |position| 2^-51 r at most. A bf16 result
adds half a step, 2^-8 of the value."""

import math

import numpy as np
import pytest

from oracle import paged as op

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


BF16, F32 = torch.bfloat16, torch.float32


def draw(shape, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, dtype=dtype, device="cuda", generator=g)


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def check(got, x, pos, sections, dtype, **kw):
    ref = op.rope_axes(f64(x), pos, sections, **kw)
    half = x.shape[-1] // 2
    r = np.abs(f64(x))
    r = np.concatenate([r[..., :half] + r[..., half:]] * 2, -1)
    tol = r * (2 ** -20.9 + np.abs(pos).max(initial=0) * 2.0 ** -51) + 1e-38
    if dtype == BF16:
        tol = tol + 2 ** -8 * (np.abs(ref) + tol)
    err = np.abs(f64(got) - ref)
    assert got.dtype == dtype and (err <= tol).all(), (err / tol).max()


CASES = [
    # n, l, hq, hk, d, sections, spectrum
    (1, 1, 1, 1, 16, (8,), "joint"),
    (2, 7, 4, 2, 64, (8, 12, 12), "joint"),
    (3, 33, 5, 1, 128, (16, 24, 24), "joint"),
    (1, 129, 9, 8, 80, (10, 0, 30), "axis"),
    (2, 5, 3, 3, 256, (32, 32, 32, 32), "axis"),
    (65, 1, 17, 0, 32, (1, 15), "axis"),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,l,hq,hk,d,sections,spectrum", CASES)
@pytest.mark.parametrize("inverse", [False, True])
def test_matches_the_definition(n, l, hq, hk, d, sections, spectrum, inverse, dtype):
    import blockwise_exact_attention_gb300 as bea
    q, k = draw((n, l, hq, d), dtype, 1), draw((n, l, hk, d), dtype, 2) if hk else None
    pos = np.random.default_rng(3).integers(-100, 5000, (len(sections), n, l)).astype(np.int32)
    p = torch.from_numpy(pos).cuda()
    qo, ko = bea.rope_axes(q, k, p, sections, spectrum=spectrum, inverse=inverse)
    check(qo, q, pos, sections, dtype, spectrum=spectrum, inverse=inverse)
    if hk:
        check(ko, k, pos, sections, dtype, spectrum=spectrum, inverse=inverse)
    else:
        assert ko is None


def test_f32_head_dim_of_eight():
    import blockwise_exact_attention_gb300 as bea
    q = draw((2, 3, 2, 24), F32, 4)
    pos = np.arange(6, dtype=np.int32).reshape(1, 2, 3)
    check(bea.rope_axes(q, None, torch.from_numpy(pos).cuda(), (12,))[0], q, pos, (12,), F32)


def test_far_positions_and_other_bases():
    import blockwise_exact_attention_gb300 as bea
    q = draw((1, 6, 2, 64), F32, 5)
    pos = np.array([[[0, 1, -(2 ** 31), 2 ** 31 - 1, 123456789, -7]]], dtype=np.int32)
    p = torch.from_numpy(pos).cuda()
    for base in (10000.0, 500000.0, 1.0, 0.5):          # 0.5: frequencies above one radian a position
        check(bea.rope_axes(q, None, p, (32,), base)[0], q, pos, (32,), F32, base=base)


def test_strides_broadcast_positions_and_in_place():
    import blockwise_exact_attention_gb300 as bea
    n, l, hq, hk, d = 2, 19, 6, 2, 64
    sections = (8, 24)
    qkv = draw((n, l, hq + 2 * hk, d), BF16, 6)
    keep = qkv.clone()
    q, k, v = qkv.split((hq, hk, hk), 2)                # views of one fused projection
    pos = np.random.default_rng(7).integers(0, 99, (2, 1, l)).astype(np.int32)
    p = torch.from_numpy(pos).cuda().expand(2, n, l)
    full = np.broadcast_to(pos, (2, n, l))
    qo, ko = bea.rope_axes(q, k, p, sections)
    check(qo, q, full, sections, BF16)
    check(ko, k, full, sections, BF16)
    out = torch.full((n, l, hq, 2 * d), 7.0, dtype=BF16, device="cuda")
    bea.rope_axes(q, None, p, sections, q_out=out[..., :d])
    assert torch.equal(out[..., :d], qo) and (out[..., d:] == 7).all()
    xt = q.transpose(1, 2).contiguous().transpose(1, 2)  # heads before the sequence in memory
    assert torch.equal(bea.rope_axes(xt, None, p, sections)[0], qo)
    assert torch.equal(bea.rope_axes(q[:1].expand(n, l, hq, d), None, p, sections)[0][1], qo[0])
    bea.rope_axes(q, k, p, sections, q_out=q, k_out=k)   # in place, in the fused tensor
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, keep[:, :, hq + hk:])
    back, _ = bea.rope_axes(q.float(), None, p, sections, inverse=True)
    assert (back - keep[:, :, :hq].float()).abs().max() <= 2 ** -8 * 2 * keep.float().abs().max()


def test_offsets_past_32_bits():
    import blockwise_exact_attention_gb300 as bea
    l, h, d = 70001, 256, 128                            # 2.3e9 elements
    q = torch.zeros((1, l, h, d), dtype=BF16, device="cuda")
    q[0, -3:] = draw((3, h, d), BF16, 8)
    pos = torch.arange(l, dtype=torch.int32, device="cuda")[None, None]
    out, _ = bea.rope_axes(q, None, pos, (64,))
    check(out[:, -3:], q[:, -3:], f64(pos[:, :, -3:]), (64,), BF16)
    assert not out[0, :-3].any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients(dtype):
    import blockwise_exact_attention_gb300 as bea
    n, l, hq, hk, d, sections = 2, 13, 4, 2, 64, (8, 12, 12)
    q, k = draw((n, l, hq, d), dtype, 9).requires_grad_(), draw((n, l, hk, d), dtype, 10).requires_grad_()
    gq, gk = draw((n, l, hq, d), dtype, 11), draw((n, l, hk, d), dtype, 12)
    pos = np.random.default_rng(13).integers(0, 300, (3, n, l)).astype(np.int32)
    p = torch.from_numpy(pos).cuda()
    qo, ko = bea.rotary_axes(q, k, p, sections)
    dq, dk = torch.autograd.grad((qo, ko), (q, k), (gq, gk))
    check(dq, gq, pos, sections, dtype, inverse=True)
    check(dk, gk, pos, sections, dtype, inverse=True)
    # one gradient alone, an expanded gradient, a broadcast input, no k
    (dk2,) = torch.autograd.grad(bea.rotary_axes(q, k, p, sections)[1], k, gk)
    assert torch.equal(dk2, dk)
    (dq2,) = torch.autograd.grad(bea.rotary_axes(q, k, p, sections)[0].sum(), q)
    check(dq2, torch.ones_like(q), pos, sections, dtype, inverse=True)
    one = q.detach()[:1].clone().requires_grad_()
    out, none = bea.rotary_axes(one.expand(n, l, hq, d), None, p, sections)
    assert none is None
    (d1,) = torch.autograd.grad(out, one, gq)
    assert torch.allclose(d1, dq.float().sum(0, keepdim=True).to(dtype), atol=2 ** -6, rtol=2 ** -6)
    assert bea.device_status() == 0


def test_gradient_by_differences():
    import blockwise_exact_attention_gb300 as bea
    q, g = draw((1, 4, 2, 32), F32, 14).requires_grad_(), draw((1, 4, 2, 32), F32, 15)
    p = torch.tensor([[[0, 3, 50, 7]], [[2, 0, 1, 99]]], dtype=torch.int32, device="cuda")
    (dq,) = torch.autograd.grad(bea.rotary_axes(q, None, p, (4, 12))[0], q, g)
    for at in [(0, 1, 0, 3), (0, 3, 1, 20), (0, 2, 0, 31)]:
        step = torch.zeros_like(q)
        step[at] = 0.5                                  # linear in q: no truncation error
        with torch.no_grad():
            hi, lo = (bea.rotary_axes(q + s, None, p, (4, 12))[0] for s in (step, -step))
        diff = ((hi - lo).double() * g.double()).sum().item()
        # the two rows' roundings: at most 2^-20.9 (|u| + |v|) |g| each, |x| < 5 here
        assert abs(diff - dq[at].item()) <= 2 * 2 * 2 ** -20.9 * 10 * 5


def test_gradient_of_the_gradient():
    import blockwise_exact_attention_gb300 as bea
    q, g = draw((1, 3, 2, 16), F32, 16).requires_grad_(), draw((1, 3, 2, 16), F32, 17).requires_grad_()
    p = torch.arange(3, dtype=torch.int32, device="cuda")[None, None]
    out, _ = bea.rotary_axes(q, None, p, (8,))
    (dq,) = torch.autograd.grad(out, q, g, create_graph=True)
    w = draw((1, 3, 2, 16), F32, 18)
    (dg,) = torch.autograd.grad(dq, g, w)
    assert torch.equal(dg, bea.rope_axes(w, None, p, (8,))[0])


def test_captured_forward_and_backward_replay():
    import blockwise_exact_attention_gb300 as bea
    n, l, h, d = 1, 40, 4, 64
    q = draw((n, l, h, d), BF16, 19).requires_grad_()
    g = draw((n, l, h, d), BF16, 20)
    p = torch.arange(l, dtype=torch.int32, device="cuda").expand(1, n, l)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, _ = bea.rotary_axes(q, None, p, (32,))
        torch.autograd.grad(out, q, g)
    torch.cuda.current_stream().wait_stream(side)
    del out
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = bea.rotary_axes(q, None, p, (32,))
        (dq,) = torch.autograd.grad(out, q, g)
    for seed in (21, 22):
        with torch.no_grad():
            q.copy_(draw((n, l, h, d), BF16, seed))
            g.copy_(draw((n, l, h, d), BF16, seed + 10))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.detach(), bea.rope_axes(q.detach(), None, p, (32,))[0])
        assert torch.equal(dq, bea.rope_axes(g, None, p, (32,), inverse=True)[0])


def test_capture_over_a_live_eager_graph_is_refused():
    """Its backward pass would end the process: the forward call refuses."""
    import blockwise_exact_attention_gb300 as bea
    q = draw((1, 4, 2, 32), BF16, 25).requires_grad_()
    p = torch.arange(4, dtype=torch.int32, device="cuda").expand(1, 1, 4)
    out, _ = bea.rotary_axes(q, None, p, (16,))           # on the default stream, kept alive
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="captured"):
            bea.rotary_axes(q, None, p, (16,))
        inside, _ = bea.rope_axes(q, None, p, (16,))      # the plain call has no such tie
    del out
    again = torch.cuda.CUDAGraph()
    with torch.cuda.graph(again):
        out, _ = bea.rotary_axes(q, None, p, (16,))
    again.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, inside)


def test_written_tensors_are_known_to_autograd():
    import blockwise_exact_attention_gb300 as bea
    q = draw((1, 3, 2, 16), F32, 26).requires_grad_()
    p = torch.arange(3, dtype=torch.int32, device="cuda").expand(1, 1, 3)
    with pytest.raises(ValueError, match="requires grad"):
        bea.rope_axes(q, None, p, (8,), q_out=q)
    x = q * 1.0
    y = (x * x).sum()                                     # keeps x for its gradient
    with torch.no_grad():
        bea.rope_axes(x, None, p, (8,), q_out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    out, _ = bea.rotary_axes(q, None, p2 := p.contiguous(), (8,))
    p2.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
    before = x._version
    with torch.no_grad(), pytest.raises(RuntimeError, match="SHAPE"):   # a refused call writes nothing
        bea.rope_axes(x[:, :2], None, p, (8,), q_out=x)
    assert x._version == before
    with torch.inference_mode():
        z = q.clone()
        bea.rope_axes(z, None, p, (8,), q_out=z)
    assert torch.equal(z, bea.rope_axes(q.detach(), None, p, (8,))[0])


def test_no_forward_mode():
    import blockwise_exact_attention_gb300 as bea
    from torch.autograd import forward_ad
    q = draw((1, 3, 2, 16), F32, 27)
    p = torch.arange(3, dtype=torch.int32, device="cuda").expand(1, 1, 3)
    with forward_ad.dual_level():
        with pytest.raises(NotImplementedError):
            bea.rotary_axes(forward_ad.make_dual(q, q), None, p, (8,))


def test_launches_are_counted():
    import blockwise_exact_attention_gb300 as bea
    q = draw((1, 3, 2, 16), F32, 28).requires_grad_()
    p = torch.arange(3, dtype=torch.int32, device="cuda").expand(1, 1, 3)
    bea.launches_since_reset(reset=True)
    out, _ = bea.rotary_axes(q, None, p, (8,))
    assert bea.launches_since_reset() == 1
    torch.autograd.grad(out.sum(), q)
    assert bea.launches_since_reset(reset=True) == 2 and bea.launches_since_reset() == 0


def test_pending_negation_is_refused():
    import blockwise_exact_attention_gb300 as bea
    q = torch._neg_view(draw((1, 3, 2, 16), F32, 29))
    p = torch.arange(3, dtype=torch.int32, device="cuda").expand(1, 1, 3)
    with pytest.raises(ValueError, match="resolve_neg"):
        bea.rope_axes(q, None, p, (8,))


def test_another_stream():
    import blockwise_exact_attention_gb300 as bea
    q = draw((1, 500, 8, 128), BF16, 23)
    p = torch.arange(500, dtype=torch.int32, device="cuda").expand(1, 1, 500)
    want, _ = bea.rope_axes(q, None, p, (64,))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, _ = bea.rope_axes(q, None, p, (64,))
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


def test_python_refusals():
    import blockwise_exact_attention_gb300 as bea
    q = draw((1, 2, 2, 64), BF16, 24)
    p = torch.zeros((1, 1, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        bea.rope_axes(q, None, p[0], (32,))
    with pytest.raises(ValueError):
        bea.rope_axes(q, q.cpu(), p, (32,))
    with pytest.raises(TypeError):
        bea.rope_axes(q.half(), None, p, (32,))
    with pytest.raises(RuntimeError, match="DTYPE"):
        bea.rope_axes(q, q.float(), p, (32,))
    with pytest.raises(RuntimeError, match="DTYPE"):
        bea.rope_axes(q, None, p.float(), (32,))
    with pytest.raises(RuntimeError, match="ARG"):
        bea.rope_axes(q, None, p, (32,), q_out=torch.empty_like(q[:, :1]).expand_as(q))
    with pytest.raises(RuntimeError, match="ARG"):
        bea.rope_axes(q, None, p, (32,), k_out=q)
    assert bea.device_status() == 0
