"""The operators together: a batch of requests served from a paged cache, token
by token, against the framework's own attention over each request's whole
sequence."""

import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


@pytest.mark.parametrize("h,h_kv,d,page,left", [(8, 2, 128, 16, -1), (4, 4, 64, 20, 40)])
def test_serving(h, h_kv, d, page, left):
    """Prompts are planned, rotated and written in one ragged step, then every
    request adds a token a step; request 1 ends half way and its row starts over.
    The last token's attention out of the cache is what flash_mha_fwd gives for
    the request's whole sequence: both accumulate in fp32 and differ by the bf16
    rounding of P in the latter (2^-8 of A <= max |v|) and of both outputs."""
    import blockwise_exact_attention_gb300 as bea
    torch.manual_seed(0)
    rows, sections, scale = 4, (d // 8, d // 8, d // 4), 1.0 / math.sqrt(d)
    cache = bea.PagedKVCache(200, page, h_kv, d, rows, 400)
    seqs = [[] for _ in range(rows)]                     # (k, v) of every token, turned

    def step(new, capacity):
        plan = cache.plan(i32(new), capacity)
        q = torch.randn(1, capacity, h, d, device="cuda").to(BF16)
        k = torch.randn(1, capacity, h_kv, d, device="cuda").to(BF16)
        v = torch.randn(1, capacity, h_kv, d, device="cuda").to(BF16)
        pos = torch.stack([plan.positions, plan.positions // 7, plan.positions % 7])[:, None]
        q, k = bea.rope_axes(q, k, pos, sections)
        cache.write(k, v, plan.slot_map)
        at = 0
        for r, a in enumerate(new):
            if a < 0:
                seqs[r] = []
            for _ in range(max(a, 0)):
                seqs[r].append((k[0, at], v[0, at], q[0, at]))
                at += 1
        assert plan.cu_new.tolist()[-1] == at and cache.lens.tolist() == [len(s) for s in seqs]
        last = torch.zeros(rows, 1, h, d, dtype=BF16, device="cuda")
        for r, s in enumerate(seqs):
            if s:
                last[r, 0] = s[-1][2]
        out, lse = cache.decode(last, scale, left)
        for r, s in enumerate(seqs):
            if not s:
                assert not out[r].any() and torch.isneginf(lse[r]).all()
                continue
            ks, vs = (torch.stack([t[i] for t in s])[None] for i in (0, 1))
            ref, ref_lse = bea.flash_mha_fwd(last[r:r + 1], ks, vs, scale, True, (left, 0), out_dtype=torch.float32)
            assert (lse[r] - ref_lse[0]).abs().max() <= 1e-5
            bound = 2 ** -8 * vs.float().abs().max() + 2 ** -8 * ref.abs() + 1e-6
            assert ((out[r].float() - ref[0]).abs() <= bound).all()

    step([50, 7, 0, 1], 64)
    for t in range(20):
        new = [1, 1, int(t > 3), 1]
        if t == 10:
            new[1] = -1
        step(new, 8)
    step([100, 3, -1, 40], 150)
    step([1, 1, 30, 1], 33)
    assert bea.device_status() == 0


def test_serving_step_as_a_graph():
    """Plan, rotation, write and attention of a decode step captured once and
    replayed: the state on the GPU goes on from replay to replay."""
    import blockwise_exact_attention_gb300 as bea
    torch.manual_seed(1)
    rows, h, h_kv, d, page = 3, 4, 2, 64, 16
    caches = [bea.PagedKVCache(64, page, h_kv, d, rows, 300) for _ in range(2)]
    q, k, v = (torch.zeros(rows, 1, x, d, dtype=BF16, device="cuda") for x in (h, h_kv, h_kv))
    new = i32([0, 0, 0])

    def step(cache):
        plan = cache.plan(new, rows)
        # the tokens of the step in row order: each row adds one
        qr, kr = bea.rope_axes(q, k, plan.positions.view(1, rows, 1), (d // 2,))
        cache.write(kr, v, plan.slot_map)
        return cache.decode(qr, 0.125)

    step(caches[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step(caches[0])
    new.copy_(i32([1, 1, 1]))
    for t in range(40):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda"))
        graph.replay()
        ref, ref_lse = step(caches[1])
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    assert caches[0].lens.tolist() == [40, 40, 40] == caches[1].lens.tolist()
    assert bea.device_status() == 0


def test_train_through_rotation_and_attention():
    """q and k turned, then attention, gradients to the unturned q, k and v: equal
    to the attention's gradients turned back by hand."""
    import blockwise_exact_attention_gb300 as bea
    torch.manual_seed(2)
    n, l, h, h_kv, d, sections = 1, 200, 4, 2, 64, (8, 12, 12)
    q, k, v = (torch.randn(n, l, x, d, device="cuda").to(BF16).requires_grad_() for x in (h, h_kv, h_kv))
    g = torch.randn(n, l, h, d, device="cuda").to(BF16)
    pos = torch.randint(0, 50, (3, n, l), device="cuda").to(I32)
    out = bea.flash_attention(*bea.rotary_axes(q, k, pos, sections), v, is_causal=True)
    out.backward(g)
    qr, kr = bea.rope_axes(q.detach(), k.detach(), pos, sections)
    o, lse = bea.flash_mha_fwd(qr, kr, v.detach(), None, True)
    dq, dk, dv = bea.flash_mha_bwd(g, qr, kr, v.detach(), o, lse, None, True)
    dq, dk = bea.rope_axes(dq, dk, pos, sections, inverse=True)
    assert torch.equal(k.grad, dk) and torch.equal(v.grad, dv)
    assert (q.grad.float() - dq.float()).abs().max() <= 1e-2     # the backward sums dQ in any order
    assert bea.device_status() == 0


def test_inputs_from_another_stream():
    """Keys, lengths and tables that a slow kernel on another stream writes last, read right after an event, behind an
    early-launched call on this stream; and results read by another stream behind an event."""
    import blockwise_exact_attention_gb300 as bea
    torch.manual_seed(3)
    n, h, h_kv, d, page = 3, 4, 2, 64, 16
    k, v = torch.randn(2, 200, page, h_kv, d, device="cuda").to(BF16)
    q = torch.randn(n, 1, h, d, device="cuda").to(BF16)
    table = torch.arange(198, dtype=I32, device="cuda").view(n, 66)
    big = torch.randn(3000, 3000, device="cuda")
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    small = torch.zeros(1, 1, 2, 64, dtype=BF16, device="cuda")
    pos = torch.zeros(1, 1, 1, dtype=I32, device="cuda")
    for t in range(20):
        want_lens = i32([1000 - t, 3 + t, 0 if t % 2 else 500])
        want_k = k * (1.0 + 0.125 * (t % 4))
        want = bea.paged_decode(q, want_k, v, table, want_lens, 0.1)
        lens, kk = torch.zeros_like(want_lens), torch.zeros_like(k)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(3):
                big = big @ big * 1e-3
            kk.copy_(want_k + 0 * big.sum().nan_to_num(0, 0, 0).to(BF16))
            lens.copy_(want_lens)
            ready = side.record_event()
        bea.rope_axes(small, None, pos, (32,))
        here.wait_event(ready)
        got = bea.paged_decode(q, kk, v, table, lens, 0.1)
        done = here.record_event()
        with torch.cuda.stream(side):
            side.wait_event(done)
            copies = [x.clone() for x in got]
        torch.cuda.synchronize()
        for a, b in zip(copies, want):
            assert torch.equal(a, b), t
