"""Rotary and paged calls directly behind the attention's kernels on one stream:
they read, and write over, what the kernel before them leaves, without a
synchronisation between, and give what a synchronised run gives."""

import pytest

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
    return torch.randn(shape, device="cuda", generator=g).to(dtype)


@pytest.mark.parametrize("n,l,h,d", [(1, 256, 1, 128), (2, 1000, 4, 64), (1, 4096, 16, 128)])
def test_behind_a_forward(n, l, h, d):
    import blockwise_exact_attention_gb300 as bea
    q, k, v = (draw((n, l, h, d), BF16, s) for s in (1, 2, 3))
    pos = torch.arange(l, dtype=I32, device="cuda").expand(1, n, l)
    slots = torch.randperm(n * l, device="cuda").to(I32)
    out, lse = bea.flash_mha_fwd(q, k, v, 0.1, True)
    torch.cuda.synchronize()
    want = bea.rope_axes(out, None, pos, (d // 2,))[0]
    torch.cuda.synchronize()
    cache = torch.zeros((n * l, 1, h, d), dtype=BF16, device="cuda")
    want_cache = torch.zeros_like(cache)
    bea.paged_write(out, out, slots, want_cache, torch.zeros_like(cache))
    for _ in range(20):
        got, got_lse = torch.full_like(out, 7), torch.full_like(lse, 7)
        kc, vc = torch.zeros_like(cache), torch.zeros_like(cache)
        torch.cuda.synchronize()
        bea.flash_mha_fwd(q, k, v, 0.1, True, out=got, lse=got_lse)
        turned, _ = bea.rope_axes(got, None, pos, (d // 2,))
        bea.flash_mha_fwd(q, k, v, 0.1, True, out=got, lse=got_lse)
        bea.paged_write(got, got, slots, kc, vc)
        torch.cuda.synchronize()
        assert torch.equal(turned, want) and torch.equal(kc, want_cache) and torch.equal(vc, want_cache)
        bea.flash_mha_fwd(q, k, v, 0.1, True, out=got)
        bea.rope_axes(q, None, pos, (d // 2,), q_out=got, inverse=True)      # written over at once
        torch.cuda.synchronize()
        assert torch.equal(got, bea.rope_axes(q, None, pos, (d // 2,), inverse=True)[0])


@pytest.mark.parametrize("n,l,h,d", [(1, 256, 2, 128), (1, 2048, 8, 64)])
def test_behind_a_staged_backward(n, l, h, d):
    """The gradients that a K/V block's backward adds to, turned back at once."""
    import blockwise_exact_attention_gb300 as bea
    q, k, v, do = (draw((n, l, h, d), BF16, s) for s in (4, 5, 6, 7))
    pos = torch.arange(l, dtype=I32, device="cuda").expand(1, n, l)
    out, lse = bea.flash_mha_fwd(q, k, v, 0.1, True)
    ws = torch.empty(bea.bwd_workspace_bytes(q), dtype=torch.uint8, device="cuda")
    base = [draw((n, l, h, d), F32, s) for s in (8, 9)]

    def block(sync):
        dk, dv = (b.clone() for b in base)
        bea.flash_mha_bwd_prepare(do, out, lse, ws)
        if sync:
            torch.cuda.synchronize()
        bea.flash_mha_bwd_kv_block(do, q, k, v, dk, dv, workspace=ws, softmax_scale=0.1, is_causal=True, accumulate=True)
        if sync:
            torch.cuda.synchronize()
        return bea.rope_axes(dk, dv, pos, (d // 2,), inverse=True)

    want = block(True)
    for _ in range(20):
        got = block(False)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
