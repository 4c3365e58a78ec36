"""The softmax weights of paged_decode, as exact as fp32 holds them.

Two keys, the first of score 0 and value 0, the second of score -x and value 1: the output is w = p / (1 + p), p =
exp(-x), so what is lost of one weight shows in full. u = 2^-23. The score is one exact product; its exponent x log2(e)
is rounded twice (the constant and the product, u x in p at most), the exponential adds 2^-22, three terms and their
sum in the matrix product 3 u and 2 * 2^-24 of p, the sum 1 + p, its reciprocal and the last product 2^-24 each, and
where the keys lie in several warps and CTAs each of two merges a product and a sum above and below, 4 * 2^-24:
  |out - w| <= w (2 u + u x + 3 u + u + 1.5 u + 4 u) < w u (x + 12)."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def two_keys(n, h, d, dtype, apart):
    """n requests of two keys `apart` places from one another, which lie before and behind keys of weight 0."""
    g = torch.Generator(device="cuda")
    g.manual_seed(h + d)
    x = (4 * torch.rand(n, device="cuda", generator=g)).to(BF16)
    length = apart + 2
    k = torch.zeros((n, length, 1, d), dtype=dtype, device="cuda")
    v = torch.zeros((n, length, 1, d), dtype=dtype, device="cuda")
    k[:, 1:, 0, 0] = -2.0 ** 30                             # weight 0 between them
    k[:, -1, 0, 0] = -x.to(dtype)
    v[:, -1] = 1
    q = torch.zeros((n, 1, h, d), dtype=dtype, device="cuda")
    q[..., 0] = 1
    table = torch.arange(n, dtype=I32, device="cuda")[:, None]
    return x.double().cpu().numpy(), q, k, v, table, torch.full((n,), length, dtype=I32, device="cuda")


@pytest.mark.parametrize("apart", [0, 40, 3000])
@pytest.mark.parametrize("h,d,dtype", [(1, 64, BF16), (8, 128, BF16), (13, 128, BF16), (16, 64, BF16), (3, 64, F32)])
def test_one_weight(h, d, dtype, apart):
    import blockwise_exact_attention_gb300 as bea
    x, *args = two_keys(200 if apart < 3000 else 20, h, d, dtype, apart)
    out, lse = bea.paged_decode(*args, 1.0, out_dtype=F32)
    w = (np.exp(-x) / (1 + np.exp(-x)))[:, None, None, None]
    err = np.abs(out.double().cpu().numpy() - w)
    tol = w * 2.0 ** -23 * (x[:, None, None, None] + 12)
    assert (err <= tol).all(), (err / tol).max()
    ref = np.log1p(np.exp(-x))[:, None, None]
    # the sum's share of the above, at most (2 + x + 2) u p / (1 + p) < 3 u; log2 of the sum, at most 1, and ln 2 times
    # it, two units in the last place each
    assert np.abs(lse.double().cpu().numpy() - ref).max() <= 2.0 ** -23 * 7


def test_an_infinite_value_keeps_the_sign():
    """Whatever bits a weight has, none of its terms is 0 where an infinite value stands."""
    import blockwise_exact_attention_gb300 as bea
    for h, d in ((2, 64), (9, 128)):
        x, q, k, v, table, lens = two_keys(200, h, d, BF16, 0)
        k[::2, 1, 0, 0] = 0                                 # a weight of one bit
        k[::20, 1, 0, 0] = -60                              # and a small one
        v[:, -1, 0, ::2], v[:, -1, 0, 1::2] = float("inf"), float("-inf")
        for dtype in (F32, BF16):
            out, lse = bea.paged_decode(q, k, v, table, lens, 1.0, out_dtype=dtype)
            assert torch.isposinf(out[..., ::2]).all() and torch.isneginf(out[..., 1::2]).all()
            assert torch.isfinite(lse).all()


def test_many_requests_some_of_them_cut():
    """More requests than a launch takes, long ones in each launch: the launches share a workspace and each has its join."""
    import math
    from oracle import paged as op
    import blockwise_exact_attention_gb300 as bea
    n, page, d, h = 1030, 16, 64, 4
    rng = np.random.default_rng(7)
    lens = [int(x) for x in rng.integers(0, 30, n)]
    for r in (3, 700, 1022, 1023, 1024, 1029):
        lens[r] = 4000 + r
    counts = [-(-x // page) for x in lens]
    width = max(counts)
    perm = rng.permutation(sum(counts) + 2)
    table, at = np.full((n, width), -1, dtype=np.int32), 0
    for r, c in enumerate(counts):
        table[r, :c] = perm[at:at + c]
        at += c
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    k, v = (torch.randn((len(perm), page, 2, d), device="cuda", generator=g).to(BF16) for _ in range(2))
    q = torch.randn((n, 1, h, d), device="cuda", generator=g).to(BF16)
    scale = 1.0 / math.sqrt(d)
    out, lse = bea.paged_decode(q, k, v, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=I32, device="cuda"), scale,
                                out_dtype=F32)
    f64 = [t.double().cpu().numpy() for t in (q, k, v)]
    ref, ref_lse, a, s = op.decode(*f64, table, np.array(lens), scale)
    # scores, exponential, terms; sums over up to 5029 keys, of which a warp of the longest adds a few hundred
    u = 2.0 ** -23
    e = (d + 2) * u * s + 2.0 ** -21
    some = np.array(lens) > 0
    length = np.array(lens)[:, None, None] * u
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= ((2 * e + 2 * length)[:, None] * a + 1e-38)).all()
    le = np.abs(lse.double().cpu().numpy()[some] - ref_lse[some])
    assert (le <= (e + length)[some] + u * np.abs(ref_lse[some])).all()
    assert torch.isneginf(lse[torch.from_numpy(~some).cuda()]).all() and bea.device_status() == 0


@pytest.mark.parametrize("h,d", [(1, 64), (2, 128), (9, 128), (16, 64)])
def test_long_sums_keep_their_last_bits(h, d):
    """18 million keys of value 1 (requests that share their pages for reading), so that each warp of a GPU of 152 SMs
    adds up some 500 tiles. The output is 1; off by what sums of that length lose where each addition rounds to nearest:
    with N additions of equal numbers, the k-th at most 2^-24 k / N of the sum and as often up as down, one standard
    deviation is 2^-24 sqrt(N) / 3. N is 500 above and 2000 in each of four parts below, together 2^-24 * 11; six of
    these are 2^-18. A tile's products, which the tensor core may cut off, add three units of 2^-23 at most, the
    terms of a weight 2^-23, the merges 2^-21."""
    import blockwise_exact_attention_gb300 as bea
    page, pages = 64, 32
    n, width = 560, (512 if d == 64 else 256)
    g = torch.Generator(device="cuda")
    g.manual_seed(h)
    k = torch.zeros((pages, page, 1, d), dtype=BF16, device="cuda")
    k[..., 0] = -torch.rand((pages, page, 1), device="cuda", generator=g).to(BF16)
    v = torch.ones_like(k)
    q = torch.zeros((n, 1, h, d), dtype=BF16, device="cuda")
    q[..., 0] = 1
    table = (torch.arange(width, device="cuda") % pages).to(I32).expand(n, width).contiguous()
    lens = torch.full((n,), width * page, dtype=I32, device="cuda")
    out, lse = bea.paged_decode(q, k, v, table, lens, 1.0, out_dtype=F32)
    assert (out.double() - 1).abs().max() <= 2 ** -18 + 4 * 2 ** -23 + 2 ** -21
    ref = torch.log(torch.exp(k[..., 0].double()).sum() * (width // pages))
    # the same below, the exponentials' 2^-22 and 2^-23 of their exponents; lse itself, up to 11, in fp32
    assert (lse.double() - ref).abs().max() <= 2 ** -18 + 2 ** -21 + 2 ** -21 + 11 * 2 ** -22


def test_long_tables_need_a_workspace_and_short_ones_none():
    import blockwise_exact_attention_gb300 as bea
    q = torch.zeros((1, 1, 8, 128), dtype=BF16, device="cuda")
    cache = torch.zeros((400, 16, 2, 128), dtype=BF16, device="cuda")
    table = torch.arange(400, dtype=I32, device="cuda")[None]
    lens = torch.full((1,), 5000, dtype=I32, device="cuda")
    need = bea.paged_decode_workspace_bytes(q, cache, table)
    assert need > 0 and bea.paged_decode_workspace_bytes(q, cache, table[:, :4]) == 0
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    bea.paged_decode(q, cache, cache, table, lens, 0.1, workspace=ws[:need])
    assert (ws[need:] == 255).all()
    for bad in (ws[:need - 1], ws[16:], ws[:0]):
        with pytest.raises(RuntimeError, match="WORKSPACE"):
            bea.paged_decode(q, cache, cache, table, lens, 0.1, workspace=bad)
    assert bea.device_status() == 0
