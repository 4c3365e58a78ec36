"""The softmax weights of shared keys in paged_decode_shared, and their sums.

One weight: of the shared keys the first has score 0 and value 0, the last score -x and value 1, x another one for
each request, and all others weight 0. So the output is w = p / (1 + p), p = exp(-x), and what is lost of one weight
shows in full. u = 2^-23. The weight enters the matrix product as two bf16 terms: the first is cut off to 8 bits, the
rest, below 2^-7 of p, is rounded to 8 bits: off by 2^-15 of p at most; the last bit that is set adds u. The exponent's
two roundings are u x in p at most, the exponential 2 u, the sum 1 + p, its bits that are set, its reciprocal, the last
product and joining the parts a few u more:
  |out - w| <= w (2^-15 + u (x + 20)).
A bf16 output is that rounded once more, half a step of it, 2^-8."""

import math

import numpy as np
import pytest

from test_gpu_paged_shared import BF16, F32, i32, make, run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


@pytest.mark.parametrize("apart", [100, 3000])
@pytest.mark.parametrize("n,h,d", [(9, 3, 64), (200, 1, 128), (70, 8, 128)])
def test_one_weight(n, h, d, apart):
    g = torch.Generator(device="cuda")
    g.manual_seed(n + d)
    x = (4 * torch.rand((n, h), device="cuda", generator=g)).to(BF16)
    page, length = 128, -(-(apart + 2) // 128) * 128
    k = torch.zeros((length // page + 1, page, 1, d), dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    k[..., 1] = -2.0 ** 30                              # weight 0
    flat = k.view(-1, d)
    flat[0, 1] = flat[apart + 1, 1] = 0
    flat[apart + 1, 0] = -1
    v.view(-1, d)[apart + 1] = 1
    q = torch.zeros((n, 1, h, d), dtype=BF16, device="cuda")
    q[:, 0, :, 0], q[..., 1] = x, 1
    width = 97_000_000 // (d * 4 * page * (n - 1)) + length // page + 2
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    table[:, :length // page + 1] = torch.arange(length // page + 1, device="cuda")
    args = (q, k, v, table, i32([length + 1] * n)), (i32([0, n]), i32([length]))
    x = x.double().cpu().numpy()[:, None, :, None]
    w = np.exp(-x) / (1 + np.exp(-x))
    tol = w * (2.0 ** -15 + U * (x + 20))
    out32, lse = run(*args, 1.0, out_dtype=F32)
    err = np.abs(out32.double().cpu().numpy() - w)
    assert (err <= tol).all(), (err / tol).max()
    out, lse16 = run(*args, 1.0)
    err = np.abs(out.double().cpu().numpy() - w)
    assert (err <= tol + 2.0 ** -8 * (w + tol)).all(), (err / w).max()
    assert torch.equal(out, out32.to(BF16)) and torch.equal(lse16, lse)


@pytest.mark.parametrize("h,h_kv,d", [(8, 2, 64), (7, 1, 128), (40, 2, 128)])
def test_a_bf16_output_is_the_rounded_f32_one(h, h_kv, d):
    """Up to eight tiles of a run, that is; behind them the two are summed in other pieces."""
    x, g = make([(700, [1, 0, 17, None, 300, 31, 2]), (256, [4] * 40)], h, h_kv, d, 16, seed=h + d, qscale=4.0)
    out, lse = run(x, g, 0.1)
    out32, lse32 = run(x, g, 0.1, out_dtype=F32)
    assert torch.equal(out, out32.to(BF16)) and torch.equal(lse, lse32)


@pytest.mark.parametrize("n,h,h_kv,d,keys", [(256, 64, 2, 128, 65536), (256, 64, 2, 64, 65536), (64, 32, 8, 128, 16384)])
def test_long_sums(n, h, h_kv, d, keys):
    """Values of 1, whose output is 1, in units that a CTA follows over up to 216 tiles. 16 tiles of 2 * 8 products are
    added up by the tensor core, which may cut off a unit of 2^-23 of its sum in each: of a sum that grows evenly half
    of 256 units, 2^-16. What the weights lose is as often up as down, of 16384 keys and more together 6 * 2^-15 / sqrt(3) *
    1.2 / 128 at most (six standard deviations; scores of a standard deviation of 0.6), below 2^-19; so are the sums of
    weights, up to 216 roundings to nearest, and the parts' pieces and merges."""
    import blockwise_exact_attention_gb300 as bea
    g = torch.Generator(device="cuda")
    g.manual_seed(h + d)
    page = 128
    k = torch.randn((keys // page, page, h_kv, d), device="cuda", generator=g).to(BF16)
    q = (0.57 / (0.1 * math.sqrt(d)) * torch.randn((n, 1, h, d), device="cuda", generator=g)).to(BF16)
    table = torch.arange(keys // page, dtype=torch.int32, device="cuda").repeat(n, 1)
    x = (q, k, torch.ones_like(k), table, i32([keys] * n))
    out, lse = run(x, (i32([0, n]), i32([keys])), 0.1, out_dtype=F32)
    assert (out.double() - 1).abs().max() <= 2.0 ** -16 + 3 * 2.0 ** -19
    # lse, about 11: its sum as above, itself rounded three times
    want = bea.paged_decode(*(t[:2] if t.shape[0] == n else t for t in x), 0.1, out_dtype=F32)
    assert (lse[:2] - want[1]).abs().max() <= 2.0 ** -18
    out16, lse16 = run(x, (i32([0, n]), i32([keys])), 0.1)
    assert (out16 == 1).all() and torch.equal(lse16, lse)


@pytest.mark.parametrize("falls", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_long_runs_whose_maximum_grows(d, falls):
    """Scores that climb (or fall) by 60 along 16384 keys which a CTA follows over some 54 tiles, so that what has been
    summed is rescaled again and again. A score is within (d + 2) u S in either call, twice of it in a weight and in their sum,
    and 2^-14 of A = sum p |v| is the products'; the log-sum-exps (below 64) differ by the scores' error and what four
    roundings of 2^-18 leave."""
    import blockwise_exact_attention_gb300 as bea
    n, h, keys, page = 256, 64, 16384, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    k = (0.1 * torch.randn((keys, 1, d), device="cuda", generator=g)).to(BF16)
    ramp = torch.arange(keys, device="cuda") * (60 / keys)
    k[:, 0, 0] = ramp.flip(0) if falls else ramp
    k = k.view(keys // page, page, 1, d)
    v = (1 + torch.randn(k.shape, device="cuda", generator=g)).to(BF16)
    q = torch.randn((n, 1, h, d), device="cuda", generator=g).to(BF16)
    q[..., 0] = 1
    table = torch.arange(keys // page, dtype=torch.int32, device="cuda").repeat(n, 1)
    lens = i32([keys] * n)
    out, lse = run((q, k, v, table, lens), (i32([0, n]), i32([keys])), 1.0, out_dtype=F32)
    some = [0, 1, 100, 255]
    few = (q[some], k, v, table[some], lens[some])
    want, want_lse = bea.paged_decode(*few, 1.0, out_dtype=F32)
    size, _ = bea.paged_decode(few[0], k, v.abs(), *few[3:], 1.0, out_dtype=F32)
    s = 60 + 0.1 * d * 4                                  # no score's sum of sizes is above it
    e = 2 * (d + 2) * U * s
    assert ((out[some] - want).abs() <= (2 * e + 2.0 ** -14) * size).all()
    assert (lse[some] - want_lse).abs().max() <= e + 2.0 ** -16
    out16, _ = run((q, k, v, table, lens), (i32([0, n]), i32([keys])), 1.0)
    assert ((out16[some] - want).abs() <= (2 * e + 2.0 ** -13) * size + 2.0 ** -8 * (want.abs() + 2.0 ** -8 * size)).all()
    assert bea.device_status() == 0
