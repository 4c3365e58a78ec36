"""What is no number in paged_decode_shared: the same entries as in paged_decode,
wherever the parts of a row are cut. A part whose scores are all NaN has no maximum,
but it has keys, and what it holds belongs to the result."""

import math

import pytest

from test_gpu_paged_shared import BF16, F32, make, run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def same_pattern(x, g, dtype):
    """NaN, infinities and numbers of both outputs lie where paged_decode has them."""
    import blockwise_exact_attention_gb300 as bea
    got, want = run(x, g, 0.1, out_dtype=dtype), bea.paged_decode(*x, 0.1, out_dtype=dtype)
    assert bea.device_status() == 0
    for a, b in zip(got, want):
        for test in (torch.isnan, torch.isposinf, torch.isneginf):
            assert torch.equal(test(a), test(b)), (test.__name__, (test(a) != test(b)).nonzero()[:5].tolist())
    return got


# (rows of a block of four warps each, of one warp, of one warp with fewer parts at a time: 152 SMs times 8 and 32 rows)
SIZES = [(4, 8, 2), (60, 32, 4), (200, 32, 4)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,h,h_kv", SIZES)
def test_an_undefined_query(n, h, h_kv, dtype):
    """Of rows without own keys, with a few, and with so many that they are cut between CTAs."""
    own = [0, 5, 3000, 700] + [i % 7 for i in range(4, n)]
    x, g = make([(5 * 128, own)], h, h_kv, 128, 16, seed=n)
    q, clean = x[0], x[0].clone()
    for r in range(4):
        q.copy_(clean)
        q[r, 0, r % h, 3] = math.nan
        out, lse = same_pattern(x, g, dtype)
        assert out[r, 0, r % h].isnan().all() and lse[r, r % h].isnan().all()
        assert int(lse.isnan().sum()) == 1
    q[:, :, 0] = math.nan
    out, lse = same_pattern(x, g, dtype)
    assert torch.equal(lse[..., 0].isnan(), q[:, 0].isnan().any(-1)) and int(lse.isnan().sum()) == n + 1  # row 3's still


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,h,h_kv", SIZES)
def test_undefined_keys_of_whole_tiles(n, h, h_kv, dtype):
    """Tiles of a prefix that is cut over many CTAs, the first, the last and one inside, and all of them."""
    tiles, page = 150, 16
    x, g = make([(tiles * 128, [i % 5 for i in range(n)])], h, h_kv, 64, page, seed=n + 1)
    k, table = x[1], x[3]
    per = 128 // page
    group = h // h_kv
    for which in ([0], [tiles - 1], [77], list(range(tiles))):
        keep = k.clone()
        for t in which:
            k[table[0, t * per:(t + 1) * per].long(), :, 1] = math.nan
        out, lse = same_pattern(x, g, dtype)
        assert lse[:, group:2 * group].isnan().all() and lse[:, :group].isfinite().all()
        assert out[:, 0, group:2 * group].isnan().all() and out[:, 0, :group].isfinite().all()
        k.copy_(keep)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_undefined_own_keys(dtype):
    """All of one request's own keys, where these are one tile and where they are cut between CTAs."""
    own = [3, 6000, 9, 0]
    x, g = make([(512, own)], 8, 2, 128, 16, seed=3)
    k, table, lens = x[1], x[3], x[4]
    for r in (0, 1):
        keep = k.clone()
        pages = -(-int(lens[r]) // 16)
        k[table[r, 32:pages].long(), :, 0] = math.nan
        out, lse = same_pattern(x, g, dtype)
        assert lse[r, :4].isnan().all() and int(lse.isnan().sum()) == 4
        k.copy_(keep)


def test_undefined_values_and_all_scores_minus_infinity():
    """What is no number among the values spreads to its column, whatever the weights."""
    x, g = make([(1024, [5, 3000, 0])], 4, 2, 64, 16, seed=4)
    q, k, v, table, lens = x
    v[int(table[0, 40]), 3, 1, 9] = math.nan
    out, lse = same_pattern(x, g, BF16)
    assert out[:, 0, 2:, 9].isnan().all() and int(out.isnan().sum()) == 3 * 2 and lse.isfinite().all()
    v[int(table[0, 40]), 3, 1, 9] = 0
    k[:, :, 1], q[:, :, 2:] = -math.inf, 1.0
    for dtype in (BF16, F32):
        out, lse = same_pattern(x, g, dtype)
        assert (lse[:, 2:] == -math.inf).all()
