"""paged_decode_shared directly behind kernels that still write what it reads.

Its prefix kernel starts without a wait of its own, on the ground that the kernel
before it lets it in only after its own wait. Here queries, caches, table, lengths and
groups are each written by a long kernel right before the call, and written over right
behind it, on one stream without a synchronisation; the results are those of calls
that were waited for."""

import pytest

from test_gpu_paged_shared import BF16, F32, i32, make, run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def long_work(x):
    """Some 100 us on all SMs, on this stream."""
    for _ in range(3):
        x = torch.mm(x, x)
    return x


# (one launch of the rest; more requests and more heads to a K/V head than one takes; few rows)
CASES = [((2000, [50, 60, 700, 80, 20, 0, 9, 3000]), 32, 8, 128), ((300, [i % 5 for i in range(1100)]), 2, 1, 64),
         ((700, [5, 300, 7]), 300, 1, 64), ((5000, [1, 40, 90, 17] * 40), 16, 4, 128)]


@pytest.mark.parametrize("group,h,h_kv,d", CASES)
def test_behind_and_before_other_writers(group, h, h_kv, d):
    import blockwise_exact_attention_gb300 as bea
    x, g = make([group], h, h_kv, d, 16, seed=h + d)
    x[1].nan_to_num_(0.5), x[2].nan_to_num_(0.5, posinf=0.5)
    y, _ = make([group], h, h_kv, d, 16, seed=h + d + 100)
    y[1].nan_to_num_(0.25), y[2].nan_to_num_(0.25, posinf=0.25)
    others = (*y, i32([0, 0]), i32([0]))                  # other values, tables and lengths; nothing shared
    wanted = (*x, *g)
    want = run(x, g, 0.1, out_dtype=F32)
    args = [t.clone() for t in others]
    ws = torch.empty(bea.paged_decode_shared_workspace_bytes(x[0], x[1], x[3], g[1]), dtype=torch.uint8, device="cuda")
    work = torch.zeros(4096, 4096, dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    for turn in range(10):
        long_work(work)
        for i in (range(7), reversed(range(7)))[turn % 2]:  # the last one written is the queries, or the groups
            args[i].copy_(wanted[i])
        got = run(args[:5], args[5:], 0.1, out_dtype=F32, workspace=ws)
        for a, o in zip(args, others):
            a.copy_(o)
        ws.fill_(255)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_behind_the_calls_of_a_step():
    """Queries from the normed rotation, keys and values from the write, rows from a fork, all in one stream's order."""
    import blockwise_exact_attention_gb300 as bea
    n, h, h_kv, d, page, prompt = 24, 16, 4, 128, 16, 4000

    def steps(sync):
        done = torch.cuda.synchronize if sync else (lambda: None)
        gen = torch.Generator(device="cuda")
        gen.manual_seed(3)
        cache = bea.PagedKVCache(1200, page, h_kv, d, n, 20000, share_pages=True)
        cache.k.zero_(), cache.v.zero_()
        outs = []
        for new, capacity in [([prompt] + [0] * (n - 1), prompt), (None, 0), ([1] * n, n), ([2] * n, 2 * n), ([1] * n, n)]:
            if new is None:
                cache.fork(i32([-1] + [0] * (n - 1)))
                done()
                continue
            plan = cache.plan(i32(new), capacity)
            q, k, v = (torch.randn(1, capacity, x, d, device="cuda", generator=gen).to(BF16) for x in (h, h_kv, h_kv))
            torch.cuda.synchronize()
            done()
            q, k = bea.norm_rope_axes(q, k, plan.positions.view(1, 1, -1), (64,))
            done()
            cache.write(k, v, plan.slot_map)
            done()
            if len(set(new)) == 1:
                last = q[0, new[0] - 1::new[0]].unsqueeze(1)
                outs.append(cache.decode_shared(last, i32([0, n]), i32([prompt]), out_dtype=F32))
                cache.k[:1].add_(0)                        # behind it, a writer of what it reads
            done()
        torch.cuda.synchronize()
        assert bea.device_status() == 0
        return outs

    want = steps(True)
    for _ in range(5):
        got = steps(False)
        assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))


def test_captured_behind_its_writers():
    """The same order inside a graph, replayed with other inputs."""
    x, g = make([(2000, [50, 60, 700, 80, 20, 0, 9, 3000])], 32, 8, 128, 16, seed=1)
    x[1].nan_to_num_(0.5), x[2].nan_to_num_(0.5, posinf=0.5)
    source = x[0].clone()
    q, work = torch.zeros_like(source), torch.zeros(4096, 4096, dtype=BF16, device="cuda")

    def step():
        long_work(work)
        q.copy_(source)
        return run((q, *x[1:]), g, 0.1, out_dtype=F32)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    for seed in range(5):
        source.copy_((0.5 + seed) * torch.randn(source.shape, device="cuda"))
        q.zero_()
        graph.replay()
        graph.replay()
        want = run((source, *x[1:]), g, 0.1, out_dtype=F32)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
