"""Failure paths of the paged calls.  Nothing here faults, traps or hangs the GPU:
kvq_debug_set_paged_wait_limit makes the attention's main-loop waits give up early
(the copies in flight are waited for all the same)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_kv_cache_11_gb300 import kvq as k
    return k


def ints(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def call_of(seq, new, H=2, R=4, D=64, ps=16, dtype=torch.float16, seed=0):
    """Arguments of an attention over random pages."""
    rng = np.random.default_rng(seed)
    need = [-(-x // ps) for x in seq]
    pages = [torch.randn(sum(need), H, ps, D, device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
    scale = [torch.ones(sum(need), H, device="cuda") for _ in range(2)]
    table = np.full((len(seq), max(need)), -1)
    ids, at = rng.permutation(sum(need)), 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    q = torch.randn(sum(new), H * R, D, device="cuda").to(dtype)
    return [q, *pages, *scale, ints(table), ints(np.cumsum([0] + list(new))), ints(seq)]


@pytest.fixture
def limit(kvq):
    yield kvq.kvq_debug_set_paged_wait_limit
    kvq.kvq_debug_set_paged_wait_limit(-1)


DECODE = [((20000,), (1,)), ((5000, 3000, 17, 800), (1, 1, 1, 1)), (tuple(range(100, 4000, 60)), (2,) * 65)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("seq,new", DECODE, ids=["one", "four", "many"])
def test_a_decode_wait_that_runs_out(kvq, limit, seq, new, D):
    """It is flagged, the tickets of the shared items return to zero whichever warps
    gave up, and the next call with the same workspace is right."""
    a = call_of(seq, new, D=D)
    most = max(new)
    want = kvq.kvq_paged_attention(*a, max_new=most)
    ws = torch.zeros(kvq.kvq_paged_workspace_bytes(a[1].shape[0], 2, 16, D), dtype=torch.uint8, device="cuda")
    for rounds in (0, 1, 0, 2, 1, 3, 0):
        err = ints([0])
        limit(rounds)
        for kw in (dict(workspace=ws), dict()):  # the caller's workspace, the stream's own
            kvq.kvq_paged_attention(*a, max_new=most, error=err, **kw)
        limit(-1)
        assert err.item() == kvq.KVQ_PAGED_ERR_WAIT or (rounds > 0 and err.item() == 0)
        assert (ws[:1024] == 0).all()
        err.zero_()
        for kw in (dict(workspace=ws), dict()):
            assert torch.equal(kvq.kvq_paged_attention(*a, max_new=most, error=err, **kw), want)
        assert err.item() == 0


def test_the_cache_reports_a_wait_that_ran_out(kvq, limit):
    c = kvq.PagedCache(n_pages=400, page_size=16, n_q_heads=8, n_kv_heads=2, head_dim=64)
    a = call_of((5000,), (1,))
    table = ints(np.arange(313)[None])
    want = c.attention(a[0], table, a[6], a[7])
    limit(0)
    c.attention(a[0], table, a[6], a[7])
    limit(-1)
    with pytest.raises(kvq.KvqError, match="wait"):
        c.check()
    assert torch.equal(c.attention(a[0], table, a[6], a[7]), want)
    c.check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_prompt_wait_that_runs_out(kvq, limit, dtype, D):
    """Every role of the kernel leaves, whichever of them gave up; the next call is
    right.  (140 requests without tokens: a large batch, whose many-row requests the
    prompt kernel serves.)"""
    a = call_of((900, 300, 40) + (1,) * 140, (200, 70, 5) + (0,) * 140, D=D, dtype=dtype)
    want = kvq.kvq_paged_attention(*a, max_new=200)
    for rounds in (0, 1, 0, 2, 1, 3, 8, 0):
        err = ints([0])
        limit(rounds)
        kvq.kvq_paged_attention(*a, max_new=200, error=err)
        limit(-1)
        assert err.item() == kvq.KVQ_PAGED_ERR_WAIT or (rounds > 0 and err.item() == 0)
        err.zero_()
        assert torch.equal(kvq.kvq_paged_attention(*a, max_new=200, error=err), want)
        assert err.item() == 0


def test_requests_that_share_rows_pass_no_bound(kvq):
    """Offsets that decrease make several requests claim the same rows.  Their parts of
    the work together may pass 31 bits (here 4 requests of 34 groups and 4e7 units
    each, 2^32 and more together, over tables that nothing reads): the call is
    flagged and skipped."""
    n, batch, ps, D = 532, 8, 128, 128
    width = 1_280_000_000 // ps
    pages = [torch.zeros(4, 1, ps, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scale = [torch.ones(4, 1, device="cuda") for _ in range(2)]
    table = torch.zeros(batch, width, dtype=torch.int32, device="cuda")
    q = torch.ones(n, 1, D, dtype=torch.float16, device="cuda")
    out, err = torch.full_like(q, 5.0), ints([0])
    kvq.kvq_paged_attention(q, *pages, *scale, table, ints([0, n] * 4 + [0]), ints([width * ps] * batch),
                            max_new=n, out=out, error=err)
    assert err.item() == kvq.KVQ_PAGED_ERR_LENGTH
    assert (out == 5.0).all()


def test_a_graphs_workspace_goes_with_the_graph(kvq):
    """Captured calls leave no memory behind when their graphs are gone (the next call
    frees it), and another capture of the same stream does not take it from a graph
    that is still there."""
    import gc
    import time
    a = call_of((5000, 3000), (1, 1), D=128)
    want = kvq.kvq_paged_attention(*a)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def capture():
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = kvq.kvq_paged_attention(*a)
        return g, out

    def allocated():
        gc.collect()
        kvq.kvq_paged_attention(*a)
        torch.cuda.synchronize()
        return torch.cuda.memory_allocated()

    before = allocated()
    graphs = [capture() for _ in range(3)]
    assert allocated() - before >= 3 * kvq.kvq_paged_workspace_bytes(a[1].shape[0], 2, 16, 128)
    for _ in range(3):
        for g, out in graphs:
            out.zero_()
            g.replay()
            assert torch.equal(out, want)
    del g, out, graphs
    for _ in range(100):  # (a graph is destroyed in its own time)
        after = allocated()
        if after == before:
            break
        time.sleep(0.05)
    assert after == before, (before, after)


def test_a_step_that_the_free_stack_cannot_serve_in_full(kvq):
    """The requests that fit are served, nothing of the others is stored, and their step
    made again with pages gives what it would have given."""
    # another batch is another split: each result is off by at most 2^-11 of the values'
    # size (their weights' rounding) and of itself, and by a few fp32 steps
    def same(x, y):
        x, y = x.float(), y.float()
        return bool(((x - y).abs() <= 2.1 * 2.0 ** -11 * (v.abs().max() + y.abs())).all())
    H, R, D, ps = 2, 2, 64, 16
    torch.manual_seed(7)
    ctx, new = [20, 16, 30, 5], [3, 20, 5, 4]  # fresh pages: 0, 2, 1, 0
    n_pages = 12

    def state(free):
        torch.manual_seed(8)
        c = kvq.PagedCache(n_pages=n_pages, page_size=ps, n_q_heads=H * R, n_kv_heads=H, head_dim=D)
        table, stack, n_free = ints(np.full((4, 6), -1)), ints(range(n_pages)), ints([n_pages])
        z = ints([0] * 4)
        cu, seq, slots, left = c.plan(z, ints(ctx), table, stack, n_free, sum(ctx))
        c.store(*(torch.randn(sum(ctx), H, D, device="cuda").half() for _ in range(2)), slots)
        assert left.item() == n_pages - 6
        return c, table, stack, seq, ints([free])

    torch.manual_seed(9)
    k, v = (torch.randn(sum(new), H, D, device="cuda").half() for _ in range(2))
    q = torch.randn(sum(new), H * R, D, device="cuda").half()
    whole, table, stack, seq0, n_free = state(6)
    cu, seq, slots, _ = whole.plan(seq0, ints(new), table, stack, n_free, sum(new))
    whole.store(k, v, slots)
    want = whole.attention(q, table, cu, seq, max_new=max(new))
    whole.check()

    c, table, stack, seq0, n_free = state(1)  # request 1 needs two pages
    cu, seq, slots, left = c.plan(seq0, ints(new), table, stack, n_free, sum(new))
    assert seq.tolist() == [23, 16, 30, 9] and left.item() == 1
    c.store(k, v, slots)
    out = c.attention(q, table, cu, seq, max_new=max(new))
    with pytest.raises(kvq.KvqError, match="free stack"):
        c.check()
    for a, b in ((0, 3), (28, 32)):  # requests 0 and 3
        assert same(out[a:b], want[a:b])
    again = ints([0, 20, 5, 0])
    cu, seq, slots, left = c.plan(seq, again, table, ints(range(n_pages)), ints([6]), 25)
    assert seq.tolist() == [23, 36, 35, 9] and left.item() == 3
    c.store(k[3:28], v[3:28], slots)
    out = c.attention(q[3:28], table, cu, seq, max_new=20)
    assert same(out, want[3:28])
    c.check()
