"""Failure paths of the paged 4-bit cache: waits that run out, offsets that share
rows, workspaces of graphs, two appends at once."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    from bit_kv_cache_11_gb300 import kvq as k
    return k


@pytest.fixture
def limit(kvq):
    yield kvq.kvq_debug_set_paged_wait_limit
    kvq.kvq_debug_set_paged_wait_limit(-1)


def ints(x):
    return torch.from_numpy(np.asarray(x).astype(np.int32)).cuda()


def pool_of(n_pages, H, ps, D, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = [torch.randint(0, 256, (n_pages, H, ps, D // 2), dtype=torch.uint8, device="cuda", generator=g) for _ in "kv"]
    meta = [torch.rand(n_pages, H, ps, D // 32, 2, device="cuda", generator=g) * 0.3 for _ in "kv"]
    for m in meta:
        m[..., 1] -= 2.0
    return codes + [m.half() for m in meta]


def call_of(seq, new, H=2, R=4, D=64, ps=16, dtype=torch.float16):
    need = [-(-x // ps) for x in seq]
    table = np.full((len(seq), max(need)), -1)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = np.arange(at, at + n)
        at += n
    q = torch.randn(sum(new), H * R, D, device="cuda").to(dtype)
    return [q, *pool_of(at, H, ps, D), ints(table), ints(np.concatenate([[0], np.cumsum(new)])), ints(seq)]


DECODE = [((20000,), (1,)), ((5000, 3000, 17, 800), (1, 1, 1, 1)), (tuple(range(100, 4000, 60)), (2,) * 65)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("seq,new", DECODE, ids=["one", "four", "many"])
def test_a_decode_wait_that_runs_out(kvq, limit, seq, new, D):
    """It is flagged, the tickets of the shared items return to zero, and the next
    call with the same workspace is right."""
    a = call_of(seq, new, D=D)
    most = max(new)
    want = kvq.kvq_paged4_attention(*a, max_new=most)
    ws = torch.zeros(kvq.kvq_paged4_workspace_bytes(a[1].shape[0], 2, 16, D), dtype=torch.uint8, device="cuda")
    for rounds in (0, 1, 0, 2, 1, 3, 0):
        err = ints([0])
        limit(rounds)
        for kw in (dict(workspace=ws), dict()):
            kvq.kvq_paged4_attention(*a, max_new=most, error=err, **kw)
        limit(-1)
        assert err.item() == kvq.KVQ_PAGED_ERR_WAIT or (rounds > 0 and err.item() == 0)
        assert (ws[:1024] == 0).all()
        err.zero_()
        for kw in (dict(workspace=ws), dict()):
            assert torch.equal(kvq.kvq_paged4_attention(*a, max_new=most, error=err, **kw), want)
        assert err.item() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_prompt_wait_that_runs_out(kvq, limit, dtype, D):
    a = call_of((900, 300, 40) + (1,) * 140, (200, 70, 5) + (0,) * 140, D=D, dtype=dtype)
    want = kvq.kvq_paged4_attention(*a, max_new=200)
    for rounds in (0, 1, 0, 2, 1, 3, 8, 0):
        err = ints([0])
        limit(rounds)
        kvq.kvq_paged4_attention(*a, max_new=200, error=err)
        limit(-1)
        assert err.item() == kvq.KVQ_PAGED_ERR_WAIT or (rounds > 0 and err.item() == 0)
        err.zero_()
        assert torch.equal(kvq.kvq_paged4_attention(*a, max_new=200, error=err), want)
        assert err.item() == 0


def test_requests_that_share_rows_pass_no_bound(kvq):
    """Parts of the work that together pass 31 bits are flagged and skipped."""
    n, batch, ps, D = 532, 8, 128, 128
    width = 1_280_000_000 // ps
    pool = pool_of(4, 1, ps, D)
    table = torch.zeros(batch, width, dtype=torch.int32, device="cuda")
    q = torch.ones(n, 1, D, dtype=torch.float16, device="cuda")
    out, err = torch.full_like(q, 5.0), ints([0])
    kvq.kvq_paged4_attention(q, *pool, table, ints([0, n] * 4 + [0]), ints([width * ps] * batch), max_new=n, out=out,
                             error=err)
    assert err.item() == kvq.KVQ_PAGED_ERR_LENGTH
    assert (out == 5.0).all()


def test_both_kinds_of_pages_share_a_streams_workspace(kvq):
    """Calls over E4M3 and over 4-bit pages one after the other on one stream."""
    a = call_of((5000, 3000), (1, 1), D=128)
    p8 = [torch.randn(502, 2, 16, 128, device="cuda").to(torch.float8_e4m3fn) for _ in "kv"]
    b = [a[0], *p8, *(torch.ones(502, 2, device="cuda") for _ in "kv"), *a[5:]]
    want = kvq.kvq_paged4_attention(*a), kvq.kvq_paged_attention(*b)
    for _ in range(30):
        got = kvq.kvq_paged4_attention(*a), kvq.kvq_paged_attention(*b)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = kvq.kvq_paged4_attention(*a), kvq.kvq_paged_attention(*b), kvq.kvq_paged4_attention(*a)
    for _ in range(10):
        for o in out:
            o.fill_(3.0)
        g.replay()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]) and torch.equal(out[2], want[0])


@pytest.mark.parametrize("cls", ["PagedCache", "PagedCache4"])
def test_two_appends_at_once(kvq, cls):
    """Appends of different requests on two streams into one cache, queries in
    their own place."""
    H, D, ps, T = 4, 128, 32, 96
    one, two = (getattr(kvq, cls)(n_pages=16, page_size=ps, n_q_heads=8, n_kv_heads=H, head_dim=D) for _ in "ab")
    turns = kvq.kvq_rotary_turns(D)
    parts = []
    for i in range(2):
        k, v = (torch.randn(T, H, D, device="cuda").half() for _ in "kv")
        q = torch.randn(T, 8, D, device="cuda").half()
        ang = kvq.kvq_rotary_angles(ints(np.arange(T) + 1000 * i), turns)
        parts.append((k, v, ints(np.arange(T) + 8 * ps * i), ang, q))
    want = [one.append(*p[:4], q=p[4]) for p in parts]
    streams = [torch.cuda.Stream() for _ in "ab"]
    torch.cuda.synchronize()
    for p, s in zip(parts, streams):
        assert two.append(*p[:4], q=p[4], q_out=p[4], stream=s) is p[4]
    torch.cuda.synchronize()
    for p, w in zip(parts, want):
        assert torch.equal(p[4], w)
    for a, b in zip(one._pool(), two._pool()):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    two.check()


@pytest.mark.parametrize("cls", ["PagedCache", "PagedCache4"])
def test_many_tokens_at_once(kvq, cls):
    """A step of 70001 tokens, queries in the same call, against turning and storing."""
    H, D, ps, T = 2, 64, 64, 70001
    one, two = (getattr(kvq, cls)(n_pages=1100, page_size=ps, n_q_heads=6, n_kv_heads=H, head_dim=D) for _ in "ab")
    k, v = (torch.randn(T, H, D, device="cuda").bfloat16() for _ in "kv")
    q = torch.randn(T, 6, D, device="cuda").bfloat16()
    ids = torch.randperm(1100, device="cuda")
    t = torch.arange(T, device="cuda")
    slots = (ids[t // ps] * ps + t % ps).int()
    for rot, inter in ((64, False), (32, True), (20, False)):
        ang = kvq.kvq_rotary_angles(t.int(), kvq.kvq_rotary_turns(rot))
        got = one.append(k, v, slots, ang, interleaved=inter, q=q)
        two.store(kvq.kvq_rotate(k, ang, inter), v, slots)
        assert torch.equal(got, kvq.kvq_rotate(q, ang, inter))
        for a, b in zip(one._pool(), two._pool()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    one.check()
