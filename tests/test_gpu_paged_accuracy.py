"""The paged attention held to the bound of tests/paged_ref.py's `row`, under
which every 16 tokens of an output count (tests/test_paged_bounds_cpu.py)."""
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import paged_ref as ref  # noqa: E402

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


def e4m3(codes):
    return torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn)


def f32(x):
    return torch.from_numpy(np.asarray(x, np.float32)).cuda()


def check(got, want, bound):
    d = np.abs(got.double().cpu().numpy() - want)
    worst = float((d / bound).max())
    assert worst <= 1.0, worst


@pytest.mark.parametrize("n,kernel", [(1, "decode"), (70, "prompt")])
@pytest.mark.parametrize("D", [64, 128])
def test_one_token_before_many_small_ones(kvq, n, kernel, D):
    """A token whose weight is 2^25 times another's, but whose value is 0: the others
    carry the result together.  (fp16 weights of at most 1 would lose half of it.)"""
    rng = np.random.default_rng(D + n)
    ps, T, log2 = 64, 4096 + n, ref.WEIGHT_LOG2[kernel]
    n_pages = -(-T // ps)
    k = np.zeros((n_pages, 1, ps, D))
    k[..., 0], k[..., 1] = -16.0, -rng.uniform(0.5, 1.5, (n_pages, 1, ps))  # scores -23.8 .. -25.3 in log2
    k[0, 0, 0] = 0.0
    v = rng.uniform(0.5, 1.0, k.shape)
    v[0, 0, 0] = 0.0
    codes = [ref.e4m3_code(k), ref.e4m3_code(v)]
    scale = [np.ones((n_pages, 1))] * 2
    q = np.zeros((n, 1, D))
    q[..., :2] = 1.0
    want, bound = ref.rows(q, *codes, *scale, np.arange(n_pages)[None], [0, n], [T], ps, 1.0, 0, log2, 2.0 ** -11)
    assert (want > 1e-4).all() and (bound < want * 2.0 ** -4).all()
    # 300 requests over the same pages: whole runs of tokens to a warp of the decode
    # kernel; the prompt kernel serves one of them, the others have no new token
    batch = 300
    new = [n] * batch if kernel == "decode" else [0] * 7 + [n] + [0] * 292
    q = np.concatenate([q] * (sum(new) // n))
    got = kvq.kvq_paged_attention(torch.from_numpy(q).half().cuda(), *map(e4m3, codes), *map(f32, scale),
                                  ints(np.tile(np.arange(n_pages), (batch, 1))), ints(np.cumsum([0] + new)),
                                  ints([T] * batch), max_new=n, softmax_scale=1.0)
    for b in range(0, len(q), n):
        check(got[b:b + n], want, bound)


@pytest.mark.parametrize("n,idle", [(1, 0), (70, 140)])
def test_huge_scores(kvq, n, idle):
    """Scores of up to 2^24 in size, where a maximum and the exponents below it are
    rounded apart: the largest takes all, so an output is a value (and a weight over
    the sum of weights, both rounded to 2^-11 at most)."""
    rng = np.random.default_rng(n)
    ps, D, T = 16, 64, 700
    n_pages = -(-T // ps)
    vc = ref.e4m3_code(rng.standard_normal((n_pages, 1, ps, D)))
    table = np.concatenate([np.arange(n_pages)[None], np.full((idle, n_pages), -1)])
    cu, seq = np.array([0] + [n] * (idle + 1)), np.array([T] + [0] * idle)
    for top, others in ((256.0, 224.0), (-224.0, -256.0)):
        for at in (0, 333, T - n):
            k = np.zeros((n_pages, 1, ps, D))
            k[..., 0] = others
            k[at // ps, 0, at % ps, 0] = top
            for e in (12, 16, 17, 18, 19, 20, 22, 24):
                q = torch.zeros(n, 1, D, dtype=torch.float16, device="cuda")
                q[..., 0] = 2.0
                got = kvq.kvq_paged_attention(q, e4m3(ref.e4m3_code(k)), e4m3(vc), f32(np.full((n_pages, 1), 0.5)),
                                              f32(np.ones((n_pages, 1))), ints(table), ints(cu), ints(seq),
                                              max_new=n, softmax_scale=2.0 ** (e - 8))
                want = np.broadcast_to(ref.E4M3[vc[at // ps, 0, at % ps]], (n, 1, D))
                check(got, want, np.abs(want) * (2.0 ** -10 + 2.0 ** -11) + 2.0 ** -25)


@pytest.mark.parametrize("case", ref.SHARES, ids=str)
def test_every_share_counts(kvq, case):
    s = ref.shares_case(case)
    want, bound = ref.shares_want(s)
    err = ints([0])
    got = kvq.kvq_paged_attention(s["q"].cuda(), *map(e4m3, s["stale"]), *map(f32, s["scale"]), ints(s["table"]),
                                  ints(s["cu"]), ints(s["seq"]), max_new=s["max_new"], window=s["window"],
                                  softmax_scale=s["softmax_scale"], error=err)
    assert err.item() == 0
    check(got, want, bound)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,kernel", [(1, "decode"), (70, "prompt")])
def test_a_negative_softmax_scale(kvq, n, kernel, dtype):
    s = ref.shares_case((16, 64, 2, 1, "bf16" if dtype == torch.bfloat16 else "fp16", [300, 9], [n, n], 0, kernel))
    s["softmax_scale"] = -0.2
    want, bound = ref.shares_want(s)
    got = kvq.kvq_paged_attention(s["q"].cuda(), *map(e4m3, s["stale"]), *map(f32, s["scale"]), ints(s["table"]),
                                  ints(s["cu"]), ints(s["seq"]), max_new=s["max_new"], softmax_scale=-0.2)
    check(got, want, bound)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_serving_loop_against_its_own_pages(kvq, dtype):
    """Prompts, decode steps, drafted tokens and a chunk: every output against the
    attention over the codes and scales that the cache holds, and those against the
    exact keys and values (half a step of E4M3, twice where a page's scale grew)."""
    rng = np.random.default_rng(17)
    H, R, D, ps, B = 2, 4, 128, 16, 5
    c = kvq.PagedCache(n_pages=80, page_size=ps, n_q_heads=H * R, n_kv_heads=H, head_dim=D)
    ctx, table = ints([0] * B), ints(np.full((B, 24), -1))
    free, n_free = ints(rng.permutation(80)), ints([80])
    hist = [[np.zeros((0, H, D))] * 2 for _ in range(B)]
    half_step = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    for new in [[40, 3, 0, 17, 70], [1] * 5, [1, 0, 5, 1, 2]] + [[1] * 5] * 6 + [[30, 4, 0, 1, 33]]:
        n = sum(new)
        k, v = (torch.from_numpy(rng.standard_normal((n + 2, H, D))).to(dtype).cuda() for _ in range(2))
        q = torch.from_numpy(rng.standard_normal((n + 2, H * R, D))).to(dtype).cuda()
        cu, seq, slots, left = c.plan(ctx, ints(new), table, free, n_free, n + 2)
        c.store(k, v, slots)
        out = c.attention(q, table, cu, seq, max_new=max(new))
        ctx, n_free = seq, left
        codes = [p.view(torch.uint8).cpu().numpy() for p in (c.k_pages, c.v_pages)]
        scale = [p.double().cpu().numpy() for p in (c.k_scale, c.v_scale)]
        at, tab = np.concatenate([[0], np.cumsum(new)]), table.cpu().numpy()
        want, bound = ref.rows(q[:n].double().cpu().numpy(), *codes, *scale, tab, at, seq.tolist(), ps, D ** -0.5, 0,
                               ref.WEIGHT_LOG2["prompt"], half_step)
        check(out[:n], want, bound)
        for b in range(B):
            for i, x in enumerate((k, v)):
                hist[b][i] = np.concatenate([hist[b][i], x[at[b]:at[b + 1]].double().cpu().numpy()])
                t = np.arange(len(hist[b][i]))
                pg = tab[b][t // ps]
                held = ref.E4M3[codes[i][pg, :, t % ps]] * scale[i][pg][..., None]
                # 2^-4 of a value, or half a step of E4M3's subnormals, 2^-10 of the scale
                assert (np.abs(held - hist[b][i]) <= 2 * np.maximum(2.0 ** -4 * np.abs(hist[b][i]),
                                                                    2.0 ** -10 * scale[i][pg][..., None])).all()
    c.check()
