"""The attention over 4-bit pages held to the bound of tests/paged_ref.py's `row` at
each kernel's own weights, under which every 16 tokens of an output count
(tests/test_paged4_bounds_cpu.py)."""
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import paged4_ref  # noqa: E402
import paged4_shares as shares  # noqa: E402
import paged_ref  # noqa: E402

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


def gpu(pool):
    return [torch.from_numpy(p).cuda() for p in pool]


def check(got, want, bound):
    d = np.abs(got.double().cpu().numpy() - want)
    worst = float((d / bound).max())
    assert worst <= 1.0, worst


@pytest.mark.parametrize("case", paged_ref.SHARES, ids=str)
def test_every_share_counts(kvq, case):
    s = shares.shares_case(case)
    want, bound = shares.shares_want(s)
    err = ints([0])
    got = kvq.kvq_paged4_attention(s["q"].cuda(), *gpu(s["pool"]), ints(s["table"]), ints(s["cu"]), ints(s["seq"]),
                                   max_new=s["max_new"], window=s["window"], softmax_scale=s["softmax_scale"], error=err)
    assert err.item() == 0
    check(got, want, bound)


@pytest.mark.parametrize("n,kernel", [(1, "decode"), (70, "prompt")])
@pytest.mark.parametrize("D", [64, 128])
def test_one_token_before_many_small_ones(kvq, n, kernel, D):
    """A token whose weight is 2^23 times another's, but whose value is 0: the others
    carry the result together."""
    k, v, q, T, ps, want, bound = shares.one_before_many(D, n, kernel)
    n_pages, batch = len(k[0]), 300
    # whole runs of tokens to a warp of the decode kernel; the prompt kernel serves one
    # request, the others have no new token
    new = [n] * batch if kernel == "decode" else [0] * 7 + [n] + [0] * 292
    q = np.concatenate([q] * (sum(new) // n))
    got = kvq.kvq_paged4_attention(torch.from_numpy(q).half().cuda(), *gpu(shares.pool(k, v)),
                                   ints(np.tile(np.arange(n_pages), (batch, 1))), ints(np.cumsum([0] + new)),
                                   ints([T] * batch), max_new=n, softmax_scale=1.0)
    for b in range(0, len(q), n):
        check(got[b:b + n], want, bound)


@pytest.mark.parametrize("n,idle", [(1, 0), (70, 140)])
def test_huge_scores(kvq, n, idle):
    """Scores of up to 2^24 in size: the largest takes all, so an output is a value (and a
    weight over the sum of weights, both rounded to 2^-11 at most)."""
    rng = np.random.default_rng(n)
    ps, D, T = 16, 64, 700
    n_pages = -(-T // ps)
    v = shares.held(rng.standard_normal((n_pages, 1, ps, D)))
    table = np.concatenate([np.arange(n_pages)[None], np.full((idle, n_pages), -1)])
    cu, seq = np.array([0] + [n] * (idle + 1)), np.array([T] + [0] * idle)
    for top, others in ((256.0, 224.0), (-224.0, -256.0)):
        for at in (0, 333, T - n):
            k = np.zeros((n_pages, 1, ps, D))
            k[..., 0] = others
            k[at // ps, 0, at % ps, 0] = top
            k = shares.held(k)
            for e in (12, 16, 17, 18, 19, 20, 22, 24):
                q = torch.zeros(n, 1, D, dtype=torch.float16, device="cuda")
                q[..., 0] = 2.0
                got = kvq.kvq_paged4_attention(q, *gpu(shares.pool(k, v)), ints(table), ints(cu), ints(seq),
                                               max_new=n, softmax_scale=2.0 ** (e - 9))
                want = np.broadcast_to(v[3][at // ps, 0, at % ps], (n, 1, D))
                check(got, want, np.abs(want) * (2.0 ** -10 + 2.0 ** -11) + 2.0 ** -25)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_serving_loop_against_its_own_pages(kvq, dtype):
    """Prompts, decode steps, drafted tokens and a chunk, with positions: every output
    against the attention over what the cache holds, and that against the turned keys and
    the values: half a step of the group, the step's rounding (2^-11 of it, 15 times),
    the value's rounding to fp16 before and behind."""
    rng = np.random.default_rng(23)
    H, R, D, ps, B = 2, 4, 128, 16, 5
    c = kvq.PagedCache4(n_pages=80, page_size=ps, n_q_heads=H * R, n_kv_heads=H, head_dim=D)
    ctx, table, turns = ints([0] * B), ints(np.full((B, 24), -1)), kvq.kvq_rotary_turns(D)
    free, n_free = ints(rng.permutation(80)), ints([80])
    hist = [[np.zeros((0, H, D))] * 2 for _ in range(B)]
    half_step = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    for new in [[40, 3, 0, 17, 70], [1] * 5, [1, 0, 5, 1, 2]] + [[1] * 5] * 4 + [[30, 4, 0, 1, 33]]:
        n = sum(new)
        k, v = (torch.from_numpy(rng.standard_normal((n + 2, H, D))).to(dtype).cuda() for _ in range(2))
        q = torch.from_numpy(rng.standard_normal((n + 2, H * R, D))).to(dtype).cuda()
        positions = ints([0] * (n + 2))
        cu, seq, slots, left = c.plan(ctx, ints(new), table, free, n_free, n + 2, positions=positions)
        ang = kvq.kvq_rotary_angles(positions, turns)
        q = c.append(k, v, slots, ang, q=q)
        out = c.attention(q, table, cu, seq, max_new=max(new))
        ctx, n_free = seq, left
        vals = []
        for i, (codes, meta) in enumerate(((c.k_codes, c.k_meta), (c.v_codes, c.v_meta))):
            m = meta.cpu().numpy()
            vals.append(paged4_ref.values(paged4_ref.unpack(codes.cpu().numpy(), i == 0), m[..., 0], m[..., 1]))
        at, tab = np.concatenate([[0], np.cumsum(new)]), table.cpu().numpy()
        want, bound = paged4_ref.attention(q[:n].double().cpu().numpy(), *vals, tab, at, seq.tolist(), ps, D ** -0.5, 0,
                                           paged_ref.WEIGHT_LOG2["prompt"], half_step)
        check(out[:n], want, bound)
        for b in range(B):
            for i, x in enumerate((kvq.kvq_rotate(k, ang), v)):
                hist[b][i] = np.concatenate([hist[b][i], x[at[b]:at[b + 1]].double().cpu().numpy()])
                t = np.arange(len(hist[b][i]))
                g = hist[b][i].reshape(len(t), H, D // 32, 32)
                got = vals[i][tab[b][t // ps], :, t % ps].reshape(g.shape)
                span, size = (g.max(-1) - g.min(-1))[..., None], np.abs(g).max(-1, keepdims=True)
                most = span / 30 * (1 + 2.0 ** -11) + span * 2.0 ** -11 + size * 2.0 ** -10 + 2.0 ** -21
                assert (np.abs(got - g) <= most).all()
    c.check()


def test_differences_are_fp32_numbers(kvq):
    """x - mn is rounded to fp32 before it is divided: 2^-24 above the middle between two
    codes is the middle, which goes to the even one; a step above it is not."""
    x = torch.zeros(2, 1, 64, dtype=torch.float16)
    x[:, 0, 0], x[:, 0, 1] = -832.0, 1088.0        # a step of 128, the middle of codes 6 and 7 at 0
    x[0, 0, 2], x[1, 0, 2] = 2.0 ** -24, 2.0 ** -13  # 832 + 2^-24 is no fp32 number, 832 + 2^-13 is
    pool = [torch.zeros(1, 1, 16, 32, dtype=torch.uint8, device="cuda") for _ in range(2)]
    pool += [torch.zeros(1, 1, 16, 2, 2, dtype=torch.float16, device="cuda") for _ in range(2)]
    kvq.kvq_paged4_append(x.cuda(), x.cuda(), ints([0, 1]), *pool)
    for i in range(2):
        codes = paged4_ref.unpack(pool[i].cpu().numpy(), i == 0)[0, 0, :2]
        assert codes[:, 2].tolist() == [6, 7] and (codes[:, :2] == [0, 15]).all()
        assert np.array_equal(codes, paged4_ref.quantize(x.double().numpy())[0][:, 0])
