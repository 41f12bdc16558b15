"""The paged 4-bit cache on the GPU: codes and metadata bit for bit, attention
within a bound derived in paged_ref.row."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import paged4_ref as ref  # noqa: E402
import paged_ref  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
HALF = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def kvq():
    from bit_kv_cache_11_gb300 import kvq as k
    return k


def ints(x):
    return torch.from_numpy(np.asarray(x).astype(np.int32)).cuda()


def f64(x):
    return x.double().cpu().numpy()


def empty_pool(n_pages, H, ps, D, fill=0x5a):
    codes = [torch.full((n_pages, H, ps, D // 2), fill, dtype=torch.uint8, device="cuda") for _ in range(2)]
    meta = [torch.full((n_pages, H, ps, D // 32, 2), 9.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    return codes + meta


# ---------------------------------------------------------------- append, read

def check_append(kvq, x, slots, ps, n_pages, rot=0, inter=False, q_heads=0, pads=(0, 0, 0), flags=0, q_in_place=False):
    """x: k and v, tensors [T][H][D]; every byte of the pool, the queries and what is
    read back."""
    T, H, D = x[0].shape
    dt = x[0].dtype
    rng = np.random.default_rng(T)
    put = []
    for y, pad in zip(x, pads):
        buf = torch.zeros(T, H * D + pad, dtype=dt, device="cuda")
        put.append(buf[:, :H * D].view(T, H, D))
        put[-1].copy_(y)
    kw = {}
    keys = x[0]
    if rot:
        ang = torch.from_numpy(ref.angles(rng.integers(0, 1 << 20, T), rng.integers(-(1 << 62), 1 << 62, rot // 2))).float()
        kw = dict(angles=ang.cuda(), interleaved=inter)
        turn = lambda y: torch.from_numpy(ref.rotate(y.float().numpy(), ang.numpy(), inter)).to(dt)  # noqa: E731
        keys = turn(x[0])
        if q_heads:
            q = torch.from_numpy(rng.standard_normal((T, q_heads, D))).to(dt)
            buf = torch.zeros(T, q_heads * D + pads[2], dtype=dt, device="cuda")
            qt = buf[:, :q_heads * D].view(T, q_heads, D)
            qt.copy_(q)
            kw.update(q=qt, **(dict(q_out=qt) if q_in_place else {}))
    pool, err = empty_pool(n_pages, H, ps, D), ints([0])
    before = [p.clone() for p in pool]
    got = kvq.kvq_paged4_append(*put, ints(slots), *pool, error=err, **kw)
    assert err.item() == flags
    if q_heads:
        assert torch.equal(got.cpu().view(torch.int16), turn(q).view(torch.int16))
    else:
        assert got is None
    slots = np.asarray(slots)
    real = (slots >= 0) & (slots < n_pages * ps)
    back = kvq.kvq_paged4_read(ints(slots), *pool, error=err)
    for i, y in enumerate((keys, x[1])):
        with np.errstate(over="ignore"):
            codes, step, mn = ref.quantize(f64(y)[real])
        want, meta = f64(before[i]).astype(np.uint8), before[2 + i].cpu().numpy()
        want[slots[real] // ps, :, slots[real] % ps] = ref.pack(codes, i == 0)
        meta[slots[real] // ps, :, slots[real] % ps] = np.stack([step, mn], -1)
        assert np.array_equal(pool[i].cpu().numpy(), want)
        assert np.array_equal(pool[2 + i].cpu().numpy().view(np.int16), meta.view(np.int16))
        val = np.zeros((T, H, D))
        val[real] = ref.values(codes, step, mn)
        assert np.array_equal(f64(back[i]), val)


def data(rng, T, H, D, dtype):
    loud = np.where(rng.random((H, D)) < 0.03, 6.0, 1.0)
    k = rng.standard_normal((T, H, D)) * loud
    v = rng.standard_normal((T, H, D)) * np.exp2(rng.integers(-12, 5, (T, H, 1)))
    return [torch.from_numpy(y).to(DT[dtype]) for y in (k, v)]


# page size, head_dim, kv heads, tokens, rotary_dim, interleaved, query heads
APPEND = [
    (16, 64, 1, 1, 0, False, 0), (16, 64, 2, 37, 64, False, 4), (32, 128, 3, 50, 128, False, 3),
    (64, 128, 8, 33, 128, True, 32), (128, 64, 2, 300, 16, True, 2), (128, 128, 1, 700, 24, False, 5),
    (64, 64, 5, 100, 62, True, 0), (16, 128, 2, 129, 96, False, 16), (32, 64, 1, 1000, 2, False, 1),
    (64, 128, 4, 1500, 128, False, 8), (16, 64, 12, 777, 64, False, 12),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", APPEND, ids=str)
def test_append(kvq, case, dtype):
    ps, D, H, T, rot, inter, q_heads = case
    rng = np.random.default_rng(sum(case))
    n_pages = -(-T // ps) + 3
    slots = rng.permutation(n_pages * ps)[:T]
    slots[rng.random(T) < 0.1] = -1
    check_append(kvq, data(rng, T, H, D, dtype), slots, ps, n_pages, rot, inter, q_heads)
    # consecutive slots, as a prompt's; strides; the queries in their own place
    check_append(kvq, data(rng, T, H, D, dtype), np.arange(T) + 5, ps, n_pages, rot, inter, q_heads, (8, 40, 16),
                 q_in_place=True)


def test_append_edges(kvq):
    """Constant groups, a step that underflows, ties, -0, the widest group, and
    bf16 numbers beyond fp16's."""
    D, T = 64, 9
    k = np.zeros((T, 1, D))
    k[0] = 3.25
    k[1, 0, ::2] = 2.0 ** -24                      # a step of 2^-24 / 15: zero
    k[2, 0] = np.arange(D) % 32 * 0.5              # ties at every other value
    k[3, 0] = -0.0
    k[4, 0, 5], k[4, 0, 6] = 65504.0, -65504.0
    k[5, 0, 40] = -1.0
    k[6, 0] = np.linspace(-1, 1, D)
    k[7, 0, :32], k[7, 0, 32:] = 2.0 ** -14, 60000.0
    k[8, 0] = 2.0 ** -24 * np.arange(D)
    for dt in (torch.float16, torch.bfloat16):
        x = torch.from_numpy(k).to(dt)
        check_append(kvq, [x, -x], np.arange(T), 16, 1)
        big = x.clone()
        if dt == torch.bfloat16:
            big[0, 0, 3], big[1, 0, 40] = 3e38, -1e30
            check_append(kvq, [big, x], np.arange(T), 16, 1)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_append_nonfinite(kvq, dtype):
    rng = np.random.default_rng(1)
    for odd in (float("inf"), -float("inf"), float("nan")):
        x = data(rng, 40, 2, 64, dtype)
        x[1][7, 1, 9] = odd
        check_append(kvq, x, np.arange(40), 16, 3, flags=16)
        x[0][3, 0, 63] = odd
        check_append(kvq, x, np.arange(40), 16, 3, flags=16)
        # one without a slot is not looked at
        check_append(kvq, x, np.where(np.isin(np.arange(40), (3, 7)), -1, np.arange(40)), 16, 3)


def test_append_flags_bad_slots(kvq):
    rng = np.random.default_rng(2)
    slots = np.arange(30)
    slots[[4, 20]] = 3 * 16, (1 << 31) - 1
    check_append(kvq, data(rng, 30, 2, 128, "fp16"), slots, 16, 3, flags=2)


def test_a_group_differs_by_half_a_step(kvq):
    """What the cache promises: every value within half a step, and its rounding."""
    rng = np.random.default_rng(3)
    x = data(rng, 200, 4, 128, "fp16")
    pool = empty_pool(13, 4, 16, 128)
    slots = ints(np.arange(200))
    kvq.kvq_paged4_append(x[0].cuda(), x[1].cuda(), slots, *pool)
    for i, y in enumerate(kvq.kvq_paged4_read(slots, *pool)):
        g = f64(x[i]).reshape(200, 4, 4, 32)
        span = (g.max(-1) - g.min(-1))[..., None]
        # the step's rounding moves code 15 by 15 half steps of it
        bound = span / 30 * (1 + 2.0 ** -11) + span * 2.0 ** -11 + np.abs(g).max(-1, keepdims=True) * 2.0 ** -11 + 2.0 ** -24 * 8
        assert (np.abs(f64(y).reshape(g.shape) - g) <= bound).all()


# ---------------------------------------------------------------- attention

def pages_of(rng, n_pages, H, ps, D, amp=1.0):
    """Random pages as a pool's buffers and as values."""
    codes = [rng.integers(0, 16, (n_pages, H, ps, D)).astype(np.uint8) for _ in range(2)]
    step = [(rng.uniform(0.05, 0.3, (n_pages, H, ps, D // 32)) * amp).astype(np.float16) for _ in range(2)]
    mn = [(-7.5 * s.astype(np.float64) + rng.standard_normal(s.shape) * 0.1 * amp).astype(np.float16) for s in step]
    return codes, step, mn


def to_gpu(codes, step, mn):
    pool = [torch.from_numpy(ref.pack(codes[i], i == 0)).cuda() for i in range(2)]
    return pool + [torch.from_numpy(np.stack([step[i], mn[i]], -1)).cuda() for i in range(2)]


def check_attention(kvq, case, seed=0, **over):
    ps, D, H, R, dtype, ctx, new, window = case
    idle = over.get("idle", 0)
    ctx, new = list(ctx) + [0] * idle, list(new) + [0] * idle
    rng = np.random.default_rng(seed + ps + D + H + R + sum(ctx) + sum(new) + window)
    B, T = len(ctx), sum(new)
    seq = np.array(ctx) + np.array(new)
    need = -(-seq // ps)
    n_pages = int(need.sum()) + 2
    codes, step, mn = pages_of(rng, n_pages, H, ps, D, over.get("page_amp", 1.0))
    vals = [ref.values(codes[i], step[i], mn[i]) for i in range(2)]
    ids = rng.permutation(n_pages)
    table = np.full((B, max(1, int(need.max())) + 1), -1, np.int32)
    used = np.zeros((n_pages, ps), bool)
    at = 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        for i in range(need[b]):
            used[ids[at + i], :max(0, min(ps, seq[b] - i * ps))] = True
        at += need[b]
    # rows that hold no token: NaN and infinities
    for i in range(2):
        step[i].transpose(0, 2, 1, 3)[~used] = np.nan
        mn[i].transpose(0, 2, 1, 3)[~used] = -np.inf
    pool = to_gpu(codes, step, mn)
    cu = np.concatenate([[0], np.cumsum(new)])
    pad = over.get("pad", 3)  # rows of no request
    wide = torch.from_numpy(rng.standard_normal((T + pad, H * R, D)) * over.get("amp", 1.0)).to(DT[dtype])
    buf = torch.zeros(T + pad, H * R * D + 16, dtype=DT[dtype])
    buf[:, :H * R * D] = wide.reshape(T + pad, -1)
    qt = buf.cuda()[:, :H * R * D].view(T + pad, H * R, D)
    out = torch.full((T + pad, H * R, D), 777.0, dtype=DT[dtype], device="cuda")
    err = ints([0])
    sm = over.get("scale", D ** -0.5)
    kw = dict(max_new=over.get("max_new", max(new)), softmax_scale=sm, window=window, error=err)
    args = (qt, *pool, ints(table), ints(cu), ints(seq))
    got = kvq.kvq_paged4_attention(*args, out=out, **kw)
    again = kvq.kvq_paged4_attention(*args, **kw)
    torch.cuda.synchronize()
    assert got is out and err.item() == 0
    assert torch.equal(out[:T], again[:T])
    want, bound = ref.attention(f64(wide)[:T], *vals, table, cu, seq, ps, sm, window,
                                paged_ref.WEIGHT_LOG2["prompt"], HALF[dtype])
    worst = float((np.abs(f64(out[:T]) - want) / bound).max())
    assert worst <= 1.0, worst
    assert (out[T:] == 777.0).all()


# page size, head_dim, kv heads, query heads a kv head, type, cached, new, window
DECODE = [
    (16, 64, 2, 1, "fp16", [0], [1], 0),
    (64, 128, 2, 1, "fp16", [256], [1], 0),
    (16, 128, 1, 1, "bf16", [15, 16, 17, 0, 31, 32], [1] * 6, 0),
    (32, 128, 2, 4, "bf16", [100, 3, 257, 1, 64], [1] * 5, 0),
    (64, 64, 3, 8, "fp16", [63, 64, 127, 500], [1] * 4, 0),
    (128, 64, 1, 2, "bf16", [1, 200, 128], [1] * 3, 0),
    (128, 128, 1, 5, "fp16", [400, 127], [1] * 2, 0),
    (64, 128, 1, 16, "fp16", [130, 5], [1] * 2, 0),
    (64, 128, 2, 4, "fp16", [5000], [1], 0),            # an item over many CTAs
    (16, 64, 1, 1, "bf16", [3000, 2, 90], [1] * 3, 0),
    (16, 128, 2, 2, "fp16", [300, 40, 7], [1] * 3, 33),  # window
    (64, 64, 1, 4, "bf16", [300, 40, 64], [1] * 3, 1),   # a window of the token itself
    (32, 128, 2, 2, "fp16", [70, 0, 33], [1, 0, 1], 0),  # a request without new tokens
    (32, 64, 2, 1, "fp16", list(range(0, 400, 9)), [1] * 45, 0),
    (128, 64, 1, 16, "bf16", [700, 64], [1, 1], 200),
]
MULTI = [
    (16, 64, 2, 8, "fp16", [100, 3, 0, 700], [5, 5, 3, 1], 0),
    (64, 128, 2, 4, "bf16", [60, 200], [5, 4], 0),
    (32, 128, 1, 1, "fp16", [0, 31], [9, 33], 0),
    (16, 64, 1, 8, "bf16", [500, 11], [5, 7], 40),
    (128, 128, 1, 3, "fp16", [120, 0, 250], [20, 1, 64], 0),
    (64, 64, 2, 2, "fp16", [0, 10], [150, 0], 0),
    (64, 128, 1, 5, "bf16", [0, 77], [130, 70], 65),
    (16, 128, 2, 1, "fp16", [0, 300], [520, 270], 0),
    (128, 128, 1, 8, "bf16", [100, 3], [65, 9], 0),
    (32, 128, 1, 2, "fp16", [50, 0, 7], [129, 1, 300], 100),
    (64, 128, 3, 1, "bf16", [1000], [257], 0),
    (64, 64, 1, 1, "fp16", [3], [600], 0),
    (128, 64, 1, 4, "bf16", [300, 0], [70, 140], 50),
]


@pytest.mark.parametrize("case", DECODE, ids=str)
def test_decode(kvq, case):
    check_attention(kvq, case)


@pytest.mark.parametrize("idle", [0, 140])
@pytest.mark.parametrize("case", MULTI, ids=str)
def test_several_new_tokens(kvq, case, idle):
    """(140 requests without tokens: a large batch, whose many-row requests the
    kernel of the prompts serves.)"""
    check_attention(kvq, case, idle=idle)


def test_a_mixed_batch(kvq):
    for ps, D, dtype in ((64, 128, "bf16"), (16, 64, "fp16"), (128, 128, "fp16")):
        for idle in (0, 80):
            check_attention(kvq, (ps, D, 2, 4, dtype, [900, 37, 0, 200, 0, 3], [1, 4, 300, 17, 33, 0], 0), idle=idle)
            check_attention(kvq, (ps, D, 2, 4, dtype, [900, 37, 0, 200], [1, 4, 300, 17], 50), idle=idle)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 3.0])
def test_any_softmax_scale(kvq, scale):
    check_attention(kvq, (16, 64, 1, 2, "fp16", [60], [1], 0), scale=scale)
    check_attention(kvq, (16, 64, 1, 1, "bf16", [60], [150], 0), scale=scale, idle=150)


@pytest.mark.parametrize("new,idle", [(1, 0), (130, 140)])
@pytest.mark.parametrize("D", [64, 128])
def test_large_values_are_attended_as_they_are_held(kvq, D, new, idle):
    """A value is the fp16 number nearest to code * step + minimum.  At sizes of
    500 that rounding moves a score by 0.01 .. 0.02 here, thirty times what the
    bound leaves."""
    case = (32, D, 2, 2, "fp16", [300, 40], [new, 3], 0)
    check_attention(kvq, case, page_amp=100.0, amp=0.02 * (128 / D) ** 0.5, idle=idle)


def test_max_new_may_be_a_loose_bound(kvq):
    check_attention(kvq, (32, 128, 1, 2, "fp16", [50, 7], [3, 1], 0), max_new=5000)
    check_attention(kvq, (32, 64, 1, 1, "bf16", [50, 7], [1, 1], 0), max_new=4)


def simple(rng, n_pages=12, H=1, ps=16, D=64, seq=(100, 40), new=(1, 1), R=2, dtype=torch.float16):
    idle = 150 if max(new) > 60 else 0
    seq, new = tuple(seq) + (0,) * idle, tuple(new) + (0,) * idle
    pool = to_gpu(*pages_of(rng, n_pages, H, ps, D))
    need = [-(-x // ps) for x in seq]
    table = np.full((len(seq), max(need)), -1)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = np.arange(at, at + n)
        at += n
    q = torch.from_numpy(rng.standard_normal((sum(new), H * R, D))).to(dtype).cuda()
    return [q, *pool, ints(table), ints(np.concatenate([[0], np.cumsum(new)])), ints(seq)]


@pytest.mark.parametrize("new", [(1, 1), (70, 33)])
def test_bad_pages_are_flagged_and_skipped(kvq, new):
    """A page id outside the pool hides its tokens, whatever lies around."""
    for bad in (-1, 12, 1 << 30, -(1 << 31)):
        args = simple(np.random.default_rng(2), new=new, seq=(100, 48))
        whole = kvq.kvq_paged4_attention(*args, max_new=max(new))
        err = ints([0])
        args[5][0, 2] = bad  # tokens 32 .. 47 of request 0
        got = kvq.kvq_paged4_attention(*args, max_new=max(new), error=err)
        assert err.item() == kvq.KVQ_PAGED_ERR_BAD_PAGE
        assert torch.isfinite(got).all()
        assert torch.equal(got[new[0]:], whole[new[0]:])
        # the tokens that are left, as if their pages followed one another
        if new == (1, 1):
            table = args[5].clone()
            table[0, 2:6] = table[0, 3:7].clone()
            seq = args[7].clone()
            seq[0] -= 16
            want = kvq.kvq_paged4_attention(*args[:5], table, args[6], seq, max_new=1)
            assert (got[:1] - want[:1]).abs().max() <= 2.0 ** -9 * want.abs().max()


def test_lengths_that_break_the_contract_are_skipped(kvq):
    for new in ((1, 1), (70, 33)):
        n = sum(new)
        for cu, seq in (([0, new[0], n + 5], None), ([0, -3, 2], None), ([-1, new[0], n], None),
                        (None, [-5, 40]), (None, [100, 1 << 30]), ([0, n, new[0]], None)):
            args = simple(np.random.default_rng(4), new=new)
            for i, bad in ((6, cu), (7, seq)):
                if bad:
                    args[i] = args[i].clone()
                    args[i][:len(bad)] = ints(bad)
            err, out = ints([0]), torch.full_like(args[0], 5.0)
            kvq.kvq_paged4_attention(*args, max_new=max(new), error=err, out=out)
            assert err.item() == kvq.KVQ_PAGED_ERR_LENGTH
            assert torch.isfinite(out).all()


@pytest.mark.parametrize("new", [(1, 1), (100, 5)])
def test_nan_queries_stay_in_their_rows(kvq, new):
    args = simple(np.random.default_rng(5), new=new, seq=(120, 40))
    want = kvq.kvq_paged4_attention(*args, max_new=max(new))
    args[0] = args[0].clone()
    args[0][0, 1, 3] = float("nan")
    got = kvq.kvq_paged4_attention(*args, max_new=max(new))
    assert torch.isnan(got[0, 1]).all()
    got[0, 1] = want[0, 1]
    assert torch.equal(got, want)


def test_a_query_that_sees_nothing_gives_zeros(kvq):
    for new in ((3, 2), (90, 70)):
        args = simple(np.random.default_rng(8), seq=(0, 40), new=new)
        err = ints([0])
        out = kvq.kvq_paged4_attention(*args, max_new=max(new), error=err)
        assert (out[:new[0]] == 0).all() and err.item() == 0
        early = max(0, new[1] - 40)
        assert (out[new[0]:new[0] + early] == 0).all()
        assert torch.isfinite(out).all() and (out[new[0] + early:] != 0).any()


@pytest.mark.parametrize("new", [(1, 1), (90, 70)])
def test_the_widest_window_is_none(kvq, new):
    args = simple(np.random.default_rng(9), seq=(0, 40), new=new)
    want = kvq.kvq_paged4_attention(*args, max_new=max(new))
    for window in (40, 112, 1 << 30, (1 << 31) - 1):
        assert torch.equal(kvq.kvq_paged4_attention(*args, max_new=max(new), window=window), want), window


def test_a_pool_beyond_four_gigabytes(kvq):
    """Pages at the end of a pool whose codes alone take 4.6 GB a side."""
    ps, D, H, T = 128, 128, 8, 300
    n_pages = 70000
    codes = [torch.zeros(n_pages, H, ps, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    meta = [torch.zeros(n_pages, H, ps, D // 32, 2, dtype=torch.float16, device="cuda") for _ in range(2)]
    pool = codes + meta
    ids = np.array([n_pages - 1, n_pages - 2, 65536])
    pos = np.arange(T)
    slots = ids[pos // ps] * ps + pos % ps
    k, v = (torch.randn(T, H, D, device="cuda").half() for _ in range(2))
    kvq.kvq_paged4_append(k, v, ints(slots), *pool)
    small = empty_pool(3, H, ps, D)
    kvq.kvq_paged4_append(k, v, ints(pos), *small)
    for a, b in zip(kvq.kvq_paged4_read(ints(slots), *pool), kvq.kvq_paged4_read(ints(pos), *small)):
        assert torch.equal(a, b)
    for n, idle in ((1, 0), (100, 0), (100, 30)):
        q = torch.randn(n, 2 * H, D, device="cuda").half()
        rest = (ints([0] + [n] * (idle + 1)), ints([T] + [0] * idle))
        wide = lambda t: ints(np.concatenate([[t], np.zeros((idle, 3))]))  # noqa: E731
        a = kvq.kvq_paged4_attention(q, *pool, wide(ids), *rest, max_new=n)
        b = kvq.kvq_paged4_attention(q, *small, wide([0, 1, 2]), *rest, max_new=n)
        assert torch.equal(a, b) and a.abs().max() > 0


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("batch,most_ctx,most_new,short", [(1, 0, 1, 0), (5, 90, 40, 0), (300, 500, 9, 0), (64, 60, 30, 20),
                                                           (4096, 3, 2, 0)])
def test_plan_positions(kvq, batch, most_ctx, most_new, short):
    """Every new token's position, with the plan's other outputs as without; requests
    that the stack cannot serve get theirs too."""
    rng = np.random.default_rng(batch + short)
    ctx, new = rng.integers(0, most_ctx + 1, batch), rng.integers(0, most_new + 1, batch)
    ps, n = 16, int(new.sum())
    pages = int((-(-(ctx + new) // ps)).sum())
    have = -(-ctx // ps)
    table = rng.integers(0, pages + 1, (batch, int((-(-(ctx + new) // ps)).max()) + 1))
    stack = pages - int(have.sum()) - short
    free = ints(rng.permutation(max(stack, 0) + 5))
    args = (ints(ctx), ints(new))
    t1, t2 = ints(table), ints(table)
    pos = torch.full((n + 6,), -9, dtype=torch.int32, device="cuda")
    a = kvq.kvq_paged_plan(*args, t1, free, ints([max(stack, 0)]), ps, n + 5)
    b = kvq.kvq_paged_plan(*args, t2, free, ints([max(stack, 0)]), ps, n + 5, positions=pos)
    assert torch.equal(t1, t2) and all(torch.equal(x, y) for x, y in zip(a, b))
    want = np.concatenate([c + np.arange(m) for c, m in zip(ctx, new)] + [np.zeros(5), [-9]])
    assert np.array_equal(f64(pos), want)


@pytest.mark.parametrize("cls", ["PagedCache", "PagedCache4"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_serving_steps(kvq, cls, dtype):
    """plan, angles, append (queries and keys turned) and attention over prompts,
    decode steps, drafted tokens and a chunk: equal to the separate calls, and to
    attention over the turned keys within the codes' half steps."""
    rng = np.random.default_rng(11)
    H, R, D, ps, B, n_pages = 2, 4, 128, 16, 5, 80
    cache = getattr(kvq, cls)(n_pages=n_pages, page_size=ps, n_q_heads=H * R, n_kv_heads=H, head_dim=D)
    other = getattr(kvq, cls)(n_pages=n_pages, page_size=ps, n_q_heads=H * R, n_kv_heads=H, head_dim=D)
    turns = kvq.kvq_rotary_turns(64, factor=4.0, original_len=4096)
    ctx, n_free, free = ints([0] * B), ints([n_pages]), ints(rng.permutation(n_pages))
    table = ints(np.full((B, 24), -1))
    hist = [[np.zeros((0, H, D))] * 2 for _ in range(B)]
    for new in [[40, 3, 0, 17, 70], [1] * 5, [1, 0, 5, 1, 2]] + [[1] * 5] * 14 + [[30, 4, 0, 1, 33]]:
        n = sum(new)
        k, v = (torch.from_numpy(rng.standard_normal((n + 2, H, D))).to(dtype).cuda() for _ in range(2))
        q = torch.from_numpy(rng.standard_normal((n + 2, H * R, D))).to(dtype).cuda()
        pos = torch.full((n + 2,), -7, dtype=torch.int32, device="cuda")
        was = f64(ctx).astype(int)
        cu, seq, slots, left = cache.plan(ctx, ints(new), table, free, n_free, n + 2, positions=pos)
        want_pos = np.concatenate([was[b] + np.arange(new[b]) for b in range(B)] + [np.zeros(2)])
        assert np.array_equal(f64(pos), want_pos)
        ang = kvq.kvq_rotary_angles(pos, turns, magnitude=1.1)
        tq = cache.append(k, v, slots, ang, q=q)
        tk = kvq.kvq_rotate(k, ang)
        assert torch.equal(tq, kvq.kvq_rotate(q, ang))
        other.store(tk, v, slots)
        for a, b in zip(cache._pool(), other._pool()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        out = cache.attention(tq, table, cu, seq, max_new=max(new))
        ctx, n_free = seq, left
        cuh = np.concatenate([[0], np.cumsum(new)])
        for b in range(B):
            if not new[b]:
                continue
            hist[b] = [np.concatenate([h, f64(x[cuh[b]:cuh[b + 1]])]) for h, x in zip(hist[b], (tk, v))]
            K, V = hist[b]
            for j in (0, new[b] - 1):
                p = len(K) - new[b] + j
                for hq in range(H * R):
                    z = K[:p + 1, hq // R] @ f64(tq[cuh[b] + j, hq]) * D ** -0.5
                    w = np.exp(z - z.max())
                    want = (w / w.sum()) @ V[:p + 1, hq // R]
                    d = f64(out[cuh[b] + j, hq]) - want
                    # half a step of a group of 32 normal numbers is about 0.14 at most: a bound on the rms
                    assert np.sqrt((d * d).mean()) < 0.15 + 0.1 * np.abs(want).max()
    cache.check()


@pytest.mark.parametrize("cls", ["PagedCache", "PagedCache4"])
def test_a_step_in_a_graph(kvq, cls):
    """A captured step (plan, angles, append, attention) replayed gives what the
    eager calls give, with eager calls of both kinds of pages in between."""
    rng = np.random.default_rng(12)
    H, R, D, ps, B, n_pages = 2, 4, 64, 16, 5, 80
    c = getattr(kvq, cls)(n_pages=n_pages, page_size=ps, n_q_heads=H * R, n_kv_heads=H, head_dim=D)
    ctx, n_free, free = ints([40, 3, 9, 17, 70]), ints([60]), ints(rng.permutation(n_pages))
    table = np.full((B, 24), -1)
    table[:, :6] = np.arange(30).reshape(5, 6)
    free = ints(np.concatenate([np.arange(30, 80), np.zeros(30)]))
    n_free, table = ints([50]), ints(table)
    k, v = (torch.randn(B, H, D, device="cuda").half() for _ in range(2))
    q = torch.randn(B, H * R, D, device="cuda").half()
    new, pos, turns = ints([1] * B), ints([0] * B), kvq.kvq_rotary_turns(D)

    def one():
        cu, seq, slots, left = c.plan(ctx, new, table, free, n_free, B, positions=pos)
        tq = c.append(k, v, slots, kvq.kvq_rotary_angles(pos, turns), q=q)
        out = c.attention(tq, table, cu, seq)
        ctx.copy_(seq)
        n_free.copy_(left)
        return out

    held = [*c._pool(), table, ctx, n_free]
    save = [t.clone() for t in held]

    def restore():
        for t, s in zip(held, save):
            t.copy_(s)

    want = [one().clone() for _ in range(20)]
    restore()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = one()
    restore()
    more = simple(rng, n_pages=64, seq=(900, 40))
    plain = kvq.kvq_paged4_attention(*more)
    for i in range(20):
        g.replay()
        assert torch.equal(out, want[i]), i
        assert torch.equal(kvq.kvq_paged4_attention(*more), plain)
    c.check()


def test_two_graphs_at_the_same_time(kvq):
    rng = np.random.default_rng(13)
    calls = [simple(rng, n_pages=700, H=2, seq=(5000, 3000), R=4),
             simple(rng, n_pages=700, H=2, seq=(2000, 6000), new=(2, 1), R=4)]
    want = [kvq.kvq_paged4_attention(*a, max_new=2) for a in calls]
    streams, graphs, outs = [torch.cuda.Stream() for _ in range(2)], [], []
    torch.cuda.synchronize()
    for a, s in zip(calls, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(3):
                o = kvq.kvq_paged4_attention(*a, max_new=2)
        graphs.append(g)
        outs.append(o)
    for _ in range(30):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_streams_and_workspaces_of_the_callers_choice(kvq):
    rng = np.random.default_rng(14)
    a = simple(rng, n_pages=700, H=2, seq=(5000, 3000), R=4)
    want = kvq.kvq_paged4_attention(*a)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(20):
        for s in (s1, s2.cuda_stream):
            o = torch.empty_like(want)
            kvq.kvq_paged4_attention(*a, out=o, stream=s)
            outs.append(o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    ws = torch.zeros(kvq.kvq_paged4_workspace_bytes(700, 2, 16, 64), dtype=torch.uint8, device="cuda")
    assert torch.equal(kvq.kvq_paged4_attention(*a, workspace=ws), want)
    assert (ws[:1024] == 0).all()


def test_cache_reports_what_was_flagged(kvq):
    c = kvq.PagedCache4(n_pages=4, page_size=16, n_q_heads=4, n_kv_heads=2, head_dim=64)
    x = torch.full((1, 2, 64), float("inf"), dtype=torch.float16, device="cuda")
    c.store(x, x, ints([3]))
    with pytest.raises(kvq.KvqError, match="non-finite"):
        c.check()
    k, v = c.read(ints([3, -1]))
    assert (k[0] == 65408).all() and (k[1] == 0).all() and torch.equal(k, v)
    with pytest.raises(kvq.KvqError, match="4 heads"):
        c.attention(torch.zeros(1, 2, 64, dtype=torch.float16, device="cuda"), ints([[0]]), ints([0, 1]), ints([1]))
    before = kvq.kvq_launch_count()
    c.store(x, x, ints([3]))
    assert kvq.kvq_launch_count() == before + 1
    with pytest.raises(kvq.KvqError, match="non-finite"):
        c.check()


def test_nothing_to_do(kvq):
    pool = empty_pool(4, 2, 16, 64)
    e = torch.empty(0, 2, 64, dtype=torch.float16, device="cuda")
    assert kvq.kvq_paged4_append(e, e, ints([]), *pool) is None
    assert kvq.kvq_paged4_read(ints([]), *pool)[0].shape == (0, 2, 64)
    out = kvq.kvq_paged4_attention(torch.empty(0, 4, 64, dtype=torch.float16, device="cuda"), *pool, ints([[0]]),
                                   ints([0, 0]), ints([5]))
    assert out.shape == (0, 4, 64)
