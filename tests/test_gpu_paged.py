"""The paged 8-bit cache on the GPU against 64-bit numpy: the plan's tables and
slots (equal), the store's codes and scales (equal), the attention (within the
derived tolerance of tests/paged_ref.py), and a serving loop of the three."""
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


DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
HALF = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}


def f64(x):
    return x.double().cpu().numpy()


# ---------------------------------------------------------------- plan

@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("batch,most_ctx,most_new,spare", [
    (1, 0, 1, 0), (1, 100, 1, 0), (5, 300, 1, 3), (64, 2000, 1, 0), (33, 500, 700, 11),
    (300, 200, 40, 0), (1025, 100, 3, 5), (4096, 20, 2, 0)])
def test_plan(kvq, ps, batch, most_ctx, most_new, spare):
    rng = np.random.default_rng(batch * 1000 + ps)
    ctx = rng.integers(0, most_ctx + 1, batch)
    new = rng.integers(0, most_new + 1, batch)
    if batch > 4:
        new[1] = 0
        ctx[2] = 0
        ctx[3] = max(ps, most_ctx // ps * ps)
    run_plan(kvq, rng, ctx, new, ps, spare=spare)


def run_plan(kvq, rng, ctx, new, ps, spare=0, short=0, width=None, extra_tokens=7, flags=0):
    batch = len(ctx)
    have = -(-np.maximum(ctx, 0) // ps)
    need = -(-(np.maximum(ctx, 0) + np.maximum(new, 0)) // ps) - have
    width = width or int((have + need).max()) + 2
    ids = rng.permutation(int((have + need).sum()) + spare + 1).astype(np.int32)
    table = np.full((batch, width), -7, np.int32)
    at = 0
    for b in range(batch):
        n = min(have[b], width)
        table[b, :n] = ids[at:at + n]
        at += n
    free = ids[at:]
    n_free = max(0, len(free) - short)
    n_tokens = int(np.maximum(new, 0).sum()) + extra_tokens
    want = ref.plan(ctx, new, table, free, n_free, ps, n_tokens)
    tab, err = ints(table), ints([0])
    cu, seq, slots, left = kvq.kvq_paged_plan(ints(ctx), ints(new), tab, ints(free), ints([n_free]),
                                              ps, n_tokens, error=err)
    for got, w in zip((tab, cu, seq, slots, left), want):
        assert np.array_equal(got.cpu().numpy().reshape(np.shape(w)), w)
    assert err.item() == flags, err.item()


def test_plan_when_the_stack_runs_out(kvq):
    """Requests that the stack cannot serve take nothing, those before them
    and those that need no page are served."""
    ctx, new = np.array([10, 64, 5, 30, 0, 7]), np.array([20, 65, 200, 1, 20, 3])
    for short in (0, 2, 5, 9, 20):
        run_plan(kvq, np.random.default_rng(short), ctx, new, 16, short=short, spare=0,
                 flags=kvq.KVQ_PAGED_ERR_NO_PAGES if short > 1 else 0)


def test_plan_flags_lengths(kvq):
    rng = np.random.default_rng(5)
    bad = kvq.KVQ_PAGED_ERR_LENGTH
    run_plan(kvq, rng, np.array([5, 40, 3]), np.array([2, -1, 30]), 16, flags=bad)
    run_plan(kvq, rng, np.array([5, -40, 3]), np.array([2, 1, 30]), 16, flags=bad)
    run_plan(kvq, rng, np.array([5, 40, 3]), np.array([2, 30, 30]), 16, width=4, flags=bad)
    # fewer slots than new tokens: those that fit are written
    run_plan(kvq, rng, np.array([5, 40, 3]), np.array([20, 30, 30]), 16, extra_tokens=-13, flags=bad)


# ---------------------------------------------------------------- store

def make_pool(rng, n_pages, H, ps, D, seed_scale=True):
    """Random codes without NaN and scales 2^-9 .. 2^-4, as tensors and numpy."""
    c = [rng.integers(0, 256, (n_pages, H, ps, D)).astype(np.uint8) for _ in range(2)]
    for x in c:
        x[(x & 127) == 127] = 0
    s = [2.0 ** rng.integers(-9, -3, (n_pages, H)).astype(np.float64) for _ in range(2)]
    dev = [torch.from_numpy(x).cuda().view(torch.float8_e4m3fn) for x in c]
    dsc = [torch.from_numpy(x.astype(np.float32)).cuda() for x in s]
    return c, s, dev, dsc


def check_store(kvq, rng, x, slots, ps, D, H, n_pages, dtype, fused=True, flags=0):
    T = len(slots)
    c, s, pages, scale = make_pool(rng, n_pages, H, ps, D)
    t = [torch.from_numpy(v).to(DT[dtype]) for v in x]
    if fused:  # k and v as slices of a wider projection
        buf = torch.empty(T, 2 * H * D + 8, dtype=DT[dtype])
        buf[:, :H * D] = t[0].reshape(T, -1)
        buf[:, H * D + 8:] = t[1].reshape(T, -1)
        buf = buf.cuda()
        k, v = buf[:, :H * D].view(T, H, D), buf[:, H * D + 8:].view(T, H, D)
    else:
        k, v = t[0].cuda(), t[1].cuda()
    err = ints([0])
    kvq.kvq_paged_store(k, v, ints(slots), pages[0], pages[1], scale[0], scale[1], error=err)
    for i in range(2):
        codes, sc = ref.store(f64(t[i]), slots, c[i], s[i], ps)
        assert np.array_equal(scale[i].cpu().numpy().astype(np.float64), sc)
        got = pages[i].view(torch.uint8).cpu().numpy()
        # -0 and +0 are the same value; everything else is compared as bits
        same = (got == codes) | ((got & 127) == 0) & ((codes & 127) == 0)
        assert same.all(), np.argwhere(~same)[:5]
    assert err.item() == flags


def slots_of(rng, runs, ps, n_pages, pad=0):
    """Slots of runs (first row, rows) that continue over fresh pages."""
    ids = list(rng.permutation(n_pages))
    out = []
    for row, n in runs:
        page = ids.pop()
        for _ in range(n):
            if row == ps:
                row, page = 0, ids.pop()
            out.append(page * ps + row)
            row += 1
        out += [-1] * pad
    return out


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("ps,D,H,runs,pad", [
    (64, 128, 2, [(0, 1)], 0),
    (64, 128, 3, [(5, 1), (63, 1), (0, 1), (17, 1)], 0),
    (16, 64, 1, [(3, 40), (0, 16), (15, 2), (0, 1)], 2),
    (128, 128, 2, [(0, 128), (100, 60), (1, 1)], 0),
    (32, 64, 5, [(31, 1), (7, 70), (0, 33)], 1),
    # enough tokens for the chunk kernel (over 1024)
    (64, 128, 2, [(10, 700), (0, 1), (0, 500), (63, 130)], 0),
    (16, 64, 3, [(1, 600), (15, 1), (9, 1), (0, 1), (0, 550)], 3),
    (128, 64, 1, [(127, 1000), (64, 64), (5, 9), (0, 128)], 0),
    (128, 128, 1, [(3, 300), (127, 2), (0, 128)], 0),
    (32, 128, 1, [(i % 32, 1 + i % 3) for i in range(90)] + [(0, 200)], 0),
])
def test_store(kvq, dtype, ps, D, H, runs, pad):
    rng = np.random.default_rng(ps + D + len(runs))
    n_pages = sum(n // ps + 2 for _, n in runs) + 3
    slots = slots_of(rng, runs, ps, n_pages, pad)
    T = len(slots)
    # token sizes vary over 2^12, so scales grow, stay, and reach the subnormal codes
    x = [rng.standard_normal((T, H, D)) * 2.0 ** rng.integers(-8, 4, (T, H, 1)) for _ in range(2)]
    check_store(kvq, rng, x, slots, ps, D, H, n_pages, dtype, fused=D == 128)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n", [1, 50])
def test_store_beside_rows_of_a_larger_scale(kvq, dtype, n):
    """Rows behind older ones of scales up to 2^40: codes around E4M3's least
    value and 0, for 2^-e above, at and below fp16's least number 2^-24."""
    rng = np.random.default_rng(n)
    ps, H = 64, 3
    for D in (64, 128):
        for e in (*range(20, 28), 40):
            c, s, pages, scale = make_pool(rng, 2, H, ps, D)
            for i in range(2):
                s[i][:] = 2.0 ** e
                scale[i].fill_(2.0 ** e)
            slots = np.arange(n) + ps + 9
            x = [torch.from_numpy(rng.uniform(-65504, 65504, (n, H, D))).to(DT[dtype]) for _ in range(2)]
            kvq.kvq_paged_store(x[0].cuda(), x[1].cuda(), ints(slots), *pages, *scale)
            for i in range(2):
                codes, sc = ref.store(f64(x[i]), slots, c[i], s[i], ps)
                assert np.array_equal(scale[i].cpu().numpy().astype(np.float64), sc)
                got = pages[i].view(torch.uint8).cpu().numpy()
                same = (got == codes) | ((got & 127) == 0) & ((codes & 127) == 0)
                assert same.all(), (D, e, np.argwhere(~same)[:5])


@pytest.mark.parametrize("ps,D,dtype", [(16, 64, "fp16"), (16, 128, "bf16"), (32, 128, "fp16"),
                                        (64, 64, "bf16"), (64, 128, "fp16"), (128, 128, "bf16")])
def test_store_large_calls(kvq, ps, D, dtype):
    """Over 16384 token heads: whole chunks, of long runs and of single tokens."""
    rng = np.random.default_rng(ps + D)
    H, n_pages = 24, 1500 + 3000 // ps
    runs = [(5 % ps, 700), (0, 1)] + [(int(r), 1) for r in rng.integers(0, ps, 500)] + [(ps - 1, 600)]
    slots = slots_of(rng, runs, ps, n_pages)
    x = [rng.standard_normal((len(slots), H, D)) * 2.0 ** rng.integers(-8, 4, (len(slots), H, 1))
         for _ in range(2)]
    check_store(kvq, rng, x, slots, ps, D, H, n_pages, dtype)


@pytest.mark.parametrize("T", [3, 1100])
def test_store_edges(kvq, T):
    """Zero rows, exact ties and borders of the scale (448 * 2^e and the next
    number), the type's largest and smallest values."""
    rng = np.random.default_rng(T)
    ps, D, H = 16, 64, 6
    x = np.zeros((T, H, D))
    x[:, 1] = 448.0 * 2.0 ** -3
    x[:, 2] = 448.25
    x[:, 3, :] = np.resize(ref.E4M3[1:126] + np.diff(ref.E4M3[:127])[1:] / 2, D)  # halfway
    x[:, 4, ::2] = 65504.0
    x[:, 5, 5] = 2.0 ** -24
    x[:, 5, 6] = -(2.0 ** -25)
    slots = slots_of(rng, [(0, T)], ps, T // ps + 4)
    check_store(kvq, rng, [x, -x[:, ::-1].copy()], slots, ps, D, H, T // ps + 4, "fp16")
    y = x.copy()
    y[:, 0, 3] = 1e30
    y[:, 1, 7] = 3e38
    y[:, 5, 9] = 1e-38
    check_store(kvq, rng, [y, y[:, ::-1].copy()], slots, ps, D, H, T // ps + 4, "bf16")


@pytest.mark.parametrize("T", [5, 1300])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_store_nonfinite(kvq, T, dtype):
    """Infinities saturate at a scale the finite elements set, NaN becomes 0."""
    rng = np.random.default_rng(T)
    ps, D, H = 32, 128, 2
    x = rng.standard_normal((T, H, D))
    x[1, 0, 3], x[2, 0, 9], x[T - 1, 1, 0] = np.inf, -np.inf, np.nan
    slots = slots_of(rng, [(7, T)], ps, T // ps + 4)
    check_store(kvq, rng, [x, rng.standard_normal((T, H, D))], slots, ps, D, H, T // ps + 4, dtype,
                flags=kvq.KVQ_PAGED_ERR_NONFINITE)


def test_store_page_by_page_equals_at_once(kvq):
    """Where no scale grows, token by token gives the same bytes as one call."""
    rng = np.random.default_rng(3)
    ps, D, H, T = 16, 64, 2, 40
    x = rng.uniform(0.5, 1.0, (T, H, D)) * rng.choice([-1, 1], (T, H, D))
    x[::16, :, 0] = 1.0
    k = torch.from_numpy(x).half().cuda()
    slots = ints(slots_of(rng, [(0, T)], ps, 6))
    got = []
    for step in (T, 1, 7):
        _, _, pages, scale = make_pool(np.random.default_rng(1), 6, H, ps, D)
        for i in range(0, T, step):
            kvq.kvq_paged_store(k[i:i + step], k[i:i + step], slots[i:i + step].clone(), *pages, *scale)
        got.append([z.view(torch.uint8).cpu() for z in pages] + [z.cpu() for z in scale])
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- attention

def check_attention(kvq, case, seed=0, **over):
    ps, D, H, R, dtype, ctx, new, window = case
    # requests without tokens behind the others: with many of them the call
    # counts as a large batch, whose many-row requests the prompt kernel serves
    idle = over.get("idle", 0)
    ctx, new = list(ctx) + [0] * idle, list(new) + [0] * idle
    rng = np.random.default_rng(seed + ps + D + H + R + sum(ctx) + sum(new) + window)
    B, T = len(ctx), sum(new)
    seq = np.array(ctx) + np.array(new)
    need = -(-seq // ps)
    width = max(1, int(need.max())) + 1
    n_pages = int(need.sum()) + 2
    c, s, pages, scale = make_pool(rng, n_pages, H, ps, D)
    # values of ordinary size: codes of N(0, 1) at every scale
    for i in range(2):
        c[i] = ref.e4m3_code(rng.standard_normal(c[i].shape) / s[i][..., None, None] / 8)
    ids = rng.permutation(n_pages)
    table = np.full((B, width), -1, np.int32)
    at = 0
    stale = [x.copy() for x in c]
    used = np.zeros((n_pages, ps), bool)
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        for i in range(need[b]):
            used[ids[at + i], :max(0, min(ps, seq[b] - i * ps))] = True
        at += need[b]
    # rows that hold no token are NaN codes, and so are unused pages
    for x in stale:
        x.transpose(0, 2, 1, 3)[~used] = 0x7F
    pages = [torch.from_numpy(x).cuda().view(torch.float8_e4m3fn) for x in stale]
    cu = np.concatenate([[0], np.cumsum(new)])
    pad = over.get("pad", 3)  # rows of no request
    q = (rng.standard_normal((T + pad, H * R, D)) * over.get("amp", 1.0))
    wide = torch.from_numpy(q).to(DT[dtype])
    buf = torch.zeros(T + pad, H * R * D + 16, dtype=DT[dtype])
    buf[:, :H * R * D] = wide.reshape(T + pad, -1)
    qt = buf.cuda()[:, :H * R * D].view(T + pad, H * R, D)
    out = torch.full((T + pad, H * R, D), 777.0, dtype=DT[dtype], device="cuda")
    err = ints([0])
    sm = D ** -0.5
    kw = dict(max_new=over.get("max_new", max(new)), softmax_scale=sm, window=window, error=err)
    args = (qt, *pages, *scale, ints(table), ints(cu), ints(seq))
    got = kvq.kvq_paged_attention(*args, out=out, **kw)
    again = kvq.kvq_paged_attention(*args, **kw)
    torch.cuda.synchronize()
    assert got is out and err.item() == 0
    assert torch.equal(out[:T], again[:T])
    want, size, reach = ref.attention(f64(wide)[:T], c[0], c[1], s[0], s[1], table, cu, seq, ps, sm, window)
    tol = ref.tolerance(want, size, reach, HALF[dtype], max(seq), (448 * s[1]).max())
    d = np.abs(f64(out[:T]) - want)
    worst = float((d / tol).max())
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
]
MULTI = [
    (16, 64, 2, 8, "fp16", [100, 3, 0, 700], [5, 5, 3, 1], 0),
    (64, 128, 2, 4, "bf16", [60, 200], [5, 4], 0),
    (32, 128, 1, 1, "fp16", [0, 31], [9, 33], 0),
    (16, 64, 1, 8, "bf16", [500, 11], [5, 7], 40),
    (128, 128, 1, 3, "fp16", [120, 0, 250], [20, 1, 64], 0),
    (64, 64, 2, 2, "fp16", [0, 10], [150, 0], 0),
    (64, 128, 1, 5, "bf16", [0, 77], [130, 70], 65),
    # several row tiles of a request, a last one of few rows
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
    check_attention(kvq, case, idle=idle)


@pytest.mark.parametrize("D", [64, 128])
def test_around_the_turn_to_the_prompt_kernel(kvq, D):
    """Rows just below, at and above what one kernel leaves to the other."""
    for new in (31, 32, 33, 48, 49):
        check_attention(kvq, (32, D, 1, 1, "fp16", [200, 9], [new, 3], 0), idle=140)
    for new in (265, 266, 267, 400):
        check_attention(kvq, (64, D, 4, 1, "bf16", [30], [new], 0), idle=3)


def test_a_mixed_batch(kvq):
    """Decodes, drafted tokens, a short and a long prompt in one call."""
    for ps, D, dtype in ((64, 128, "bf16"), (16, 64, "fp16"), (128, 128, "fp16")):
        for idle in (0, 80):
            check_attention(kvq, (ps, D, 2, 4, dtype, [900, 37, 0, 200, 0, 3], [1, 4, 300, 17, 33, 0], 0), idle=idle)
            check_attention(kvq, (ps, D, 2, 4, dtype, [900, 37, 0, 200], [1, 4, 300, 17], 50), idle=idle)


def test_the_largest_batch(kvq):
    """4096 requests, of no token to three pages, in both kernels' batches."""
    rng = np.random.default_rng(1)
    ctx = [int(x) for x in rng.integers(0, 40, 4096)]
    check_attention(kvq, (16, 64, 1, 1, "fp16", ctx, [int(x) for x in rng.integers(0, 3, 4096)], 0))
    new = [0] * 4096
    new[17], new[4095], new[300] = 60, 70, 1
    check_attention(kvq, (16, 128, 1, 1, "bf16", ctx, new, 0))
    args = simple(rng)
    big = [ints(np.zeros((4097, 2))), ints(np.zeros(4098)), ints(np.zeros(4097))]
    with pytest.raises(kvq.KvqError) as e:
        kvq.kvq_paged_attention(*args[:5], *big)
    assert e.value.status == kvq.KVQ_ERR_UNSUPPORTED


def test_new_tokens_behind_other_rows(kvq):
    """The first request's rows need not be row 0; rows before it are left."""
    args = simple(np.random.default_rng(3))
    want = kvq.kvq_paged_attention(*args)
    q = torch.cat([torch.full_like(args[0], 9.0), args[0]])
    out = torch.full_like(q, 5.0)
    kvq.kvq_paged_attention(q, *args[1:6], args[6] + 2, args[7], out=out)
    assert torch.equal(out[2:], want) and (out[:2] == 5.0).all()


def test_max_new_may_be_a_loose_bound(kvq):
    check_attention(kvq, (32, 128, 1, 2, "fp16", [50, 7], [3, 1], 0), max_new=5000)
    check_attention(kvq, (32, 64, 1, 1, "bf16", [50, 7], [1, 1], 0), max_new=4)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30])
def test_any_softmax_scale(kvq, scale):
    """A scale of 0 averages the values; a negative one turns the order."""
    for n, R in ((1, 2), (150, 1)):
        rng = np.random.default_rng(n)
        ps, D, T0 = 16, 64, 60
        c, s, pages, sc = make_pool(rng, 20, 1, ps, D)
        for i in range(2):
            c[i] = ref.e4m3_code(rng.standard_normal(c[i].shape) / s[i][..., None, None] / 8)
            pages[i] = torch.from_numpy(c[i]).cuda().view(torch.float8_e4m3fn)
        q = torch.from_numpy(rng.standard_normal((n, R, D))).half()
        idle = 150 if n > 1 else 0  # (a large batch: the prompt kernel)
        table = np.concatenate([np.arange(20)[None], np.full((idle, 20), -1)])
        cu, seq = np.array([0] + [n] * (idle + 1)), np.array([T0 + n] + [0] * idle)
        got = kvq.kvq_paged_attention(q.cuda(), *pages, *sc, ints(table), ints(cu), ints(seq),
                                      max_new=n, softmax_scale=scale)
        want, size, reach = ref.attention(f64(q), c[0], c[1], s[0], s[1], table, cu, seq, ps, scale)
        tol = ref.tolerance(want, size, reach, HALF["fp16"], T0 + n, (448 * s[1]).max())
        worst = float((np.abs(f64(got) - want) / tol).max())
        assert worst <= 1.0, worst


def simple(rng, n_pages=12, H=1, ps=16, D=64, seq=(100, 40), new=(1, 1), R=2, dtype=torch.float16):
    """A small call's arguments.  Calls of many rows get requests without
    tokens behind, so that the prompt kernel serves them."""
    idle = 150 if max(new) > 60 else 0
    seq, new = tuple(seq) + (0,) * idle, tuple(new) + (0,) * idle
    c, s, pages, sc = make_pool(rng, n_pages, H, ps, D)
    need = [-(-x // ps) for x in seq]
    table = np.full((len(seq), max(need)), -1)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = np.arange(at, at + n)
        at += n
    q = torch.from_numpy(rng.standard_normal((sum(new), H * R, D))).to(dtype).cuda()
    cu = np.concatenate([[0], np.cumsum(new)])
    return [q, *pages, *sc, ints(table), ints(cu), ints(seq)]


@pytest.mark.parametrize("new", [(1, 1), (70, 33)])
def test_bad_pages_are_flagged_and_skipped(kvq, new):
    """A page id outside the pool hides its tokens, whatever lies around."""
    for bad in (-1, 12, 1 << 30, -(1 << 31)):
        args = simple(np.random.default_rng(2), new=new, seq=(100, 48))
        whole = kvq.kvq_paged_attention(*args, max_new=max(new))
        err = ints([0])
        args[5][0, 2] = bad  # tokens 32 .. 47 of request 0
        got = kvq.kvq_paged_attention(*args, max_new=max(new), error=err)
        assert err.item() == kvq.KVQ_PAGED_ERR_BAD_PAGE
        assert torch.equal(got[new[0]:], whole[new[0]:]) and torch.isfinite(got).all()
        # the others of request 0 are as if those tokens had no weight: with a
        # window that leaves them out, nothing is flagged and nothing changes
        err.zero_()
        args[5][0, 2] = 2
        want = kvq.kvq_paged_attention(*args, max_new=max(new), window=20)
        args[5][0, 0] = bad
        if new[0] == 1:
            again = kvq.kvq_paged_attention(*args, max_new=1, window=20, error=err)
            assert err.item() == 0 and torch.equal(again, want)


def test_store_flags_bad_slots(kvq):
    c, s, pages, sc = make_pool(np.random.default_rng(0), 4, 2, 16, 64)
    before = [p.view(torch.uint8).clone() for p in pages]
    for T in (3, 1200):
        k = torch.ones(T, 2, 64, dtype=torch.float16, device="cuda")
        slots = np.full(T, -1)
        slots[1] = 4 * 16 + 3
        slots[2] = (1 << 31) - 5
        err = ints([0])
        kvq.kvq_paged_store(k, k, ints(slots), *pages, *sc, error=err)
        assert err.item() == kvq.KVQ_PAGED_ERR_BAD_PAGE
        assert all(torch.equal(p.view(torch.uint8), b) for p, b in zip(pages, before))


def test_lengths_that_break_the_contract_are_skipped(kvq):
    rng = np.random.default_rng(4)
    for new in ((2, 3), (90, 80)):
        args = simple(rng, seq=(100, 90), n_pages=16, new=new)
        n = sum(new)
        for seq, cu, ok in (((113, 90), None, 1), ((-5, 90), None, 1), ((100, 1 << 30), None, 0),
                            (None, (0, new[0], n + 1), 0), (None, (-1, new[0], n), 1),
                            (None, (new[0], 0, n), None)):
            a = list(args)
            idle = a[7].numel() - 2
            if seq:
                a[7] = ints(list(seq) + [0] * idle)
            if cu:
                a[6] = ints(list(cu) + [cu[-1]] * idle)
            out = torch.full_like(args[0], 5.0)
            err = ints([0])
            kvq.kvq_paged_attention(*a, max_new=max(new), out=out, error=err)
            assert err.item() == kvq.KVQ_PAGED_ERR_LENGTH
            rows = [slice(0, new[0]), slice(new[0], n)]
            for b in range(2):
                if ok is not None:
                    assert bool((out[rows[b]] == 5.0).all()) == (b != ok)
        # more new tokens than max_new
        out, err = torch.full_like(args[0], 5.0), ints([0])
        kvq.kvq_paged_attention(*args, max_new=min(new), out=out, error=err)
        assert err.item() == kvq.KVQ_PAGED_ERR_LENGTH


@pytest.mark.parametrize("new", [(1, 1), (100, 5)])
def test_nan_queries_stay_in_their_rows(kvq, new):
    for dtype in (torch.float16, torch.bfloat16):
        args = simple(np.random.default_rng(6), H=2, n_pages=16, seq=(100, 48), new=new, dtype=dtype)
        want = kvq.kvq_paged_attention(*args, max_new=max(new))
        args[0][0, 1, 3] = float("nan")
        got = kvq.kvq_paged_attention(*args, max_new=max(new))
        assert got[0, 1].isnan().all()
        rest = torch.ones(got.shape[:2], dtype=torch.bool, device="cuda")
        rest[0, 1] = False
        assert torch.equal(got[rest], want[rest])


def test_a_query_that_sees_nothing_gives_zeros(kvq):
    for new in ((3, 2), (90, 70)):
        args = simple(np.random.default_rng(8), seq=(0, 40), new=new)
        err = ints([0])
        out = kvq.kvq_paged_attention(*args, max_new=max(new), error=err)
        # request 0 holds nothing; request 1's first queries lie before token 0
        assert (out[:new[0]] == 0).all() and err.item() == 0
        early = max(0, new[1] - 40)
        assert (out[new[0]:new[0] + early] == 0).all()
        assert torch.isfinite(out).all() and (out[new[0] + early:] != 0).any()


@pytest.mark.parametrize("new", [(1, 1), (90, 70)])
def test_the_widest_window_is_none(kvq, new):
    args = simple(np.random.default_rng(9), seq=(0, 40), new=new)
    want = kvq.kvq_paged_attention(*args, max_new=max(new))
    for window in (40, 112, 1 << 30, (1 << 31) - 1):
        got = kvq.kvq_paged_attention(*args, max_new=max(new), window=window)
        assert torch.equal(got, want), window


def test_pages_with_any_scale(kvq):
    """Scales that are no powers of two: attended as they are, rounded up by a
    store that adds rows."""
    rng = np.random.default_rng(21)
    ps, D = 16, 64
    c, s, pages, sc = make_pool(rng, 4, 1, ps, D)
    for i in range(2):
        c[i] = ref.e4m3_code(rng.standard_normal(c[i].shape) * 8)
        s[i] = rng.uniform(0.01, 0.2, s[i].shape).astype(np.float32).astype(np.float64)
    pages = [torch.from_numpy(x).cuda().view(torch.float8_e4m3fn) for x in c]
    sc = [torch.from_numpy(x.astype(np.float32)).cuda() for x in s]
    q = torch.from_numpy(rng.standard_normal((2, 2, D))).half()
    table, cu, seq = np.arange(4)[None], np.array([0, 2]), np.array([55])
    got = kvq.kvq_paged_attention(q.cuda(), *pages, *sc, ints(table), ints(cu), ints(seq), max_new=2)
    want, size, reach = ref.attention(f64(q), c[0], c[1], s[0], s[1], table, cu, seq, ps, D ** -0.5)
    tol = ref.tolerance(want, size, reach, HALF["fp16"], 55, (448 * s[1]).max())
    assert float((np.abs(f64(got) - want) / tol).max()) <= 1.0
    x = torch.full((1, 1, D), 1.0, dtype=torch.float16, device="cuda")
    kvq.kvq_paged_store(x, x, ints([3 * ps + 7]), *pages, *sc)
    for i in range(2):
        now = 2.0 ** np.ceil(np.log2(s[i][3, 0]))
        assert sc[i][3, 0].item() == now
        codes = pages[i].view(torch.uint8).cpu().numpy()[3, 0, :7]
        assert np.array_equal(ref.E4M3[codes], ref.E4M3[ref.e4m3_code(ref.E4M3[c[i][3, 0, :7]] * (s[i][3, 0] / now))])


def test_values_of_very_different_pages(kvq):
    """Pages whose scales differ by 2^50: a page of huge values with little
    weight does not drown the others, a page of zeros still takes its share."""
    for n in (1, 80):
        ps, D = 16, 64
        rng = np.random.default_rng(n)
        c, s, pages, sc = make_pool(rng, 8, 1, ps, D)
        for i in range(2):
            c[i] = ref.e4m3_code(rng.standard_normal(c[i].shape))
        s[0][:] = 1.0
        s[1][:] = 1.0
        s[1][1], s[1][2], s[1][3] = 2.0 ** 35, 2.0 ** -15, 2.0 ** 10
        c[1][4] = 0
        c[0][1] = ref.e4m3_code(-8 * np.ones((1, ps, D)))  # page 1: scores near -64 sigma
        pages = [torch.from_numpy(x).cuda().view(torch.float8_e4m3fn) for x in c]
        sc = [torch.from_numpy(x.astype(np.float32)).cuda() for x in s]
        q = torch.from_numpy(np.abs(rng.standard_normal((n, 1, D)))).half()
        idle = 150 if n > 1 else 0  # (a large batch: the prompt kernel)
        table = np.concatenate([np.arange(8)[None], np.full((idle, 8), -1)])
        cu, seq = np.array([0] + [n] * (idle + 1)), np.array([ps * 8] + [0] * idle)
        got = kvq.kvq_paged_attention(q.cuda(), *pages, *sc, ints(table), ints(cu), ints(seq),
                                      max_new=n, softmax_scale=0.25)
        want, size, reach = ref.attention(f64(q), c[0], c[1], s[0], s[1], table, cu, seq, ps, 0.25)
        # the floor of a weight is 2^-25 of the largest p * scale of its row
        tol = ref.tolerance(want, size, reach, HALF["fp16"], 1, 0.0)
        tol += size.max(axis=-1, keepdims=True) * ps * 8 * 2.0 ** -25
        worst = float((np.abs(f64(got) - want) / tol).max())
        assert worst <= 1.0, worst


def test_a_pool_beyond_four_gigabytes(kvq):
    """Pages at the end of a pool of 4.6 GB (K and V each)."""
    ps, D, H = 128, 128, 8
    n_pages = 35000
    pages = [torch.zeros(n_pages, H, ps, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
             for _ in range(2)]
    scale = [torch.ones(n_pages, H, device="cuda") for _ in range(2)]
    T = 300
    ids = np.array([n_pages - 1, n_pages - 2, 32768])
    pos = np.arange(T)
    slots = ids[pos // ps] * ps + pos % ps
    k = torch.randn(T, H, D, device="cuda").half()
    v = torch.randn(T, H, D, device="cuda").half()
    kvq.kvq_paged_store(k, v, ints(slots), *pages, *scale)
    small = [torch.zeros(3, H, ps, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
             for _ in range(2)]
    small_scale = [torch.ones(3, H, device="cuda") for _ in range(2)]
    kvq.kvq_paged_store(k, v, ints(pos), *small, *small_scale)
    for n, idle in ((1, 0), (100, 0), (100, 30)):
        q = torch.randn(n, 2 * H, D, device="cuda").half()
        rest = (ints([0] + [n] * (idle + 1)), ints([T] + [0] * idle))
        wide = lambda t: ints(np.concatenate([[t], np.zeros((idle, 3))]))  # noqa: E731
        a = kvq.kvq_paged_attention(q, *pages, *scale, wide(ids), *rest, max_new=n)
        b = kvq.kvq_paged_attention(q, *small, *small_scale, wide([0, 1, 2]), *rest, max_new=n)
        assert torch.equal(a, b) and a.abs().max() > 0


# ---------------------------------------------------------------- together

def serving_state(kvq, rng, H=2, R=4, D=128, ps=16, batch=5, n_pages=80):
    cache = kvq.PagedCache(n_pages=n_pages, page_size=ps, n_q_heads=H * R, n_kv_heads=H, head_dim=D)
    return dict(cache=cache, ctx=ints([0] * batch), table=ints(np.full((batch, 24), -1)),
                free=ints(rng.permutation(n_pages)), n_free=ints([n_pages]), H=H, R=R, D=D, ps=ps,
                batch=batch)


def step(kvq, st, rng, new, dtype=torch.float16, log=None):
    """plan, store and attend for one step; advances the lengths."""
    n = int(sum(new))
    k, v = (torch.from_numpy(rng.standard_normal((n + 2, st["H"], st["D"]))).to(dtype).cuda() for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((n + 2, st["H"] * st["R"], st["D"]))).to(dtype).cuda()
    c = st["cache"]
    cu, seq, slots, left = c.plan(st["ctx"], ints(new), st["table"], st["free"], st["n_free"], n + 2)
    c.store(k, v, slots)
    out = c.attention(q, st["table"], cu, seq, max_new=int(max(new)))
    st["ctx"], st["n_free"] = seq, left
    if log is not None:
        log.append((k[:n], v[:n], q[:n], out[:n], np.concatenate([[0], np.cumsum(new)])))
    return out


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_serving_steps(kvq, dtype):
    """Prompts, decode steps, drafted tokens and a chunk over shared pages:
    every output against attention over the exact keys and values, whose codes
    err by half a step of E4M3 (2^-4 of a value, twice where a scale grew)."""
    rng = np.random.default_rng(11)
    st = serving_state(kvq, rng)
    log = []
    plans = [[40, 3, 0, 17, 70], [1, 1, 1, 1, 1], [1, 0, 5, 1, 2]] + [[1] * 5] * 14 + [[30, 4, 0, 1, 33]]
    hist = [[np.zeros((0, st["H"], st["D"]))] * 2 for _ in range(5)]
    for new in plans:
        step(kvq, st, rng, new, dtype, log)
        k, v, q, out, cu = log[-1]
        for b in range(5):
            if new[b] == 0:
                continue
            hist[b] = [np.concatenate([h, f64(x[cu[b]:cu[b + 1]])]) for h, x in zip(hist[b], (k, v))]
            K, V = hist[b]
            for j in (0, new[b] - 1):
                p = len(K) - new[b] + j
                for hq in range(st["H"] * st["R"]):
                    z = K[:p + 1, hq // st["R"]] @ f64(q[cu[b] + j, hq]) * st["D"] ** -0.5
                    w = np.exp(z - z.max())
                    want = (w / w.sum()) @ V[:p + 1, hq // st["R"]]
                    d = f64(out[cu[b] + j, hq]) - want
                    # values of size 1: codes err by 2^-4 at most, scores by
                    # about sqrt(D) * 2^-5 * 0.09 rms: a bound on the rms
                    assert np.sqrt((d * d).mean()) < 0.1 + 0.1 * np.abs(want).max()
    st["cache"].check()
    used = {int(x) for x in st["table"].flatten().tolist() if x >= 0}
    assert len(used) == 80 - st["n_free"].item()


def test_a_step_in_a_graph(kvq):
    """A captured decode step replayed with other lengths gives what the eager
    calls give, and eager calls in between do not disturb it."""
    rng = np.random.default_rng(12)
    st = serving_state(kvq, rng)
    step(kvq, st, rng, [40, 3, 9, 17, 70])
    c, B = st["cache"], 5
    k, v = (torch.randn(B, st["H"], st["D"], device="cuda").half() for _ in range(2))
    q = torch.randn(B, st["H"] * st["R"], st["D"], device="cuda").half()
    ctx, new, n_free = st["ctx"].clone(), ints([1] * B), st["n_free"].clone()

    def one():
        cu, seq, slots, left = c.plan(ctx, new, st["table"], st["free"], n_free, B)
        c.store(k, v, slots)
        out = c.attention(q, st["table"], cu, seq, max_new=1)
        ctx.copy_(seq)
        n_free.copy_(left)
        return out

    save = [t.clone() for t in (c.k_pages.view(torch.uint8), c.v_pages.view(torch.uint8), c.k_scale,
                                c.v_scale, st["table"], ctx, n_free)]

    def restore():
        for t, s in zip((c.k_pages.view(torch.uint8), c.v_pages.view(torch.uint8), c.k_scale, c.v_scale,
                         st["table"], ctx, n_free), save):
            t.copy_(s)

    want = []
    for _ in range(20):
        want.append(one().clone())
    restore()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = one()
    restore()
    other = simple(rng, n_pages=64, seq=(900, 40), new=(1, 1))
    plain = kvq.kvq_paged_attention(*other)
    for i in range(20):
        g.replay()
        assert torch.equal(out, want[i]), i
        assert torch.equal(kvq.kvq_paged_attention(*other), plain)
    c.check()


def test_two_graphs_at_the_same_time(kvq):
    """Graphs captured from one cache replay on two streams at once: they share
    no workspace."""
    rng = np.random.default_rng(13)
    calls = [simple(rng, n_pages=700, H=2, seq=(5000, 3000), new=(1, 1), R=4),
             simple(rng, n_pages=700, H=2, seq=(2000, 6000), new=(2, 1), R=4)]
    want = [kvq.kvq_paged_attention(*a, max_new=2) for a in calls]
    streams, graphs, outs = [torch.cuda.Stream() for _ in range(2)], [], []
    torch.cuda.synchronize()
    for a, s in zip(calls, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(3):
                o = kvq.kvq_paged_attention(*a, max_new=2)
        graphs.append(g)
        outs.append(o)
    for _ in range(30):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_outputs_are_the_streams_memory(kvq):
    """Memory freed on the current stream may still be in use there, so a call
    on another stream does not get it for its outputs."""
    a = simple(np.random.default_rng(13))
    want = kvq.kvq_paged_attention(*a)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = torch.empty_like(want)
    at = freed.data_ptr()
    del freed
    out = kvq.kvq_paged_attention(*a, stream=side)
    assert out.data_ptr() != at
    side.synchronize()
    assert torch.equal(out, want)
    ctx, new = ints([3, 20]), ints([1, 5])
    free, left = ints(range(9)), ints([9])
    tables = [torch.full((2, 4), 0, dtype=torch.int32, device="cuda") for _ in range(2)]
    here = kvq.kvq_paged_plan(ctx, new, tables[0], free, left, 16, 6)
    torch.cuda.synchronize()
    there = kvq.kvq_paged_plan(ctx, new, tables[1], free, left, 16, 6, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(here, there))
    with pytest.raises(kvq.KvqError, match="stream"):
        kvq.kvq_paged_attention(*a, stream=2)  # the per-thread default stream


def test_a_branch_of_a_captured_graph(kvq):
    """A call on a stream that a capture forked to: its output and workspace
    are the graph's, beside a call of the capture's own stream."""
    rng = np.random.default_rng(15)
    a = simple(rng, n_pages=700, H=2, seq=(5000, 3000), new=(1, 1), R=4)
    b = simple(rng, n_pages=700, H=2, seq=(4000, 1), new=(1, 1), R=4)
    want = [kvq.kvq_paged_attention(*x) for x in (a, b)]
    main, branch = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        branch.wait_stream(main)
        got = [kvq.kvq_paged_attention(*a), kvq.kvq_paged_attention(*b, stream=branch)]
        main.wait_stream(branch)
    for _ in range(20):
        for x in got:
            x.fill_(7.0)
        g.replay()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_streams_of_the_callers_choice(kvq):
    """Another stream than the current one, by object and by address, eager
    calls on two streams at once, and a workspace of the caller's."""
    rng = np.random.default_rng(14)
    a = simple(rng, n_pages=700, H=2, seq=(5000, 3000), new=(1, 1), R=4)
    want = kvq.kvq_paged_attention(*a)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(20):
        for s in (s1, s2.cuda_stream):
            o = torch.empty_like(want)
            kvq.kvq_paged_attention(*a, out=o, stream=s)
            outs.append(o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    n = kvq.kvq_paged_workspace_bytes(700, 2, 16, 64)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    assert torch.equal(kvq.kvq_paged_attention(*a, workspace=ws), want)
    assert (ws[:1024] == 0).all()
    with pytest.raises(kvq.KvqError):
        kvq.kvq_paged_attention(*a, workspace=ws[:-16])
    with pytest.raises(kvq.KvqError, match="stream"):
        kvq.kvq_paged_attention(*a, stream="x")


def test_cache_reports_what_was_flagged(kvq):
    c = kvq.PagedCache(n_pages=4, page_size=16, n_q_heads=4, n_kv_heads=2, head_dim=64)
    table = ints(np.full((1, 8), -1))
    c.plan(ints([0]), ints([100]), table, ints([0, 1, 2, 3]), ints([4]), 100)
    with pytest.raises(kvq.KvqError, match="free stack"):
        c.check()
    c.check()  # told once
    x = torch.full((1, 2, 64), float("inf"), dtype=torch.float16, device="cuda")
    c.store(x, x, ints([3]))
    with pytest.raises(kvq.KvqError, match="non-finite"):
        c.check()
    with pytest.raises(kvq.KvqError, match="4 heads"):
        c.attention(torch.zeros(1, 2, 64, dtype=torch.float16, device="cuda"), table, ints([0, 1]), ints([1]))
    with pytest.raises(kvq.KvqError):
        kvq.PagedCache(n_pages=4, page_size=16, n_q_heads=5, n_kv_heads=2, head_dim=64)
    before = kvq.kvq_launch_count()
    c.plan(ints([0]), ints([1]), table, ints([0, 1, 2, 3]), ints([4]), 1)
    assert kvq.kvq_launch_count() == before + 1


def test_nothing_to_do(kvq):
    c, s, pages, sc = make_pool(np.random.default_rng(0), 4, 2, 16, 64)
    e = torch.empty(0, 2, 64, dtype=torch.float16, device="cuda")
    kvq.kvq_paged_store(e, e, ints([]), *pages, *sc)
    out = kvq.kvq_paged_attention(torch.empty(0, 4, 64, dtype=torch.float16, device="cuda"), *pages,
                                  *sc, ints([[0]]), ints([0, 0]), ints([5]))
    assert out.shape == (0, 4, 64)
