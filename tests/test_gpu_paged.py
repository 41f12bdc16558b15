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
])
def test_store(kvq, dtype, ps, D, H, runs, pad):
    rng = np.random.default_rng(ps + D + len(runs))
    n_pages = sum(n // ps + 2 for _, n in runs) + 3
    slots = slots_of(rng, runs, ps, n_pages, pad)
    T = len(slots)
    # token sizes vary over 2^12, so scales grow, stay, and reach the subnormal codes
    x = [rng.standard_normal((T, H, D)) * 2.0 ** rng.integers(-8, 4, (T, H, 1)) for _ in range(2)]
    check_store(kvq, rng, x, slots, ps, D, H, n_pages, dtype, fused=D == 128)


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
]


@pytest.mark.parametrize("case", DECODE, ids=str)
def test_decode(kvq, case):
    check_attention(kvq, case)


@pytest.mark.parametrize("case", MULTI, ids=str)
def test_several_new_tokens(kvq, case):
    check_attention(kvq, case)
