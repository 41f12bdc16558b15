"""The append that turns keys and queries, into E4M3 pages: the same bits as
turning first and storing then."""
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


@pytest.fixture(scope="module")
def kvq():
    from bit_kv_cache_11_gb300 import kvq as k
    return k


def ints(x):
    return torch.from_numpy(np.asarray(x).astype(np.int32)).cuda()


def check(kvq, rng, slots, ps, D, H, n_pages, dtype, rot, inter, q_heads, in_place=False, amp=None, flags=0):
    """Against kvq_rotate and kvq_paged_store, and for small calls against numpy."""
    T = len(slots)
    fused = torch.from_numpy(rng.standard_normal((T, q_heads + 2 * H, D))).to(DT[dtype])
    if amp is not None:
        fused = (fused.double() * torch.from_numpy(amp)[:, None, None]).to(DT[dtype])
    gpu = fused.cuda()
    q, k, v = gpu[:, :q_heads], gpu[:, q_heads:q_heads + H], gpu[:, q_heads + H:]
    ang = torch.from_numpy(ref.angles(rng.integers(0, 1 << 20, T), rng.integers(-(1 << 62), 1 << 62, rot // 2))).float()
    codes = [paged_ref.e4m3_code(rng.standard_normal((n_pages, H, ps, D)) * 100) for _ in range(2)]
    scale = [2.0 ** rng.integers(-9, -5, (n_pages, H)).astype(np.float64) for _ in range(2)]

    def pool():
        return ([torch.from_numpy(c).cuda().view(torch.float8_e4m3fn) for c in codes] +
                [torch.from_numpy(s.astype(np.float32)).cuda() for s in scale])

    one, two, err, err2 = pool(), pool(), ints([0]), ints([0])
    tk, tq = kvq.kvq_rotate(k, ang.cuda(), inter), kvq.kvq_rotate(q, ang.cuda(), inter) if q_heads else None
    kvq.kvq_paged_store(tk, v, ints(slots), *two, error=err2)
    kw = dict(q=q, **(dict(q_out=q) if in_place else {})) if q_heads else {}
    got = kvq.kvq_paged_append(k, v, ints(slots), *one, ang.cuda(), inter, error=err, **kw)
    if q_heads:
        assert torch.equal(got.contiguous().view(torch.int16), tq.view(torch.int16))
        assert (got is q) == in_place
    else:
        assert got is None
    assert torch.equal(gpu[:, q_heads:].cpu().view(torch.int16), fused[:, q_heads:].contiguous().view(torch.int16))
    assert err.item() == err2.item() == flags
    for a, b in zip(one, two):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    if T <= 200 and not flags:
        x = [torch.from_numpy(ref.rotate(fused[:, q_heads:q_heads + H].float().numpy(), ang.numpy(), inter)).to(DT[dtype]),
             fused[:, q_heads + H:]]
        for i in range(2):
            c, s = paged_ref.store(x[i].double().numpy(), slots, codes[i], scale[i], ps)
            assert np.array_equal(one[i].view(torch.uint8).cpu().numpy() & 0x7f, c & 0x7f)
            assert np.array_equal(one[2 + i].double().cpu().numpy(), s)


def runs(rng, lengths, ps, n_pages, pad=0):
    """Slots of runs of tokens that begin anywhere in pages of their own."""
    ids, slots = list(rng.permutation(n_pages)), []
    for n in lengths:
        pos = int(rng.integers(0, ps))
        page = ids.pop()
        for _ in range(n):
            if pos == ps:
                pos, page = 0, ids.pop()
            slots.append(page * ps + pos)
            pos += 1
    return np.array(slots + [-1] * pad)


# page size, head_dim, kv heads, lengths of runs, rows without a slot, rotary_dim, interleaved, query heads
CASES = [
    (16, 64, 1, [1], 0, 64, False, 1), (64, 128, 8, [1] * 40, 3, 128, False, 32), (64, 128, 2, [5] * 9, 0, 128, True, 8),
    (16, 64, 3, [100, 7, 1], 2, 64, True, 3), (128, 128, 1, [300, 50], 0, 128, False, 4),
    (32, 128, 2, [700], 5, 64, False, 0), (32, 64, 5, [64, 33, 1, 1, 90], 0, 16, True, 10),
    (64, 64, 2, [3] * 30, 0, 24, False, 2), (128, 64, 1, [400], 1, 62, True, 5), (16, 128, 2, [129], 0, 2, False, 2),
    (64, 128, 8, [1500, 700], 9, 128, False, 16), (16, 64, 8, [2000], 0, 32, False, 8), (64, 128, 12, [900], 0, 90, False, 12),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_append(kvq, case, dtype):
    ps, D, H, lengths, pad, rot, inter, q_heads = case
    rng = np.random.default_rng(sum(lengths) + ps + D + rot)
    n_pages = sum(-(-n // ps) + 1 for n in lengths) + 2
    slots = runs(rng, lengths, ps, n_pages, pad)
    check(kvq, rng, slots, ps, D, H, n_pages, dtype, rot, inter, q_heads)
    check(kvq, rng, slots, ps, D, H, n_pages, dtype, rot, inter, q_heads, in_place=True)


@pytest.mark.parametrize("T", [3, 1200])
def test_sizes_of_every_kind_and_nonfinite_values(kvq, T):
    rng = np.random.default_rng(T)
    amp = np.exp2(rng.integers(-20, 14, T).astype(np.float64))
    slots = runs(rng, [T], 64, T // 64 + 3)
    check(kvq, rng, slots, 64, 128, 4, T // 64 + 3, "bf16", 128, False, 4, amp=amp)
    amp[1] = np.inf
    check(kvq, rng, slots, 64, 128, 4, T // 64 + 3, "bf16", 128, False, 4, amp=amp, flags=16)
    check(kvq, rng, slots, 64, 128, 4, T // 64 + 3, "fp16", 96, True, 0, amp=amp, flags=16)


def test_slots_outside_the_pool(kvq):
    rng = np.random.default_rng(0)
    slots = np.arange(50)
    # (the ends of runs: a page's rows have to follow one another without a gap)
    slots[[0, 49]] = 4 * 16, (1 << 31) - 1
    check(kvq, rng, slots, 16, 64, 2, 4, "fp16", 64, False, 2, flags=2)
