"""Stores whose runs begin beside one another, so that one warp stores a whole run:
runs of one token and up to a page, around the 32 whose slots a warp reads at once."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import paged4_ref  # noqa: E402
import paged_ref  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def ints(x):
    return torch.from_numpy(np.asarray(x).astype(np.int32)).cuda()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("lead", [0, 5, 7])
@pytest.mark.parametrize("ps,D,H", [(128, 128, 2), (128, 64, 1), (64, 128, 3), (32, 64, 2), (16, 64, 4)])
def test_runs_of_every_length(ps, D, H, lead, dtype):
    """`lead` single tokens move the runs within the store's chunks of eight tokens; a
    token without a slot and a run at the last token are among them."""
    from bit_kv_cache_11_gb300 import kvq
    rng = np.random.default_rng(ps + D + lead)
    lengths = [1] * lead + [n for n in (31, 1, 32, 1, 1, 33, 2, 34, 1, 63, 1, 64, 1, 65, 1, 127, 1, 128) if n <= ps]
    n_pages = len(lengths) + 3
    ids = rng.permutation(n_pages)
    slots = []
    for i, n in enumerate(lengths):
        row = int(rng.integers(0, ps - n + 1))
        slots += list(ids[i] * ps + row + np.arange(n)) + [-1] * (i == lead + 2)
    T = len(slots)
    x = [torch.from_numpy(rng.standard_normal((T, H, D)) * np.exp2(rng.integers(-6, 7, (T, 1, 1)))).to(DT[dtype])
         for _ in range(2)]
    codes = [paged_ref.e4m3_code(rng.standard_normal((n_pages, H, ps, D)) * 100) for _ in range(2)]
    scale = [2.0 ** rng.integers(-9, -5, (n_pages, H)).astype(np.float64) for _ in range(2)]
    ang = torch.from_numpy(paged4_ref.angles(rng.integers(0, 1 << 20, T), rng.integers(-(1 << 62), 1 << 62, D // 2))).float()
    for turn in (False, True):
        pool = ([torch.from_numpy(c).cuda().view(torch.float8_e4m3fn) for c in codes] +
                [torch.from_numpy(s.astype(np.float32)).cuda() for s in scale])
        err = ints([0])
        args = (x[0].cuda(), x[1].cuda(), ints(slots), *pool)
        if turn:
            kvq.kvq_paged_append(*args, ang.cuda(), error=err)
        else:
            kvq.kvq_paged_store(*args, error=err)
        assert err.item() == 0
        for i in range(2):
            y = x[i]
            if turn and i == 0:
                y = torch.from_numpy(paged4_ref.rotate(y.float().numpy(), ang.numpy(), False)).to(DT[dtype])
            c, s = paged_ref.store(y.double().numpy(), np.array(slots), codes[i], scale[i], ps)
            assert np.array_equal(pool[i].view(torch.uint8).cpu().numpy() & 0x7f, c & 0x7f)
            assert np.array_equal(pool[i].view(torch.uint8).cpu().numpy()[c & 0x7f != 0], c[c & 0x7f != 0])
            assert np.array_equal(pool[2 + i].double().cpu().numpy(), s)
