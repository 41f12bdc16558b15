"""The paged store's whole chunks (calls of many tokens x heads) at the inputs where
a code can go wrong, and keys and values of different strides."""
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import paged_ref as ref  # noqa: E402

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def kvq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_kv_cache_11_gb300 import kvq as k
    return k


def ints(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def check(kvq, x, slots, ps, n_pages, dtype, strides=(0, 0), flags=0):
    """x: keys and values [T][H][D] in float64; strides: elements between tokens beyond
    their own."""
    rng = np.random.default_rng(n_pages)
    T, H, D = x[0].shape
    codes = [rng.integers(0, 256, (n_pages, H, ps, D)).astype(np.uint8) for _ in range(2)]
    for c in codes:
        c[(c & 127) == 127] = 0
    scale = [2.0 ** rng.integers(-9, -3, (n_pages, H)).astype(np.float64) for _ in range(2)]
    pages = [torch.from_numpy(c).cuda().view(torch.float8_e4m3fn) for c in codes]
    sc = [torch.from_numpy(s.astype(np.float32)).cuda() for s in scale]
    t = [torch.from_numpy(v).to(DT[dtype]) for v in x]
    dev = []
    for v, more in zip(t, strides):
        buf = torch.full((T, H * D + more), float("nan"), dtype=DT[dtype], device="cuda")
        buf[:, :H * D] = v.reshape(T, -1).cuda()
        dev.append(buf[:, :H * D].view(T, H, D))
    err = ints([0])
    kvq.kvq_paged_store(*dev, ints(slots), *pages, *sc, error=err)
    assert err.item() == flags
    for i in range(2):
        want, ws = ref.store(t[i].double().numpy(), slots, codes[i], scale[i], ps)
        assert np.array_equal(sc[i].cpu().numpy().astype(np.float64), ws)
        got = pages[i].view(torch.uint8).cpu().numpy()
        same = (got == want) | ((got & 127) == 0) & ((want & 127) == 0)  # -0 is 0
        assert same.all(), np.argwhere(~same)[:5]


def run_slots(first, n, ps, n_pages, seed=0):
    """Slots of one run of n tokens from row `first` of a page on."""
    ids = np.random.default_rng(seed).permutation(n_pages)
    pos = first + np.arange(n)
    return ids[pos // ps] * ps + pos % ps


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("ps,D", [(16, 64), (32, 64), (64, 64), (128, 64), (16, 128), (64, 128), (128, 128)])
def test_whole_chunks_with_nonfinite_and_extreme_values(kvq, ps, D, dtype):
    rng = np.random.default_rng(ps + D)
    T, H = 1300, 16  # 20800 token heads
    x = [rng.standard_normal((T, H, D)) * 2.0 ** rng.integers(-8, 4, (T, H, 1)) for _ in range(2)]
    x[0][1, 0, 3], x[0][70, 1, 9], x[0][T - 1, 2, 0] = np.inf, -np.inf, np.nan
    x[1][300, 3], x[1][301:340, 4] = np.nan, np.inf
    x[0][:, 5] = 0.0
    x[0][:, 6] = 448.0 * 2.0 ** -3
    x[1][:, 6] = 448.25
    x[1][:, 7] = np.resize(ref.E4M3[1:126] + np.diff(ref.E4M3[:127])[1:] / 2, D)  # halfway
    x[0][:, 8, ::2] = 65504.0
    x[0][:, 9] = 0.0
    x[0][:, 9, 5], x[0][:, 9, 6] = 2.0 ** -24, -(2.0 ** -25)
    if dtype == "bf16":
        x[0][:, 10, 3], x[0][:, 11, 7], x[1][:, 11, 9] = 1e30, 3e38, 1e-38
    check(kvq, x, run_slots(7, T, ps, T // ps + 4), ps, T // ps + 4, dtype, strides=(8, 8),
          flags=kvq.KVQ_PAGED_ERR_NONFINITE)


@pytest.mark.parametrize("T,H", [(5, 2), (1300, 16)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_keys_and_values_of_different_strides(kvq, T, H, dtype):
    rng = np.random.default_rng(T)
    x = [rng.standard_normal((T, H, 64)) for _ in range(2)]
    for strides in ((0, 72), (128, 0), (8, 1024)):
        check(kvq, x, run_slots(3, T, 32, T // 32 + 4), 32, T // 32 + 4, dtype, strides=strides)
