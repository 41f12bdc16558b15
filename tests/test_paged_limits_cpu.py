"""Limits of the paged calls, refused on the host before any device work."""
import ctypes

import pytest

pytest.importorskip("torch")

A = 1 << 20  # an aligned address that no call may touch


@pytest.fixture(scope="module")
def kvq():
    from bit_kv_cache_11_gb300 import build
    build.build()
    from bit_kv_cache_11_gb300 import kvq as k
    return k


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
def test_positions_stay_inside_31_bits(kvq, ps):
    """A table whose last tokens lie within a batch of tiles of 2^31 is refused: positions
    behind them would wrap."""
    pool = kvq.kvq_paged_pool(A, A, A, A, 8, 2, ps, 64)
    n = kvq.kvq_paged_workspace_bytes(8, 2, ps, 64)
    for pages in ((1 << 31) // ps - 1, (1 << 31) // ps - 4096 // ps + 1):
        got = kvq._lib.kvq_paged_attention(ctypes.byref(pool), A, 0, 256, A, 256, 5, 4, A, pages, A, A, 3, 2,
                                           0.1, 0, A, n, None, None)
        assert got == kvq.KVQ_ERR_UNSUPPORTED, pages
