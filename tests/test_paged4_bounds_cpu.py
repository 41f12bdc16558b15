"""The bound that the GPU tests hold the attention over 4-bit pages to is tight enough
to matter: an output that left out any 16 of its tokens, or nothing but zeros, would
break it."""
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import paged4_shares as shares  # noqa: E402
import paged_ref  # noqa: E402

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("case", paged_ref.SHARES, ids=str)
def test_sixteen_tokens_count(case):
    s = shares.shares_case(case)
    found, zeros = {}, {}

    def each(b, j, hq, parts, out, bound):
        key = b, j, hq // case[3]
        zeros[key] = max(zeros.get(key, 0.0), (np.abs(out) / bound).max())
        n = len(parts) // 16 * 16
        if n and j in (0, int(s["cu"][b + 1] - s["cu"][b]) - 1):
            lost = np.add.reduceat(parts[:n], np.arange(0, n, 16), axis=0)
            # (a group of heads is checked together: what is lost is lost to all of them)
            found[key] = np.maximum(found.get(key, 0.0), (np.abs(lost) / bound).max(1))

    shares.shares_want(s, each)
    assert found and min(x.min() for x in found.values()) > 2
    assert min(zeros.values()) > 8


@pytest.mark.parametrize("n,kernel", [(1, "decode"), (70, "prompt")])
@pytest.mark.parametrize("D", [64, 128])
def test_many_small_weights_are_seen(D, n, kernel):
    *_, out, bound = shares.one_before_many(D, n, kernel)
    assert (out > 1e-4).all() and (bound < out * 2.0 ** -4).all()


def test_codes_of_a_pool_are_its_values():
    rng = np.random.default_rng(1)
    import paged4_ref
    k, v = shares.held(rng.standard_normal((3, 2, 16, 64))), shares.held(rng.standard_normal((3, 2, 16, 64)))
    p = shares.pool(k, v)
    for i, side in enumerate((k, v)):
        meta = p[2 + i]
        assert np.array_equal(paged4_ref.values(paged4_ref.unpack(p[i], i == 0), meta[..., 0], meta[..., 1]), side[3])
