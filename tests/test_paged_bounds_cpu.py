"""The bound that the GPU tests hold the paged attention to (tests/paged_ref.py)
is tight enough to matter: an output that left out any 16 of its tokens would
break it, whatever the kernel's own error within the bound."""
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import paged_ref as ref  # noqa: E402

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("case", ref.SHARES, ids=str)
def test_sixteen_tokens_count(case):
    s = ref.shares_case(case)
    found = {}

    def each(b, j, hq, parts, out, bound):
        n = len(parts) // 16 * 16
        if n and j in (0, int(s["cu"][b + 1] - s["cu"][b]) - 1):
            lost = np.add.reduceat(parts[:n], np.arange(0, n, 16), axis=0)
            # (a group of heads is checked together: what is lost is lost to all of them)
            key = b, j, hq // case[3]
            found[key] = np.maximum(found.get(key, 0.0), (np.abs(lost) / bound).max(1))

    ref.shares_want(s, each)
    assert found and min(x.min() for x in found.values()) > 2
