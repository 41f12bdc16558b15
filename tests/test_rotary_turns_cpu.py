"""The held frequencies against 60 digits (no GPU)."""
import decimal
import os
import sys
from decimal import Decimal as D

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

torch = pytest.importorskip("torch")

PI = D("3.14159265358979323846264338327950288419716939937510582097494459")
DEFAULT = dict(base=10000.0, factor=1.0, original_len=0.0, low=1.0, high=32.0)


@pytest.fixture(scope="module")
def kvq():
    from bit_kv_cache_11_gb300 import build
    build.build()
    from bit_kv_cache_11_gb300 import kvq as k
    return k


@pytest.mark.parametrize("dim", [2, 6, 24, 64, 90, 128, 256])
@pytest.mark.parametrize("kw", [dict(), dict(base=500000.0), dict(base=1e6), dict(base=1.5), dict(factor=8.0),
                                dict(factor=32.0, original_len=8192.0),
                                dict(base=5e5, factor=8.0, original_len=8192.0, low=1.0, high=4.0),
                                dict(factor=7.3, original_len=100.0, low=0.7, high=1.4),
                                dict(factor=40.0, original_len=6.0, low=0.0, high=1.0)], ids=str)
def test_turns_within_their_bound(kvq, kw, dim):
    """Relative roundings with u = 2^-53: pow 2u (one unit in the last place), 2 pi's double
    0.35u, each operation u.  A plain f / factor / (2 pi) has 2 + 1 + 1.35 = 4.35u, of at
    most 1 / (2 pi) = 0.16 of a turn: below 2^-53.  By parts, r = original_len f / (2 pi)
    has 4.35u; keep = (r - low) / (high - low) between its ends, r <= high <= 2 (high -
    low), is off by 4.35u * 2 + u + 2u = 11.7u, f keep + f / factor (1 - keep) by those of
    f, the 2u of f and at most four operations, 17.7u, and with the division by 2 pi 19.1u
    of 0.16: below 2^-51."""
    got = kvq.kvq_rotary_turns(dim, device="cpu", **kw).tolist()
    p = {k: D(v) for k, v in {**DEFAULT, **kw}.items()}
    with decimal.localcontext() as c:
        c.prec = 60
        ratio = (-D(2) / D(dim) * p["base"].ln()).exp()
        for i, g in enumerate(got):
            f = ratio ** i
            keep = D(0)
            if p["original_len"]:
                keep = min(D(1), max(D(0), (p["original_len"] * f / (2 * PI) - p["low"]) / (p["high"] - p["low"])))
            f = f * keep + f / p["factor"] * (1 - keep)
            off = abs(D(g) / D(2) ** 64 - f / (2 * PI))
            assert off <= D(2) ** (-51 if p["original_len"] else -53), (i, float(off))
