"""Host-side checks of the paged 4-bit cache's calls (no GPU): refusals, the
structs, and the reference's own arithmetic."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import paged4_ref as ref  # noqa: E402

torch = pytest.importorskip("torch")

A = 1 << 20  # an aligned address that no call may touch


@pytest.fixture(scope="module")
def kvq():
    from bit_kv_cache_11_gb300 import build
    build.build()
    from bit_kv_cache_11_gb300 import kvq as k
    return k


def pool(k, **over):
    f = dict(k_codes=A, v_codes=A, k_meta=A, v_meta=A, n_pages=8, n_kv_heads=2, page_size=16, head_dim=64)
    f.update(over)
    return k.kvq_paged4_pool(*f.values())


def test_pool_check(kvq):
    k = kvq
    ok = k.kvq_paged4_pool_check
    for ps in (16, 32, 64, 128):
        for d in (64, 128):
            assert ok(100, 8, ps, d) == k.KVQ_OK
    for bad in ((0, 8, 16, 64), (5, 0, 16, 64), (5, 8, 0, 64), (5, 8, 16, 0), (-1, 8, 16, 64)):
        assert ok(*bad) == k.KVQ_ERR_INVALID_ARG, bad
    for bad in ((5, 8, 8, 64), (5, 8, 256, 64), (5, 8, 16, 96), (5, 8, 16, 256), (1 << 24, 8, 16, 64)):
        assert ok(*bad) == k.KVQ_ERR_UNSUPPORTED, bad
    assert k._lib.kvq_paged4_pool_check(None) == k.KVQ_ERR_INVALID_ARG


def test_read_refusals(kvq):
    k = kvq

    def call(p=None, slots=A, n=3, ko=A, vo=A, err=None):
        return k._lib.kvq_paged4_read(ctypes.byref(p or pool(k)), slots, n, ko, vo, err, None)

    assert call(n=0) == k.KVQ_OK and call(ko=None, vo=None) == k.KVQ_OK
    for over in (dict(slots=None), dict(slots=A + 2), dict(n=-1), dict(ko=A + 8), dict(vo=A + 4), dict(err=A + 1),
                 dict(p=pool(k, k_codes=None)), dict(p=pool(k, v_meta=A + 8)), dict(p=pool(k, n_kv_heads=0))):
        assert call(**over) == k.KVQ_ERR_INVALID_ARG, over
    assert call(p=pool(k, page_size=20)) == k.KVQ_ERR_UNSUPPORTED
    assert k._lib.kvq_paged4_read(None, A, 3, A, A, None, None) == k.KVQ_ERR_INVALID_ARG


def test_attention_refusals(kvq):
    k = kvq
    n = ctypes.c_size_t(0)
    assert k._lib.kvq_paged4_workspace_bytes(ctypes.byref(pool(k)), ctypes.byref(n)) == k.KVQ_OK
    ws = n.value
    assert ws == k.kvq_paged4_workspace_bytes(8, 2, 16, 64) and ws > 1024
    assert k._lib.kvq_paged4_workspace_bytes(ctypes.byref(pool(k)), None) == k.KVQ_ERR_INVALID_ARG
    assert k._lib.kvq_paged4_workspace_bytes(None, ctypes.byref(n)) == k.KVQ_ERR_INVALID_ARG
    good = dict(p=None, q=A, dtype=1, qs=256, out=A, os=256, n=5, heads=4, table=A, max_pages=4, cu=A, seq=A, batch=3,
                max_new=2, scale=0.1, window=0, ws=A, n_ws=ws, err=None)

    def call(**over):
        f = dict(good)
        f.update(over)
        f["p"] = ctypes.byref(f["p"] or pool(k))
        return k._lib.kvq_paged4_attention(*f.values(), None)

    assert call(n=0) == k.KVQ_OK
    inf, nan = float("inf"), float("nan")
    for over in (dict(q=None), dict(out=None), dict(q=A + 8), dict(out=A + 4), dict(dtype=5), dict(qs=248), dict(os=128),
                 dict(n=-1), dict(heads=0), dict(heads=5), dict(table=None), dict(max_pages=0), dict(cu=None),
                 dict(seq=None), dict(batch=0), dict(max_new=0), dict(scale=inf), dict(scale=nan), dict(window=-1),
                 dict(ws=None), dict(ws=A + 8), dict(n_ws=ws - 1), dict(err=A + 2), dict(p=pool(k, k_codes=None)),
                 dict(p=pool(k, k_meta=A + 8)), dict(p=pool(k, head_dim=-64))):
        assert call(**over) == k.KVQ_ERR_INVALID_ARG, over
    for over in (dict(heads=34, qs=34 * 64, os=34 * 64), dict(batch=4097), dict(max_pages=1 << 28),
                 dict(n=1 << 28, max_new=1 << 28)):
        assert call(**over) == k.KVQ_ERR_UNSUPPORTED, over


def test_structs_match_the_header(kvq, tmp_path):
    k = kvq
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src, structs = tmp_path / "l.c", (k.kvq_paged4_pool, k.kvq_rotary)
    body = "".join(f'printf("%zu ", offsetof({s.__name__}, {f}));' for s in structs for f, _ in s._fields_)
    body += "".join(f'printf("%zu ", sizeof({s.__name__}));' for s in structs)
    src.write_text(f'#include <stddef.h>\n#include <stdio.h>\n#include "kvq.h"\nint main(void) {{{body} return 0; }}\n')
    exe = tmp_path / "l"
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    assert got == [getattr(s, f).offset for s in structs for f, _ in s._fields_] + [ctypes.sizeof(s) for s in structs]


def refused(kvq, word, fn, *a, **kw):
    with pytest.raises(kvq.KvqError, match=word) as e:
        fn(*a, **kw)
    assert e.value.status == kvq.KVQ_ERR_INVALID_ARG


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def test_binding_refuses_pools_and_arguments(kvq):
    codes, meta = torch.zeros(7, 2, 16, 32, dtype=torch.uint8), torch.zeros(7, 2, 16, 2, 2, dtype=torch.float16)
    p = [codes, codes, meta, meta]
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    f = kvq.kvq_paged4_attention
    tail = [i32(3, 4), i32(4), i32(3)]
    refused(kvq, "CUDA device", f, q, *p, *tail)
    refused(kvq, "CUDA device", kvq.kvq_paged4_read, i32(3), *p)
    for i, bad, word in ((0, codes.int(), "uint8"), (1, codes[:6], "uint8"), (0, codes[0], "uint8"),
                         (2, meta.float(), "float16"), (3, meta[..., 0], "float16"), (2, meta[:, :, :, :1], "float16")):
        bad_pool = list(p)
        bad_pool[i] = bad
        refused(kvq, word, f, q, *bad_pool, *tail)
        refused(kvq, word, kvq.kvq_paged4_read, i32(3), *bad_pool)
    refused(kvq, "64", f, torch.zeros(5, 4, 32, dtype=torch.float16), *p, *tail)
    refused(kvq, "max_new", f, q, *p, *tail, max_new=0)
    refused(kvq, "out", f, q, *p, *tail, out=q.half())
    refused(kvq, "block_table", f, q, *p, i32(2, 4), *tail[1:])
    refused(kvq, "slots", kvq.kvq_paged4_read, i32(3).long(), *p)
    with pytest.raises(kvq.KvqError):
        kvq.PagedCache4(n_pages=4, page_size=16, n_q_heads=4, n_kv_heads=2, head_dim=96, device="cpu")
    refused(kvq, "multiple", kvq.PagedCache4, 4, 16, 5, 2, 64, device="cpu")


def test_reference_codes():
    """Packing is its own inverse, words by hand, and values within half a step."""
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 16, (5, 3, 64)).astype(np.uint8)
    for key in (False, True):
        assert np.array_equal(ref.unpack(ref.pack(codes, key), key), codes)
    one = np.arange(8, dtype=np.uint8)[None]
    assert ref.pack(one, False).view("<u4")[0, 0] == 0x76543210
    assert ref.pack(one, True).view("<u4")[0, 0] == 0x75316420
    x = rng.standard_normal((50, 64)).astype(np.float16)
    c, s, m = ref.quantize(x)
    d = np.abs(ref.values(c, s, m) - x.astype(np.float64)).reshape(50, 2, 32)
    assert (d <= s.astype(np.float64)[..., None] * (0.5 + 15 * 2.0 ** -11) + 2.0 ** -10 * 4).all()
    wide = np.zeros((1, 32))
    wide[0, :2] = np.inf, -np.inf
    v = ref.values(*ref.quantize(wide))
    assert np.isfinite(v).all() and abs(v[0, 0] - ref.MOST) <= 65 and v[0, 1] == -ref.MOST
