"""Host-side checks of the paged 8-bit cache's calls (no GPU): every refusal of
the C ABI and of the Python binding happens before any device work, and the
64-bit reference of the tests agrees with itself."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import paged_ref as ref  # noqa: E402

torch = pytest.importorskip("torch")

A = 1 << 20  # an aligned address that no call may touch


@pytest.fixture(scope="module")
def kvq():
    from bit_kv_cache_11_gb300 import build
    build.build()
    from bit_kv_cache_11_gb300 import kvq as k
    return k


def pool(k, **over):
    f = dict(k_pages=A, v_pages=A, k_scale=A, v_scale=A, n_pages=8, n_kv_heads=2, page_size=16,
             head_dim=64)
    f.update(over)
    return k.kvq_paged_pool(*f.values())


def test_pool_check(kvq):
    k = kvq
    ok = lambda *a: k.kvq_paged_pool_check(*a)  # noqa: E731
    for ps in (16, 32, 64, 128):
        for d in (64, 128):
            assert ok(100, 8, ps, d) == k.KVQ_OK
    for bad in ((0, 8, 16, 64), (5, 0, 16, 64), (5, 8, 0, 64), (5, 8, 16, 0), (-1, 8, 16, 64)):
        assert ok(*bad) == k.KVQ_ERR_INVALID_ARG, bad
    for bad in ((5, 8, 8, 64), (5, 8, 256, 64), (5, 8, 48, 64), (5, 8, 16, 96), (5, 8, 16, 256),
                (1 << 24, 8, 16, 64)):
        assert ok(*bad) == k.KVQ_ERR_UNSUPPORTED, bad
    assert ok((1 << 27) - 1, 1, 16, 64) == k.KVQ_OK  # slots fit 31 bits


def test_plan_refusals(kvq):
    k = kvq
    good = dict(ctx=A, new=A + 64, batch=4, table=A, max_pages=8, free=A, n_free_pages=10,
                n_free=A, ps=16, n_tokens=9, cu=A + 128, seq=A + 192, slots=A, left=A + 256,
                err=None, stream=None)
    names = list(good)

    def call(**over):
        f = dict(good)
        f.update(over)
        return k._lib.kvq_paged_plan(*[f[n] for n in names])

    for over in (dict(batch=0), dict(batch=-3), dict(max_pages=0), dict(n_free_pages=-1),
                 dict(n_tokens=-1), dict(ps=0), dict(ctx=None), dict(new=None), dict(table=None),
                 dict(n_free=None), dict(cu=None), dict(seq=None), dict(left=None),
                 dict(slots=None), dict(slots=A + 4), dict(free=None), dict(ctx=A + 2),
                 dict(err=A + 1), dict(seq=A), dict(seq=A + 64), dict(left=A), dict(cu=A)):
        if over == dict(left=A):
            over = dict(left=A, n_free=A)
        assert call(**over) == k.KVQ_ERR_INVALID_ARG, over
    for over in (dict(ps=24), dict(ps=256), dict(batch=4097), dict(max_pages=1 << 28)):
        assert call(**over) == k.KVQ_ERR_UNSUPPORTED, over


def test_store_refusals(kvq):
    k = kvq

    def call(p=None, kk=A, v=A, dtype=0, ks=128, vs=128, slots=A, n=3, err=None):
        return k._lib.kvq_paged_store(ctypes.byref(p or pool(k)), kk, v, dtype, ks, vs, slots, n,
                                      err, None)

    assert k._lib.kvq_paged_store(None, A, A, 0, 128, 128, A, 1, None, None) == k.KVQ_ERR_INVALID_ARG
    assert call(n=0) == k.KVQ_OK
    for over in (dict(kk=None), dict(v=None), dict(kk=A + 8), dict(v=A + 2), dict(dtype=2),
                 dict(dtype=-1), dict(ks=120), dict(vs=127), dict(ks=132), dict(slots=None),
                 dict(n=-1), dict(err=A + 3), dict(p=pool(k, k_pages=None)),
                 dict(p=pool(k, v_pages=A + 8)), dict(p=pool(k, k_scale=None)),
                 dict(p=pool(k, v_scale=A + 2)), dict(p=pool(k, n_pages=0))):
        assert call(**over) == k.KVQ_ERR_INVALID_ARG, over
    assert call(p=pool(k, page_size=20)) == k.KVQ_ERR_UNSUPPORTED
    assert call(p=pool(k, n_kv_heads=70000, n_pages=1), ks=70000 * 64, vs=70000 * 64) \
        == k.KVQ_ERR_UNSUPPORTED


def test_attention_refusals(kvq):
    k = kvq
    n = ctypes.c_size_t(0)
    assert k._lib.kvq_paged_workspace_bytes(ctypes.byref(pool(k)), ctypes.byref(n)) == k.KVQ_OK
    ws = n.value
    assert ws == k.kvq_paged_workspace_bytes(8, 2, 16, 64) and ws > 1024
    assert k._lib.kvq_paged_workspace_bytes(ctypes.byref(pool(k)), None) == k.KVQ_ERR_INVALID_ARG
    good = dict(p=None, q=A, dtype=1, qs=256, out=A, os=256, n=5, heads=4, table=A, max_pages=4,
                cu=A, seq=A, batch=3, max_new=2, scale=0.1, window=0, ws=A, n_ws=ws, err=None)

    def call(**over):
        f = dict(good)
        f.update(over)
        f["p"] = ctypes.byref(f["p"] or pool(k))
        return k._lib.kvq_paged_attention(*f.values(), None)

    assert call(n=0) == k.KVQ_OK
    inf, nan = float("inf"), float("nan")
    for over in (dict(q=None), dict(out=None), dict(q=A + 8), dict(out=A + 4), dict(dtype=5),
                 dict(qs=248), dict(qs=260), dict(os=128), dict(n=-1), dict(heads=0),
                 dict(heads=5), dict(table=None), dict(max_pages=0), dict(cu=None), dict(seq=None),
                 dict(batch=0), dict(max_new=0), dict(scale=inf), dict(scale=nan), dict(window=-1),
                 dict(ws=None), dict(ws=A + 8), dict(n_ws=ws - 1), dict(err=A + 2),
                 dict(p=pool(k, k_pages=None)), dict(p=pool(k, head_dim=-64))):
        assert call(**over) == k.KVQ_ERR_INVALID_ARG, over
    for over in (dict(heads=34, qs=34 * 64, os=34 * 64),      # 17 query heads a kv head
                 dict(batch=4097), dict(max_pages=1 << 28),
                 dict(n=1 << 28, max_new=1 << 28)):           # rows beyond 2^28
        assert call(**over) == k.KVQ_ERR_UNSUPPORTED, over


def test_pool_struct_matches_the_header(kvq, tmp_path):
    k = kvq
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "l.c"
    fields = [f for f, _ in k.kvq_paged_pool._fields_]
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "kvq.h"\nint main(void) {'
                   + "".join(f'printf("%zu ", offsetof(kvq_paged_pool, {f}));' for f in fields)
                   + 'printf("%zu %d %d %d %d %d %d %d", sizeof(kvq_paged_pool), KVQ_DTYPE_FP16, '
                     'KVQ_DTYPE_BF16, KVQ_PAGED_ERR_WAIT, KVQ_PAGED_ERR_BAD_PAGE, '
                     'KVQ_PAGED_ERR_NO_PAGES, KVQ_PAGED_ERR_LENGTH, KVQ_PAGED_ERR_NONFINITE);'
                     'return 0; }\n')
    exe = tmp_path / "l"
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    want = [getattr(k.kvq_paged_pool, f).offset for f in fields] + [ctypes.sizeof(k.kvq_paged_pool)]
    want += [k.KVQ_DTYPE_FP16, k.KVQ_DTYPE_BF16, k.KVQ_PAGED_ERR_WAIT, k.KVQ_PAGED_ERR_BAD_PAGE,
             k.KVQ_PAGED_ERR_NO_PAGES, k.KVQ_PAGED_ERR_LENGTH, k.KVQ_PAGED_ERR_NONFINITE]
    assert got == want


# ---- the binding: what is wrong is said before a device is asked for ---------

def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def fp8(*s):
    return torch.zeros(*s, dtype=torch.uint8).view(torch.float8_e4m3fn)


def refused(kvq, word, fn, *a, **kw):
    with pytest.raises(kvq.KvqError, match=word) as e:
        fn(*a, **kw)
    assert e.value.status == kvq.KVQ_ERR_INVALID_ARG


def test_binding_refuses_plan_arguments(kvq):
    f = kvq.kvq_paged_plan
    ok = [i32(3), i32(3), i32(3, 4), i32(9), i32(1), 16, 5]
    refused(kvq, "CUDA device", f, *ok)
    for i, bad, word in ((0, i32(3).long(), "ctx_len"), (0, [1, 2], "must be a tensor"),
                         (1, i32(2), "new_len"), (2, i32(2, 4), "block_table"),
                         (2, i32(12), "block_table"), (2, i32(3, 8)[:, ::2], "block_table"),
                         (3, i32(9).float(), "free_pages"), (4, i32(0), "n_free"),
                         (5, 16.5, "page_size"), (6, -1, "n_tokens"), (6, 1 << 40, "n_tokens")):
        a = list(ok)
        a[i] = bad
        refused(kvq, word, f, *a)
    refused(kvq, "cu_new", f, *ok, cu_new=i32(3))
    refused(kvq, "slots", f, *ok, slots=i32(4))


def test_binding_refuses_store_arguments(kvq):
    f = kvq.kvq_paged_store
    x = torch.zeros(5, 2, 64, dtype=torch.float16)
    ok = [x, x, i32(5), fp8(7, 2, 16, 64), fp8(7, 2, 16, 64), torch.zeros(7, 2), torch.zeros(7, 2)]
    refused(kvq, "CUDA device", f, *ok)
    for i, bad, word in ((0, x.float(), "float16 or bfloat16"), (1, x.bfloat16(), "same type"),
                         (1, x[:4], "same type"), (2, i32(4), "slots"), (2, i32(5).long(), "slots"),
                         (3, torch.zeros(7, 2, 16, 64, dtype=torch.uint8), "float8_e4m3fn"),
                         (4, fp8(7, 2, 32, 64), "k_pages and v_pages"),
                         (5, torch.zeros(7, 3), "k_scale"), (6, torch.zeros(7, 2).double(), "scale")):
        a = list(ok)
        a[i] = bad
        refused(kvq, word, f, *a)
    wrong = torch.zeros(5, 3, 64, dtype=torch.float16)
    refused(kvq, r"\[tokens\]\[2\]\[64\]", f, wrong, wrong, *ok[2:])
    turned = torch.zeros(2, 5, 64, dtype=torch.float16).transpose(0, 1)
    refused(kvq, "contiguous", f, turned, turned, *ok[2:])


def test_binding_refuses_attention_arguments(kvq):
    f = kvq.kvq_paged_attention
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    ok = [q, fp8(7, 2, 16, 64), fp8(7, 2, 16, 64), torch.zeros(7, 2), torch.zeros(7, 2), i32(3, 4),
          i32(4), i32(3)]
    refused(kvq, "CUDA device", f, *ok)
    for i, bad, word in ((0, q.double(), "float16 or bfloat16"), (0, q[0], "n_q_heads"),
                         (0, torch.zeros(5, 4, 32, dtype=torch.float16), "64"),
                         (5, i32(2, 4), "block_table"), (6, i32(3), "cu_new"),
                         (7, i32(3).long(), "seq_len"), (7, i32(2), "block_table")):
        a = list(ok)
        a[i] = bad
        refused(kvq, word, f, *a)
    refused(kvq, "max_new", f, *ok, max_new=0)
    refused(kvq, "window", f, *ok, window=-1)
    refused(kvq, "softmax_scale", f, *ok, softmax_scale="x")
    refused(kvq, "out", f, *ok, out=q.half())
    refused(kvq, "out", f, *ok, out=torch.zeros(5, 64, 4, dtype=torch.bfloat16).transpose(1, 2))


def test_e4m3_table_and_rounding():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(v), np.isnan(ref.E4M3))
    assert np.array_equal(v[~np.isnan(v)], ref.E4M3[~np.isnan(v)])
    rng = np.random.default_rng(0)
    x = np.clip(rng.standard_normal(50000) * np.exp2(rng.integers(-12, 9, 50000)), -448, 448)
    mid = (ref.E4M3[:126] + ref.E4M3[1:127]) / 2  # exact ties
    x = np.concatenate([x, mid, -mid]).astype(np.float32)
    t = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_code(x), t)
