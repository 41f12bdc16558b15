"""Host-side checks of the rotary calls and of the appends that turn (no GPU)."""
import ctypes
import os
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


def refused(kvq, word, fn, *a, **kw):
    with pytest.raises(kvq.KvqError, match=word) as e:
        fn(*a, **kw)
    assert e.value.status == kvq.KVQ_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(), dict(base=500000.0), dict(factor=8.0), dict(factor=32.0, original_len=8192.0),
                                dict(factor=8.0, original_len=8192.0, low=1.0, high=4.0), dict(base=1e6, factor=1.0)])
@pytest.mark.parametrize("dim", [2, 24, 64, 128, 256])
def test_turns(kvq, dim, kw):
    """Within float64's rounding of f / (2 pi): a few steps of 2^-53 of it."""
    got = kvq.kvq_rotary_turns(dim, device="cpu", **kw)
    assert got.dtype == torch.int64 and got.shape == (dim // 2,)
    names = dict(original_len="original")
    f = ref.frequencies(dim, **{names.get(k, k): v for k, v in kw.items()})
    for g, x in zip(got.tolist(), f):
        want = x / (2 * np.pi) * 2.0 ** 64
        assert abs(g - want) <= want * 2.0 ** -48 + 0.5
        assert 0 < g < 1 << 62
    if "factor" not in kw:
        assert got[0].item() == round(2.0 ** 64 / (2 * np.pi))


def test_scaling_by_parts_keeps_the_fast_pairs(kvq):
    plain = kvq.kvq_rotary_turns(128, device="cpu").double()
    part = kvq.kvq_rotary_turns(128, factor=8.0, original_len=4096.0, low=1.0, high=32.0, device="cpu").double()
    turns = 4096 * plain / 2.0 ** 64
    assert torch.equal(part[turns >= 32], plain[turns >= 32]) and (turns >= 32).any()
    slow = turns <= 1
    assert slow.any() and (part[slow] * 8 / plain[slow] - 1).abs().max() < 1e-12
    assert ((part <= plain) & (part >= plain / 8 * (1 - 1e-12))).all()


def test_turns_refusals(kvq):
    k = kvq
    buf = (ctypes.c_int64 * 128)()
    nan, inf = float("nan"), float("inf")

    def call(t=buf, dim=64, base=1e4, factor=1.0, original=0.0, low=1.0, high=32.0):
        return k._lib.kvq_rotary_turns(t, dim, base, factor, original, low, high)

    assert call() == k.KVQ_OK and call(dim=256) == k.KVQ_OK
    for over in (dict(t=None), dict(dim=0), dict(dim=-2), dict(dim=7), dict(base=1.0), dict(base=nan), dict(base=inf),
                 dict(factor=0.5), dict(factor=nan), dict(factor=inf), dict(original=-1.0), dict(original=nan),
                 dict(original=1.0, low=-1.0), dict(original=1.0, low=4.0, high=4.0), dict(original=1.0, high=nan)):
        assert call(**over) == k.KVQ_ERR_INVALID_ARG, over
    assert call(dim=258) == k.KVQ_ERR_UNSUPPORTED
    for dim in (0, 3, -4):
        refused(k, "rotary_dim", k.kvq_rotary_turns, dim, device="cpu")


def test_angles_refusals(kvq):
    k = kvq

    def call(pos=A, n=5, turns=A, dim=64, mag=1.0, out=A):
        return k._lib.kvq_rotary_angles(pos, n, turns, dim, mag, out, None)

    assert call(n=0, pos=None, out=None) == k.KVQ_OK
    for over in (dict(pos=None), dict(pos=A + 2), dict(n=-1), dict(turns=None), dict(turns=A + 4), dict(dim=0),
                 dict(dim=5), dict(mag=float("nan")), dict(mag=float("inf")), dict(out=None), dict(out=A + 8)):
        assert call(**over) == k.KVQ_ERR_INVALID_ARG, over
    assert call(dim=258) == k.KVQ_ERR_UNSUPPORTED


def rot(k, angles=A, dim=64, inter=0):
    return k.kvq_rotary(angles, dim, inter)


def test_rotate_refusals(kvq):
    k = kvq

    def call(r=None, x=A, dtype=0, xs=512, out=A + 4096, os=512, n=5, heads=4, D=128):
        return k._lib.kvq_rotate(ctypes.byref(r or rot(k)), x, dtype, xs, out, os, n, heads, D, None)

    assert call(n=0, x=None, out=None) == k.KVQ_OK
    assert k._lib.kvq_rotate(None, A, 0, 512, A, 512, 5, 4, 128, None) == k.KVQ_ERR_INVALID_ARG
    for over in (dict(r=rot(k, angles=None)), dict(r=rot(k, angles=A + 8)), dict(r=rot(k, dim=0)), dict(r=rot(k, dim=63)),
                 dict(r=rot(k, dim=130)), dict(r=rot(k, inter=2)), dict(x=None), dict(x=A + 8), dict(dtype=2),
                 dict(xs=504), dict(xs=516), dict(out=None), dict(out=A + 2), dict(os=511), dict(n=-1), dict(heads=0),
                 dict(D=0), dict(out=A, os=520)):
        assert call(**over) == k.KVQ_ERR_INVALID_ARG, over
    for over in (dict(D=132, xs=1024, os=1024), dict(D=264, xs=2048, os=2048)):
        assert call(**over) == k.KVQ_ERR_UNSUPPORTED, over


def pool8(k, **over):
    f = dict(k_pages=A, v_pages=A, k_scale=A, v_scale=A, n_pages=8, n_kv_heads=2, page_size=16, head_dim=64)
    f.update(over)
    return k.kvq_paged_pool(*f.values())


def pool4(k, **over):
    f = dict(k_codes=A, v_codes=A, k_meta=A, v_meta=A, n_pages=8, n_kv_heads=2, page_size=16, head_dim=64)
    f.update(over)
    return k.kvq_paged4_pool(*f.values())


@pytest.mark.parametrize("four", [False, True])
def test_append_refusals(kvq, four):
    k = kvq
    fn, make = (k._lib.kvq_paged4_append, pool4) if four else (k._lib.kvq_paged_append, pool8)
    pages, scale = ("k_codes", "v_meta") if four else ("k_pages", "v_scale")

    def call(p=None, r=0, kk=A, v=A, dtype=0, ks=128, vs=128, slots=A, n=3, q=A, qs=256, qo=A + 8192, qos=256, heads=4,
             err=None):
        return fn(ctypes.byref(p or make(k)), None if r is None else ctypes.byref(r or rot(k)), kk, v, dtype, ks, vs,
                  slots, n, q, qs, qo, qos, heads, err, None)

    assert call(n=0) == k.KVQ_OK
    assert call(n=0, q=None, qo=None, heads=0) == k.KVQ_OK
    for over in (dict(kk=None), dict(v=A + 2), dict(dtype=2), dict(ks=120), dict(vs=132), dict(slots=None), dict(n=-1),
                 dict(err=A + 3), dict(p=make(k, **{pages: None})), dict(p=make(k, **{scale: A + 2})),
                 dict(p=make(k, n_pages=0)), dict(r=rot(k, angles=None)), dict(r=rot(k, dim=66)), dict(r=rot(k, dim=1)),
                 dict(q=None), dict(qo=None), dict(heads=0), dict(heads=-1), dict(qs=248), dict(qos=260), dict(q=A + 8),
                 dict(qo=A, qos=264), dict(r=None), dict(r=rot(k, inter=-1))):
        assert call(**over) == k.KVQ_ERR_INVALID_ARG, over
    assert call(p=make(k, page_size=20)) == k.KVQ_ERR_UNSUPPORTED
    assert call(p=make(k, head_dim=96), r=rot(k), ks=192, vs=192) == k.KVQ_ERR_UNSUPPORTED
    assert call(p=make(k, n_kv_heads=70000, n_pages=1), ks=70000 * 64, vs=70000 * 64) == k.KVQ_ERR_UNSUPPORTED


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def test_binding_refuses_rotary_arguments(kvq):
    f = kvq.kvq_rotary_angles
    turns = kvq.kvq_rotary_turns(64, device="cpu")
    refused(kvq, "CUDA device", f, i32(3), turns)
    for a, word in (((i32(3).long(), turns), "positions"), (([1], turns), "positions"), ((i32(3), turns.int()), "turns"),
                    ((i32(3), turns[::2]), "turns"), ((i32(3), turns[None]), "turns"), ((i32(3), turns[:0]), "turns"),
                    ((i32(3), turns, "x"), "magnitude")):
        refused(kvq, word, f, *a)
    refused(kvq, "out", f, i32(3), turns, out=torch.zeros(3, 64))
    x, ang = torch.zeros(5, 4, 128, dtype=torch.float16), torch.zeros(5, 32, 2)
    g = kvq.kvq_rotate
    refused(kvq, "CUDA device", g, x, ang)
    for a, word in (((x.float(), ang), "float16 or bfloat16"), ((x[0], ang), "heads"), ((x, ang[:4]), "angles"),
                    ((x, ang.double()), "angles"), ((x, ang[..., 0]), "angles"), ((x, ang[:, ::2]), "angles"),
                    ((x.transpose(1, 2), ang), "contiguous")):
        refused(kvq, word, g, *a)
    refused(kvq, "out", g, x, ang, out=x.bfloat16())
    refused(kvq, "out", g, x, ang, out=torch.zeros(5, 128, 4, dtype=torch.float16).transpose(1, 2))


def fp8(*s):
    return torch.zeros(*s, dtype=torch.uint8).view(torch.float8_e4m3fn)


def test_binding_refuses_append_arguments(kvq):
    x, q, ang = torch.zeros(5, 2, 64, dtype=torch.float16), torch.zeros(5, 4, 64, dtype=torch.float16), torch.zeros(5, 32, 2)
    p8 = [fp8(7, 2, 16, 64), fp8(7, 2, 16, 64), torch.zeros(7, 2), torch.zeros(7, 2)]
    p4 = [torch.zeros(7, 2, 16, 32, dtype=torch.uint8)] * 2 + [torch.zeros(7, 2, 16, 2, 2, dtype=torch.float16)] * 2
    for f, p in ((kvq.kvq_paged_append, p8), (kvq.kvq_paged4_append, p4)):
        refused(kvq, "CUDA device", f, x, x, i32(5), *p, ang, q=q)
        for a, word in (((x, x.bfloat16(), i32(5), *p, ang), "same type"), ((x, x, i32(4), *p, ang), "slots"),
                        ((x, x, i32(5), *p, ang[:3]), "angles"), ((x, x, i32(5), *p, ang.half()), "angles"),
                        ((q, q, i32(5), *p, ang), r"\[tokens\]\[2\]\[64\]")):
            refused(kvq, word, f, *a)
        refused(kvq, "k's type", f, x, x, i32(5), *p, ang, q=q.bfloat16())
        refused(kvq, "k's type", f, x, x, i32(5), *p, ang, q=q[:4])
        refused(kvq, "q_out", f, x, x, i32(5), *p, ang, q=q, q_out=q[:4])
        refused(kvq, "q_out", f, x, x, i32(5), *p, ang, q_out=q)
    refused(kvq, "angles", kvq.kvq_paged_append, x, x, i32(5), *p8, None)
    refused(kvq, "angles", kvq.kvq_paged4_append, x, x, i32(5), *p4, q=q)


def test_binding_refuses_positions(kvq):
    ok = [i32(3), i32(3), i32(3, 4), i32(9), i32(1), 16, 5]
    refused(kvq, "positions", kvq.kvq_paged_plan, *ok, positions=i32(4))
    refused(kvq, "positions", kvq.kvq_paged_plan, *ok, positions=i32(5).long())


def test_plan_positions_refusals(kvq):
    k = kvq
    good = dict(ctx=A, new=A + 64, batch=4, table=A, max_pages=8, free=A, n_free_pages=10, n_free=A, ps=16, n_tokens=9,
                cu=A + 128, seq=A + 192, slots=A, positions=A + 512, left=A + 256, err=None, stream=None)

    def call(**over):
        return k._lib.kvq_paged_plan_positions(*{**good, **over}.values())

    for over in (dict(positions=A + 516), dict(positions=A), dict(positions=A + 64), dict(slots=A + 512), dict(batch=0),
                 dict(seq=A)):
        assert call(**over) == k.KVQ_ERR_INVALID_ARG, over
    assert call(ps=24) == k.KVQ_ERR_UNSUPPORTED
