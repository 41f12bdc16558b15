"""Rotary positions on the GPU: angles against 64 bits, turned heads bit for bit
against numpy's float32."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import paged4_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def kvq():
    from bit_kv_cache_11_gb300 import kvq as k
    return k


def ints(x):
    return torch.from_numpy(np.asarray(x).astype(np.int32)).cuda()


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


# ---------------------------------------------------------------- angles

@pytest.mark.parametrize("dim", [2, 6, 16, 64, 90, 128, 256])
@pytest.mark.parametrize("T", [1, 37, 1000])
def test_angles(kvq, dim, T):
    """An angle's rounding (2^-24 of pi / 4), the series' (a few steps of 2^-24)
    and the magnitude's: within 2^-22 of the magnitude."""
    rng = np.random.default_rng(dim + T)
    pos = rng.integers(-(1 << 31), 1 << 31, T) >> rng.integers(0, 31, T)
    turns = kvq.kvq_rotary_turns(dim, base=500000.0)
    for magnitude in (1.0, 1.37):
        got = kvq.kvq_rotary_angles(ints(pos), turns, magnitude=magnitude)
        assert got.shape == (T, dim // 2, 2) and got.dtype == torch.float32
        want = ref.angles(pos, turns.tolist(), magnitude)
        assert np.abs(got.double().cpu().numpy() - want).max() <= 2.0 ** -22 * magnitude


def test_angles_at_every_eighth(kvq):
    """Phases at and around the borders between quarters and eighths of a turn."""
    turns = [0, 1, -1, 1 << 61, (1 << 61) - 1, (1 << 61) + 1, 1 << 62, (1 << 62) - 1, (1 << 63) - 1, -(1 << 63),
             -(1 << 62), 3 << 61, -(3 << 61), (1 << 62) + (1 << 31), 7, 1 << 40]
    pos = [0, 1, -1, 2, 3, 5, 8, (1 << 31) - 1, -(1 << 31)]
    got = kvq.kvq_rotary_angles(ints(pos), torch.tensor(turns).cuda())
    assert np.abs(got.double().cpu().numpy() - ref.angles(pos, turns)).max() <= 2.0 ** -22
    assert torch.equal(got[0], torch.tensor([[1.0, 0.0]] * len(turns)).cuda())


def test_far_positions_keep_their_angle(kvq):
    """2^20 positions on, the angle is as exact as at the start: a frequency's own
    rounding is 2^-65 of a turn."""
    f = ref.frequencies(128)
    pos = np.array([(1 << 20) + 7, (1 << 24) - 1])
    got = kvq.kvq_rotary_angles(ints(pos), kvq.kvq_rotary_turns(128)).double().cpu().numpy()
    # float64's own rounding of position * f: 2^-53 of the angle, and as much of f
    slack = pos[:, None] * f * 2.0 ** -51
    want = np.stack([np.cos(pos[:, None] * f), np.sin(pos[:, None] * f)], -1)
    assert (np.abs(got - want) <= 2.0 ** -22 + slack[..., None]).all()


# ---------------------------------------------------------------- rotate

def check_rotate(kvq, T, H, D, rot, inter, dtype, pad=0, in_place=False, seed=0):
    rng = np.random.default_rng(seed + T + H + D + rot)
    x = torch.from_numpy(rng.standard_normal((T, H, D)) * np.exp2(rng.integers(-8, 9, (T, H, 1)))).to(DT[dtype])
    ang = torch.from_numpy(ref.angles(rng.integers(0, 1 << 20, T), rng.integers(-(1 << 62), 1 << 62, rot // 2),
                                      1.25)).float()
    want = torch.from_numpy(ref.rotate(x.float().numpy(), ang.numpy(), inter)).to(DT[dtype])
    buf = torch.full((T, H * D + pad), 7.0, dtype=DT[dtype], device="cuda")
    xt = buf[:, :H * D].view(T, H, D)
    xt.copy_(x)
    out = xt if in_place else None
    if pad and not in_place:
        obuf = torch.full((T, H * D + pad + 8), 7.0, dtype=DT[dtype], device="cuda")
        out = obuf[:, :H * D].view(T, H, D)
    got = kvq.kvq_rotate(xt, ang.cuda(), interleaved=inter, out=out)
    assert got is out or out is None
    assert same_bits(got.cpu(), want)
    if pad:
        assert (buf[:, H * D:] == 7.0).all()
        if not in_place:
            assert (obuf[:, H * D:] == 7.0).all() and same_bits(xt.cpu(), x)


SHAPES = [(1, 1, 64, 64), (3, 2, 128, 128), (5, 3, 128, 64), (4, 7, 80, 32), (2, 5, 96, 24), (3, 4, 64, 2),
          (2, 3, 256, 256), (7, 1, 8, 8), (6, 2, 8, 6), (5, 2, 128, 90), (3, 3, 80, 78), (33, 40, 128, 128),
          (300, 8, 64, 16), (257, 5, 96, 96), (129, 3, 128, 126)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rotate(kvq, shape, inter, dtype):
    check_rotate(kvq, *shape, inter, dtype)
    check_rotate(kvq, *shape, inter, dtype, pad=24)
    check_rotate(kvq, *shape, inter, dtype, pad=8, in_place=True)


@pytest.mark.parametrize("inter", [False, True])
def test_rotate_many_tokens(kvq, inter):
    check_rotate(kvq, 9001, 3, 128, 128, inter, "bf16")
    check_rotate(kvq, 20001, 1, 64, 32, inter, "fp16", pad=8)


def test_rotate_beyond_four_gigabytes(kvq):
    """The last of 2^31 elements and more, in place."""
    T, H, D = 132000, 128, 128
    x = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, H, D, device="cuda").bfloat16()
    ang = torch.randn(T, D // 2, 2, device="cuda")
    want = torch.from_numpy(ref.rotate(x[-3:].float().cpu().numpy(), ang[-3:].cpu().numpy(), False)).bfloat16()
    assert kvq.kvq_rotate(x, ang, out=x) is x
    assert same_bits(x[-3:].cpu(), want) and not x[:1000].any()


def test_rotate_nonfinite_stays_in_its_pair(kvq):
    x = torch.randn(4, 2, 64, device="cuda").half()
    ang = torch.randn(4, 32, 2, device="cuda")
    for inter, pair in ((False, (5, 37)), (True, (10, 11))):
        y = x.clone()
        y[1, 1, pair[0]] = float("nan")
        y[2, 0, pair[1]] = float("inf")
        a, b = kvq.kvq_rotate(x, ang, inter), kvq.kvq_rotate(y, ang, inter)
        odd = torch.zeros(4, 2, 64, dtype=torch.bool, device="cuda")
        odd[1, 1, list(pair)] = odd[2, 0, list(pair)] = True
        assert torch.equal(a[~odd], b[~odd]) and not torch.isfinite(b[odd]).any()


def test_rotary_calls_in_a_graph_and_on_streams(kvq):
    turns = kvq.kvq_rotary_turns(128)
    pos = ints([5, 70000, 3])
    x = torch.randn(3, 4, 128, device="cuda").half()
    want = kvq.kvq_rotate(x, kvq.kvq_rotary_angles(pos, turns))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = kvq.kvq_rotate(x, kvq.kvq_rotary_angles(pos, turns, stream=side), stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = kvq.kvq_rotate(x, kvq.kvq_rotary_angles(pos, turns))
    for shift in (0, 9):
        pos += shift
        g.replay()
        assert torch.equal(out, kvq.kvq_rotate(x, kvq.kvq_rotary_angles(pos, turns)))


def test_nothing_to_rotate(kvq):
    e = torch.empty(0, 4, 128, dtype=torch.float16, device="cuda")
    ang = kvq.kvq_rotary_angles(ints([]), kvq.kvq_rotary_turns(128))
    assert ang.shape == (0, 64, 2) and kvq.kvq_rotate(e, ang).shape == e.shape
