"""Rotary calls of the most tokens a call can have."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import paged4_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


def test_angles_and_heads_of_two_to_the_31_tokens():
    """2^31 - 1 tokens, 60 GB: one pair of channels of one head of eight, in place."""
    from bit_kv_cache_11_gb300 import kvq
    T = (1 << 31) - 1
    if torch.cuda.mem_get_info()[0] < 80e9:
        pytest.skip("less than 80 GB of device memory are free")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    turns = torch.tensor([0x123456789ABCDEF], device="cuda")
    ang = kvq.kvq_rotary_angles(pos, turns)
    parts = [slice(a, a + 700) for a in (0, 1000, (1 << 30) - 300, T - 1400, T - 700)]
    for s in parts:
        want = torch.from_numpy(ref.angles(pos[s].tolist(), turns.tolist()))
        assert (ang[s].double().cpu() - want).abs().max() <= 2.0 ** -22
    del pos
    x = torch.empty(T, 1, 8, dtype=torch.bfloat16, device="cuda")
    step = 1 << 28
    for a in range(0, T, step):
        x[a:a + step].normal_()
    before = [x[s].clone() for s in parts]
    assert kvq.kvq_rotate(x, ang, out=x) is x
    for s, b in zip(parts, before):
        want = torch.from_numpy(ref.rotate(b.float().cpu().numpy(), ang[s].cpu().numpy(), False)).bfloat16()
        assert torch.equal(x[s].cpu().view(torch.int16), want.view(torch.int16))
