"""Host-side limits of the rotary calls and of the appends: arrays that overlap,
sizes at the ends of their ranges (no GPU)."""
import ctypes
import os
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

A = 1 << 20  # an aligned address that no call may touch


@pytest.fixture(scope="module")
def kvq():
    from bit_kv_cache_11_gb300 import build
    build.build()
    from bit_kv_cache_11_gb300 import kvq as k
    return k


# the arrays of a plan and their elements, each in a place of its own
PLAN = dict(ctx=(A, 4), new=(A + 1024, 4), table=(A + 2048, 4 * 8), free=(A + 4096, 10), n_free=(A + 5120, 1),
            cu=(A + 6144, 5), seq=(A + 7168, 4), slots=(A + 8192, 9), left=(A + 9216, 1), err=(A + 10240, 1))


@pytest.mark.parametrize("name", PLAN)
def test_positions_overlap_no_array_of_the_plan(kvq, name):
    """Positions are 9 elements at a multiple of 16 bytes: at an array's start, and
    where only the last of one and the first of the other meet."""
    at = {k: v[0] for k, v in PLAN.items()}

    def call(positions, ps=16):
        return kvq._lib.kvq_paged_plan_positions(
            at["ctx"], at["new"], 4, at["table"], 8, at["free"], 10, at["n_free"], ps, 9, at["cu"], at["seq"],
            at["slots"], positions, at["left"], at["err"], None)

    start, n = PLAN[name]
    last = (start + 4 * (n - 1)) & ~15
    for bad in (start, last, start - 32):  # (start - 32: elements -8 .. 0)
        assert call(bad) == kvq.KVQ_ERR_INVALID_ARG, bad - start
    # beside it: nothing is refused before the page size is looked at
    for good in (start - 48, (start + 4 * n + 15) & ~15):
        assert call(good, ps=24) == kvq.KVQ_ERR_UNSUPPORTED, good - start


def test_grids_of_every_token_count(tmp_path):
    """Token counts up to 2^31 - 1, on the host code that sizes the launches."""
    nvcc = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
    if not (os.path.exists(nvcc) or shutil.which("nvcc")):
        pytest.skip("no nvcc")
    exe = tmp_path / "grid_check"
    subprocess.check_call([nvcc, "-std=c++17", "-O1", "-I", os.path.join(ROOT, "bit_kv_cache_11_gb300", "csrc"),
                           "-I", os.path.join(ROOT, "include"),
                           os.path.join(ROOT, "tests", "harness", "grid_check.cu"), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout + out.stderr
    assert "failures 0" in out.stdout


def test_token_counts_that_no_launch_takes(kvq):
    k = kvq
    r = k.kvq_rotary(A, 64, 0)
    sizes = dict(n_pages=8, n_kv_heads=2, page_size=16, head_dim=64)
    p8 = k.kvq_paged_pool(A, A, A, A, *sizes.values())
    p4 = k.kvq_paged4_pool(A, A, A, A, *sizes.values())
    ref = ctypes.byref
    most = (1 << 31) - 1
    assert k._lib.kvq_paged_store(ref(p8), A, A, 0, 128, 128, A, most, None, None) == k.KVQ_ERR_UNSUPPORTED
    for q in ((None, 0, None, 0, 0), (A, 256, A + 8192, 256, 4)):
        args = (ref(r), A, A, 0, 128, 128, A, most, *q, None, None)
        assert k._lib.kvq_paged_append(ref(p8), *args) == k.KVQ_ERR_UNSUPPORTED
        if q[0]:
            assert k._lib.kvq_paged4_append(ref(p4), *args) == k.KVQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("dim,status", [(258, "UNSUPPORTED"), ((1 << 31) + 2, "UNSUPPORTED"), ((1 << 32) + 64, "UNSUPPORTED"),
                                        (1 << 70, "UNSUPPORTED"), (64.5, "INVALID_ARG"), (float("nan"), "INVALID_ARG"),
                                        (float("inf"), "INVALID_ARG"), (None, "INVALID_ARG"), ("64", "INVALID_ARG")])
def test_rotary_dims_that_no_call_takes(kvq, dim, status):
    """Looked at before anything is allocated or cut to 32 bits."""
    with pytest.raises(kvq.KvqError, match="rotary_dim") as e:
        kvq.kvq_rotary_turns(dim, device="cpu")
    assert e.value.status == getattr(kvq, f"KVQ_ERR_{status}")


def test_rotary_dims_that_are_taken(kvq):
    assert kvq.kvq_rotary_turns(256, device="cpu").shape == (128,)
    assert torch.equal(kvq.kvq_rotary_turns(64.0, device="cpu"), kvq.kvq_rotary_turns(64, device="cpu"))


@pytest.mark.parametrize("at", range(4))
def test_pool_sizes_beyond_32_bits(kvq, at):
    """No size is cut to its low 32 bits, neither where a pool is checked nor made."""
    good = [8, 2, 16, 64]
    for check, nbytes, cache in ((kvq.kvq_paged_pool_check, kvq.kvq_paged_workspace_bytes, kvq.PagedCache),
                                 (kvq.kvq_paged4_pool_check, kvq.kvq_paged4_workspace_bytes, kvq.PagedCache4)):
        assert check(*good) == kvq.KVQ_OK and nbytes(*good) > 1024
        for beyond in (1 << 32, 1 << 70):
            bad = list(good)
            bad[at] += beyond
            assert check(*bad) == kvq.KVQ_ERR_UNSUPPORTED
            bad[at] = good[at] - beyond
            assert check(*bad) == kvq.KVQ_ERR_INVALID_ARG
            bad[at] = good[at] + beyond
            for call in (lambda: nbytes(*bad), lambda: cache(bad[0], bad[2], 2 * bad[1], bad[1], bad[3], device="cpu")):
                with pytest.raises(kvq.KvqError) as e:
                    call()
                assert e.value.status == kvq.KVQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("cls", ["PagedCache", "PagedCache4"])
def test_check_names_its_class(kvq, monkeypatch, cls):
    monkeypatch.setattr(torch.cuda, "synchronize", lambda *a: None)
    c = getattr(kvq, cls)(8, 16, 4, 2, 64, device="cpu")
    c.check()
    c.error.fill_(kvq.KVQ_PAGED_ERR_BAD_PAGE)
    with pytest.raises(kvq.KvqError, match=rf"{cls}\.check: a page id outside the pool"):
        c.check()
    c.check()
