"""What a build compiles: the library without torch, the binding when what it is
compiled against has changed."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_library_builds_without_torch():
    code = ("import sys; sys.modules['torch'] = None\n"
            "from bit_kv_cache_11_gb300 import build, kvq\n"
            "print(build.build(), kvq.kvq_launch_count())")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split()[0].endswith("libkvq.so")


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """build.build() over a folder of its own, with compilers that only touch their
    output; returns what each build ran, by the name of its output."""
    torch = pytest.importorskip("torch")
    from bit_kv_cache_11_gb300 import build as b
    ran = []

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        ran.append(os.path.basename(out).split(".tmp")[0])
        open(out, "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b.subprocess, "run", run)
    for name, value in (("OBJ", "_build"), ("LIB", "libkvq.so"), ("BIND", "_paged_bind.so")):
        monkeypatch.setattr(b, name, str(tmp_path / value))

    def built():
        del ran[:]
        b.build()
        return sorted(ran)

    return b, torch, built


def test_the_binding_follows_torch_and_its_flags(fake, monkeypatch):
    b, torch, built = fake
    binding = ["_paged_bind.so", "paged_bind.o"]
    first = built()
    assert set(binding) < set(first) and "libkvq.so" in first
    assert built() == []
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    assert built() == binding
    assert built() == []
    monkeypatch.setattr(b, "CXX", "other-g++")
    assert built() == binding
    os.remove(b.BIND)
    assert built() == binding
    assert built() == []
