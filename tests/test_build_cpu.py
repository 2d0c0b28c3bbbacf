"""The build's steps, without compiling anything: the C library does not depend on torch or on the torch-facing
calls."""
import subprocess
import sys
import types

import pytest

from precision_dense_gemm_tiled_amd import build as b


@pytest.fixture
def steps(monkeypatch, tmp_path):
    """Commands that the build runs; each writes its output. A source named in `broken` does not compile."""
    ran, broken = [], set()

    def run(cmd, **kw):
        ran.append(cmd)
        failed = any(c.endswith(name) for name in broken for c in cmd)
        if not failed:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("built")
        if failed and kw.get("check"):
            raise subprocess.CalledProcessError(1, cmd)
        return types.SimpleNamespace(returncode=int(failed), stdout="", stderr="no")

    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setattr(b, "ROOT", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libmpgemm.so"))
    monkeypatch.setattr(b, "CALLS", str(tmp_path / "_torch_calls.so"))
    return types.SimpleNamespace(ran=ran, broken=broken, lib=tmp_path / "libmpgemm.so", calls=tmp_path / "_torch_calls.so")


def test_both(steps):
    assert b.build() == str(steps.lib)
    assert steps.lib.exists() and steps.calls.exists()
    linked = [c for c in steps.ran if "-shared" in c]
    assert len(linked) == 2 and not any("torch" in a for a in linked[0])   # the library, and before the calls


def test_without_torch(steps, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)   # import torch fails
    assert b.build() == str(steps.lib)
    assert steps.lib.exists() and not steps.calls.exists()
    assert "torch" in capsys.readouterr().err
    assert not any(a.endswith(b.TORCH_SOURCE) for c in steps.ran for a in c)


def test_calls_that_do_not_compile(steps):
    steps.broken.add(b.TORCH_SOURCE)
    with pytest.raises(RuntimeError, match=b.TORCH_SOURCE):
        b.build()
    assert steps.lib.exists() and not steps.calls.exists()


def test_a_library_source_that_does_not_compile(steps):
    steps.broken.add("newton_schulz.hip")
    with pytest.raises(RuntimeError, match="newton_schulz.hip"):
        b.build()
    assert not steps.lib.exists() and not steps.calls.exists()
