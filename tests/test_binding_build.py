"""_binding.so is built for one Python and one torch: another one rebuilds it, and never loads it."""
import os
import subprocess

import pytest
import torch

from paged_decode_attention_cache_gb300 import build, ops


@pytest.fixture
def compiler(tmp_path, monkeypatch):
    """A fake g++ that writes its output file, and the list of its calls."""
    calls = []

    def run(cmd, **_):
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(f"binary {len(calls)}")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "BINDING_ABI", str(tmp_path / "objects" / "binding.abi"), raising=False)
    return calls


def test_rebuilt_for_another_torch_or_python(compiler, monkeypatch):
    build.build_binding()
    build.build_binding()
    assert len(compiler) == 1
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    build.build_binding()
    build.build_binding()
    assert len(compiler) == 2
    import sysconfig
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cpython-399" if n == "SOABI" else real(n))
    build.build_binding()
    build.build_binding()
    assert len(compiler) == 3
    # a binary without a word on what it is for (an older build's) is rebuilt too
    os.remove(build.BINDING_ABI)
    build.build_binding()
    assert len(compiler) == 4


def test_a_binary_for_another_torch_is_not_loaded(compiler, monkeypatch):
    monkeypatch.setattr(ops, "_binding", None)
    monkeypatch.setattr(ops, "lib", lambda: None)
    build.build_binding()
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    with pytest.raises(RuntimeError, match="another Python or torch"):
        ops._calls()


def test_a_failed_build_leaves_what_was_there(compiler, monkeypatch):
    build.build_binding()
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **_: subprocess.CompletedProcess(cmd, 1, "", "no"))
    with pytest.raises(RuntimeError):
        build.build_binding(force=True)
    assert build.binding_fits() and open(build.BINDING).read() == "binary 1"
