"""What build() makes where torch or the host compiler's part is missing (compilers are faked: nothing is compiled)."""
import importlib.util
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def build(monkeypatch, tmp_path):
    """The build module by itself, its outputs in tmp_path; `commands` collects what it runs, `fails` names a program that fails."""
    spec = importlib.util.spec_from_file_location("build_alone", os.path.join(ROOT, "block_sparse_gqa_causal_gb300", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    for name, at in (("BUILD", "o"), ("LIB", "libmsa.so"), ("BINDING", "_paged_binding.so")):
        monkeypatch.setattr(mod, name, str(tmp_path / at))
    monkeypatch.setattr(mod, "nvcc", lambda: "/fake/bin/nvcc")
    monkeypatch.setenv("CXX", "/fake/bin/g++")
    mod.commands, mod.fails = [], None

    def run(cmd, **kw):
        mod.commands.append(cmd)
        bad = mod.fails == os.path.basename(cmd[0])
        if not bad:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, int(bad), "", "")

    monkeypatch.setattr(mod.subprocess, "run", run)
    return mod


def test_the_library_is_built_without_torch(build, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)                  # import torch raises
    assert build.build() == build.LIB and os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert {os.path.basename(c[0]) for c in build.commands} == {"nvcc"} and len(build.commands) == len(build.sources()) + 1


def test_the_library_is_there_when_the_binding_fails(build):
    pytest.importorskip("torch")
    build.fails = "g++"
    with pytest.raises(RuntimeError, match=r"g\+\+ failed"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


def test_the_binding_follows_the_library(build):
    pytest.importorskip("torch")
    build.build()
    assert os.path.exists(build.LIB) and os.path.exists(build.BINDING)
    assert os.path.basename(build.commands[-1][0]) == "g++" and build.LIB in build.commands[-1]
    n = len(build.commands)
    build.build()
    assert len(build.commands) == n                                  # nothing is stale
    build.fails = "nvcc"
    os.remove(os.path.join(build.BUILD, "warmup.o"))
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.build()
