"""What the build step does without torch or a host compiler, and when the Python binding is stale (CPU;
compilers are stand-ins)."""
import os
import sys
import types

import pytest


@pytest.fixture
def build_lib(tmp_path, monkeypatch):
    import importlib.util

    import block_sparse_attention_sa2_gb300.build_lib as real
    spec = importlib.util.spec_from_file_location("build_lib_under_test", real.__file__)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    for name, file in (("LIB", "libsa2.so"), ("BINDING", "_cross.so"), ("BUILD", "_build")):
        monkeypatch.setattr(m, name, str(tmp_path / file))
    if hasattr(m, "BINDING_FOR"):
        monkeypatch.setattr(m, "BINDING_FOR", str(tmp_path / "_build" / "_cross.for"))
    runs = []

    def run(cmd, **kw):
        runs.append(cmd)
        if cmd[0] == "g++" and m.no_host_compiler:
            raise FileNotFoundError("g++")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(m.subprocess, "run", run)
    m.runs, m.no_host_compiler = runs, False
    return m


def test_without_torch_the_library_alone_is_built(build_lib, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch fails
    assert not build_lib.up_to_date()
    assert build_lib.build() == build_lib.LIB
    assert os.path.exists(build_lib.LIB) and not os.path.exists(build_lib.BINDING)
    assert not any(c[0] == "g++" for c in build_lib.runs) and build_lib.up_to_date()
    n = len(build_lib.runs)
    build_lib.build()
    assert len(build_lib.runs) == n


def test_without_a_host_compiler_the_library_is_there(build_lib):
    pytest.importorskip("torch")
    build_lib.no_host_compiler = True
    with pytest.raises(FileNotFoundError):
        build_lib.build()
    assert os.path.exists(build_lib.LIB) and not os.path.exists(build_lib.BINDING) and not build_lib.up_to_date()
    build_lib.no_host_compiler = False
    build_lib.build()
    assert os.path.exists(build_lib.BINDING) and build_lib.up_to_date()


@pytest.mark.parametrize("change", ["torch", "python", "unknown"])
def test_a_binding_for_another_torch_or_python_is_stale(build_lib, monkeypatch, change):
    torch = pytest.importorskip("torch")
    build_lib.build()
    assert build_lib.up_to_date()
    if change == "torch":
        monkeypatch.setattr(torch, "__version__", "0.0.1")
    elif change == "python":
        monkeypatch.setattr(sys.implementation, "cache_tag", "cpython-399")
    else:  # built by an earlier form of the build step
        os.remove(build_lib.BINDING_FOR)
    assert not build_lib.up_to_date()
    build_lib.build()
    assert build_lib.up_to_date()


def test_a_newer_source_is_built(build_lib):
    pytest.importorskip("torch")
    build_lib.build()
    later = os.path.getmtime(build_lib.LIB) + 10
    os.utime(build_lib.BINDING, (later, later))
    old = os.path.getmtime(os.path.join(build_lib.CSRC, "cross_fwd.cu")) - 10
    os.utime(build_lib.LIB, (old, old))
    assert not build_lib.up_to_date()
