"""The build's order and what makes it build again, on stand-ins: no nvcc runs."""
import os

import pytest

from trainable_block_sparse_compressed_b200 import build


def test_the_library_is_built_where_the_python_module_cannot_be(tmp_path, monkeypatch):
    """The C ABI needs neither Python's headers nor torch's."""
    src = tmp_path / "a.cu"
    src.write_text("")
    monkeypatch.setattr(build, "CSRC", str(tmp_path))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))

    def tool(cmd, **kw):        # writes what the compiler or linker was asked for
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return build.subprocess.CompletedProcess(cmd, 0, "", "")

    def no_headers():
        raise RuntimeError("g++ failed: Python.h: No such file")

    monkeypatch.setattr(build.subprocess, "run", tool)
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(build, "build_calls", no_headers)
    with pytest.raises(RuntimeError, match="Python.h"):
        build.build()
    assert os.path.exists(tmp_path / "lib.so")


def test_the_python_module_is_rebuilt_for_another_torch(tmp_path, monkeypatch):
    import torch
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build, "CALLS_FOR", str(tmp_path / "objects" / "calls.txt"), raising=False)
    monkeypatch.setattr(build, "nvcc", lambda: "/cuda/bin/nvcc")
    temporary = []

    def tool(cmd, **kw):
        temporary.append(cmd[cmd.index("-o") + 1])
        with open(temporary[-1], "w"):
            pass
        return build.subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", tool)
    build.build_calls()
    build.build_calls()
    assert len(temporary) == 1
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    build.build_calls()
    build.build_calls()
    assert len(temporary) == 2
    # a name of this process's own: another build's compiler writes elsewhere
    assert all(str(os.getpid()) in t for t in temporary)
    assert os.listdir(tmp_path / "objects") == ["calls.txt"]


def test_a_module_built_for_another_torch_is_refused(monkeypatch):
    import torch
    from trainable_block_sparse_compressed_b200 import infllmv2 as api
    api._native()
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    with pytest.raises(RuntimeError, match="built for torch"):
        api._native()
