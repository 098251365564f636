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
