"""The build's parts do not hang on one another: a C user of the library needs no torch headers."""
import ctypes
import subprocess

import pytest

from adaptive_block_sparse_b200 import build as b


def test_the_library_is_linked_where_the_binding_cannot_be_built(tmp_path, monkeypatch):
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')

    def compile_one(path, verbose, extra):
        obj = str(tmp_path / "one.o")
        subprocess.run(["g++", "-x", "c++", "-fPIC", "-c", path, "-o", obj], check=True)
        return obj

    def no_headers(verbose):
        raise RuntimeError("binding.cpp failed: torch/csrc/Exceptions.h: No such file")
    lib = tmp_path / "libnabla.so"
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(lib))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(b, "_sources", lambda: [str(src)])
    monkeypatch.setattr(b, "_compile", compile_one)
    monkeypatch.setattr(b, "_compile_binding", no_headers)
    with pytest.raises(RuntimeError, match="binding.cpp"):        # still reported
        b.build()
    assert lib.exists() and not (tmp_path / "_binding.so").exists()
    assert ctypes.CDLL(str(lib)).one() == 1
