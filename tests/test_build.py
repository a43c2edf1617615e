"""The build on its own (CPU): the library does not need the Python binding, and the binding is
built again for another PyTorch or Python."""
import ctypes
import os

import pytest
import torch

from speculative_decoding_verification_76_gb300 import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """The build with its outputs in a folder of their own and one small source."""
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libspecverify.so"))
    monkeypatch.setattr(b, "NATIVE", str(tmp_path / "_native.so"))
    monkeypatch.setattr(b, "sources", lambda: [os.path.join(b.CSRC, "kv_commit.cu")])
    binding = tmp_path / "binding.cpp"
    monkeypatch.setattr(b, "BINDING", str(binding))
    return binding


def test_the_library_is_built_where_the_binding_is_not(tree):
    tree.write_text("#include <no/such/header.h>\n")
    with pytest.raises(RuntimeError, match="no/such/header"):
        b.build()
    lib = ctypes.CDLL(b.LIB)
    assert lib.spec_kv_commit and not os.path.exists(b.NATIVE)
    # with a binding that compiles, the library stays as it is
    at = os.path.getmtime(b.LIB)
    tree.write_text("int nothing;\n")
    assert b.build() == b.LIB and os.path.exists(b.NATIVE)
    assert os.path.getmtime(b.LIB) == at


def test_the_binding_is_built_again_for_another_torch(tree, monkeypatch):
    tree.write_text("int nothing;\n")
    b.build()
    lib, native = os.path.getmtime(b.LIB), os.stat(b.NATIVE).st_mtime_ns
    b.build()
    assert os.stat(b.NATIVE).st_mtime_ns == native
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    b.build()
    assert os.stat(b.NATIVE).st_mtime_ns > native and os.path.getmtime(b.LIB) == lib
    native = os.stat(b.NATIVE).st_mtime_ns
    b.build()
    assert os.stat(b.NATIVE).st_mtime_ns == native


def test_the_library_is_built_without_torch(tree, monkeypatch):
    tree.write_text("int nothing;\n")
    monkeypatch.setitem(__import__("sys").modules, "torch", None)   # import torch fails
    assert b.build() == b.LIB
    assert ctypes.CDLL(b.LIB).spec_kv_commit and not os.path.exists(b.NATIVE)
