"""What building needs: the library only nvcc, the binding torch as well."""
import os
import stat
import sys

import pytest

from rmsnorm_fwd_bwd_add_gb300 import build as b


@pytest.fixture()
def tree(tmp_path, monkeypatch):
    """build's outputs in an empty folder, with an nvcc that only touches its output."""
    nvcc = tmp_path / "nvcc"
    nvcc.write_text("#!/bin/sh\nwhile [ $# -gt 1 ]; do [ \"$1\" = -o ] && touch \"$2\"; shift; done\n")
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(b, "_nvcc", lambda: str(nvcc))
    monkeypatch.setattr(b, "PKG_DIR", str(tmp_path))
    monkeypatch.setattr(b, "OBJ_DIR", str(tmp_path / "obj"))
    monkeypatch.setattr(b, "LIB_PATH", str(tmp_path / "lib.so"))
    return tmp_path


def test_library_is_linked_although_the_binding_fails(tree, monkeypatch):
    def fails(path):
        raise RuntimeError("g++ failed on binding.cpp")
    monkeypatch.setattr(b, "_compile_binding", fails)
    for _ in range(2):  # and what failed is tried again
        with pytest.raises(RuntimeError, match="binding"):
            b.build()
        assert os.path.exists(b.LIB_PATH)


def test_library_is_built_without_torch(tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert b.build() == b.LIB_PATH and os.path.exists(b.LIB_PATH)
    assert b.build() == b.LIB_PATH
    assert not [f for f in os.listdir(tree) if f.startswith("_binding")]


def test_both_are_built_with_torch(tree, monkeypatch):
    made = []
    monkeypatch.setattr(b, "_compile_binding", lambda path: made.append(path) or open(path, "w").close())
    assert b.build() == b.LIB_PATH and os.path.exists(b.LIB_PATH)
    assert made == [b.binding_path()]
    b.build()
    assert len(made) == 1
