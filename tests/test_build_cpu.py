"""What building needs: the library only nvcc, the binding torch as well."""
import os
import re
import shutil
import stat
import subprocess
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


def test_binding_follows_the_header(tmp_path, monkeypatch):
    """It is compiled against include/rmsnorm.h: another prototype of an entry point that
    it calls does not compile, and a newer header makes it stale."""
    if shutil.which("g++") is None or not os.path.exists(b._nvcc()):
        pytest.skip("needs g++ and the CUDA headers")
    text = open(os.path.join(b.INCLUDE, "rmsnorm.h")).read()
    src = os.path.join(b.CSRC, "binding.cpp")

    def compiles(header):
        (tmp_path / "rmsnorm.h").write_text(header)
        return subprocess.run(["g++", *b._binding_flags(), "-O0", "-fsyntax-only", "-I" + str(tmp_path), src],
                              capture_output=True).returncode == 0
    assert compiles(text)
    changed = re.sub(r"int rmsnorm_kv_release\(", "int rmsnorm_kv_release(int64_t more, ", text)
    assert changed != text and not compiles(changed)
    built = tmp_path / "built.so"
    built.write_text("")
    newest = max(os.path.getmtime(p) for p in (src, os.path.join(b.INCLUDE, "rmsnorm.h")))
    os.utime(built, (newest + 1, newest + 1))
    assert not b._binding_stale(str(built))
    monkeypatch.setattr(b, "INCLUDE", str(tmp_path))
    os.utime(tmp_path / "rmsnorm.h", (newest + 2, newest + 2))
    assert b._binding_stale(str(built))
