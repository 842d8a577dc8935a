"""What is built from what, and what is used when a part cannot be built.  The
compilers are stand-ins that write the files they are asked for."""

import os
import subprocess
import time

import pytest

from paged_kv_cache_473_b200 import _binding as bnd
from paged_kv_cache_473_b200 import build as bld


class Compilers:
    """Records commands; an output is a copy of the command line, its dependency file names the source."""

    def __init__(self, broken=()):
        self.broken, self.commands = broken, []

    def run(self, cmd, check=True, **kw):
        self.commands.append(list(cmd))
        if os.path.basename(cmd[0]) in self.broken:
            raise subprocess.CalledProcessError(1, cmd)
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w") as f:
            f.write(" ".join(cmd))
        if "-MF" in cmd:
            with open(cmd[cmd.index("-MF") + 1], "w") as f:
                f.write(f"object: {cmd[-1]}\n")

    def compiled(self):
        """Sources compiled since the last look."""
        got = sorted(os.path.basename(c[-1]) if c[-1].endswith((".cu", ".cpp")) else os.path.basename(c[c.index("-c") + 1])
                     for c in self.commands if "-c" in c)
        self.commands = []
        return got


LIBRARY = sorted(os.path.basename(u) for u in bld.UNITS)
EVERYTHING = sorted([*LIBRARY, "native_binding.cpp"])


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Empty places for what is built (the repository's own library is opened before)."""
    assert bnd.lib
    monkeypatch.setattr(bnd, "_lib_handle", bnd.lib)
    monkeypatch.setattr(bld, "LIB", str(tmp_path / "libpagedattn.so"))
    monkeypatch.setattr(bld, "NATIVE", str(tmp_path / "_native.so"))
    monkeypatch.setattr(bld, "OBJ_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(bld, "_nvcc", lambda: "nvcc")

    def use(*broken):
        c = Compilers(broken)
        monkeypatch.setattr(bld.subprocess, "run", c.run)
        return c

    return use


def test_build_makes_both_and_then_nothing(tree):
    c = tree()
    bld.build()
    assert os.path.exists(bld.LIB) and os.path.exists(bld.NATIVE)
    assert c.compiled() == EVERYTHING
    bld.build()
    assert c.compiled() == []


def test_the_library_is_built_where_the_native_module_cannot_be(tree):
    tree("g++")
    with pytest.raises(subprocess.CalledProcessError):
        bld.build()
    assert os.path.exists(bld.LIB) and not os.path.exists(bld.NATIVE)


def test_calls_that_do_not_need_the_native_module_work_without_it(tree, monkeypatch):
    tree("g++", "nvcc")
    monkeypatch.setattr(bld, "LIB", bnd.lib._name)
    monkeypatch.setattr(bnd, "_native_module", None)
    monkeypatch.setattr(bnd, "_lib_handle", None)
    assert bnd.error_string(0) == "ok"
    with pytest.raises(ImportError, match="native module"):
        bnd.qk_norm_rope(None, None, None, None)


def test_a_missing_library_is_refused(tree):
    tree("nvcc")
    with pytest.raises(ImportError, match="libpagedattn"):
        bnd._load_library()


def test_only_what_changed_is_built(tree):
    c = tree()
    bld.build()
    c.compiled()
    past = time.time() - 1000
    os.utime(bld.NATIVE, (past, past))
    os.utime(os.path.join(bld.OBJ_DIR, "native_binding.cpp.o"), (1, 1))
    bld.build()
    assert c.compiled() == ["native_binding.cpp"]
    os.utime(bld.LIB, (1, 1))
    os.utime(os.path.join(bld.OBJ_DIR, "tree_ops.cu.o"), (1, 1))
    bld.build()
    assert c.compiled() == ["tree_ops.cu"]


def test_objects_of_other_flags_are_not_reused(tree):
    c = tree()
    bld.build(force=True, extra_flags=["-DINSTRUMENTED"])
    c.compiled()
    assert bnd._build.library_up_to_date()  # as it is, for what opens it
    bld.build()
    assert c.compiled() == LIBRARY
    bld.build()
    assert c.compiled() == []
    bld.build(extra_flags=["-DINSTRUMENTED"])
    assert c.compiled() == LIBRARY
    os.utime(bld.LIB, (1, 1))
    bld.build()  # a source changed since: all units anew, not only the stale one
    assert c.compiled() == LIBRARY


def test_another_torch_makes_the_native_module_anew(tree, monkeypatch):
    import torch

    c = tree()
    bld.build()
    c.compiled()
    monkeypatch.setattr(torch, "__version__", "99.1")
    bld.build()
    assert c.compiled() == ["native_binding.cpp"]
    tree("g++")
    monkeypatch.setattr(torch, "__version__", "99.2")
    monkeypatch.setattr(bnd, "_native_module", None)
    with pytest.raises(ImportError, match="another torch"):
        bnd.qk_norm_rope(None, None, None, None)


def test_what_came_without_its_objects_is_taken_by_its_time(tree):
    c = tree()
    bld.build()
    for stamp in (bld._stamp(bld.LIB), bld._stamp(bld.NATIVE)):
        os.remove(stamp)
    c.compiled()
    bld.build()
    assert c.compiled() == []
