"""What is built from what, and what a missing torch or host compiler leaves unbuilt.  The
compilers are stand-ins that write the file they are asked for and note their call.
"""

import os
import shutil
import stat

import pytest

from paged_kv_cache_qk_gb300 import build as b

COMPILER = """#!/bin/sh
echo {name} "$@" >> {log}
while [ $# -gt 1 ]; do
  if [ "$1" = -o ]; then echo {name} > "$2"; fi
  shift
done
"""


class Tree:
    """A copy of the sources with stand-in compilers; `calls` notes what ran since last asked."""

    def __init__(self, tmp_path, monkeypatch):
        self.tmp, self.log, self.patch = tmp_path, tmp_path / "log", monkeypatch
        self.csrc = tmp_path / "csrc"
        shutil.copytree(b.CSRC, self.csrc)
        (tmp_path / "torch").mkdir()
        (tmp_path / "torch" / "version.py").write_text("")
        for f in [*self.csrc.iterdir(), tmp_path / "torch" / "version.py"]:
            os.utime(f, (1, 1))
        for name, value in dict(PKG=tmp_path, CSRC=self.csrc, BUILD=tmp_path / "_build",
                                LIB=tmp_path / "libpkvqk.so",
                                CALLS=tmp_path / "torch_calls.so").items():
            monkeypatch.setattr(b, name, str(value))
        for name in ("nvcc", "cxx"):
            path = tmp_path / name
            path.write_text(COMPILER.format(name=name, log=self.log))
            path.chmod(path.stat().st_mode | stat.S_IEXEC)
            monkeypatch.setattr(b, name, lambda path=path: str(path))
        monkeypatch.setattr(b, "torch_dir", lambda: str(tmp_path / "torch"))

    def calls(self):
        lines = self.log.read_text().splitlines() if self.log.exists() else []
        self.log.write_text("")
        return sorted({line.split()[0] for line in lines}), len(lines)

    def have(self):
        return os.path.exists(b.LIB), os.path.exists(b.CALLS)

    def touch(self, name):
        later = max(os.path.getmtime(f) for f in (b.LIB, b.CALLS)) + 5
        os.utime(self.csrc / name, (later, later))

    def settle(self):
        """Built files newer than every source."""
        newest = max(f.stat().st_mtime for f in self.csrc.iterdir()) + 5
        for f in (b.LIB, b.CALLS):
            os.utime(f, (newest, newest))


@pytest.fixture
def tree(tmp_path, monkeypatch):
    return Tree(tmp_path, monkeypatch)


def test_both_are_built_once(tree):
    assert b.build() == b.LIB
    assert tree.have() == (True, True)
    assert tree.calls() == (["cxx", "nvcc"], len(b.SOURCES) + 1 + 2)
    b.build()
    assert tree.calls() == ([], 0)
    b.build(force=True)
    assert tree.calls() == (["cxx", "nvcc"], len(b.SOURCES) + 1 + 2)


def test_without_torch_the_library_is_built(tree):
    tree.patch.setattr(b, "torch_dir", lambda: None)
    assert b.build() == b.LIB
    assert tree.have() == (True, False)
    assert tree.calls()[0] == ["nvcc"]
    b.build()                                  # and is not built again
    assert tree.calls() == ([], 0)


def test_without_a_host_compiler_the_library_is_there_before_the_error(tree):
    def missing():
        raise RuntimeError("no C++ compiler found")

    tree.patch.setattr(b, "cxx", missing)
    with pytest.raises(RuntimeError, match="no C..? compiler"):
        b.build()
    assert tree.have() == (True, False)


def test_a_failing_binding_leaves_the_library(tree):
    (tree.tmp / "cxx").write_text("#!/bin/sh\necho no headers; exit 1\n")
    with pytest.raises(RuntimeError, match="torch_calls.cpp"):
        b.build()
    assert tree.have() == (True, False)


def test_each_is_built_from_its_own_sources(tree):
    b.build()
    tree.calls()
    tree.touch("torch_calls.cpp")
    b.build()
    assert tree.calls() == (["cxx"], 2)
    tree.settle()
    for name in ("decode.cu", "score_rules.cuh", "kernels.h"):
        tree.touch(name)
        b.build()
        assert tree.calls() == (["nvcc"], len(b.SOURCES) + 1)
        tree.settle()


def test_another_torch_needs_another_binding(tree):
    """Also one whose files are older than what was built."""
    b.build()
    tree.calls()
    (tree.tmp / "other").mkdir()
    (tree.tmp / "other" / "version.py").write_text("")
    os.utime(tree.tmp / "other" / "version.py", (1, 1))
    tree.patch.setattr(b, "torch_dir", lambda: str(tree.tmp / "other"))
    b.build()
    assert tree.calls() == (["cxx"], 2)
    b.build()
    assert tree.calls() == ([], 0)
    (tree.tmp / "other" / "version.py").write_text("upgraded in place")
    os.utime(tree.tmp / "other" / "version.py", (1, 1))
    b.build()
    assert tree.calls() == (["cxx"], 2)


def test_torch_is_not_found_where_there_is_none(monkeypatch):
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: None)
    assert b.torch_dir() is None
