"""Which objects a build of the CUDA library takes over and which it compiles again, with a stand-in for nvcc that
records what it is asked to make."""
import os
import stat
import time

import pytest

from fft_long_convolution_causal_b200 import build

NVCC = """#!/bin/sh
if [ "$1" = --version ]; then echo "release $VERSION"; exit 0; fi
out= dep= src=
while [ $# -gt 0 ]; do
    case "$1" in -o) out=$2; shift;; -MF) dep=$2; shift;; *.cu) src=$1;; esac
    shift
done
echo "$(basename "$out")" >> {log}
[ -z "$FAIL" ] || {{ echo half > "$out"; exit 1; }}
[ -z "$dep" ] || echo "$out: $src {header}" > "$dep"
echo whole > "$out"
"""


@pytest.fixture()
def tree(tmp_path, monkeypatch):
    csrc, log, nvcc = tmp_path / "csrc", tmp_path / "log", tmp_path / "nvcc"
    csrc.mkdir()
    for n in ("a.cu", "b.cu", "c.cuh"):
        (csrc / n).write_text("")
    nvcc.write_text(NVCC.format(log=log, header=csrc / "c.cuh"))
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    past = time.time() - 100
    for f in csrc.iterdir():
        os.utime(f, (past, past))
    for name, value in (("CSRC", str(csrc)), ("INCLUDE", str(tmp_path / "include")), ("NVCC", str(nvcc)),
                        ("LIB", str(tmp_path / "lib.so")), ("BUILD_DIR", str(tmp_path / "objects"))):
        monkeypatch.setattr(build, name, value)
    monkeypatch.setenv("VERSION", "1")

    def made():
        """What the next build makes."""
        log.write_text("")
        if hasattr(build, "_version"):
            build._version.cache_clear()
        build.build()
        return sorted(log.read_text().split())

    return made, csrc


ALL = ["a.cu.o", "b.cu.o", "lib.so.tmp"]


def test_nothing_changed(tree):
    made, _ = tree
    assert made() == ALL
    assert made() == []


def test_a_source_and_a_header(tree):
    made, csrc = tree
    made()
    later = time.time() + 5
    os.utime(csrc / "b.cu", (later, later))
    assert made() == ["b.cu.o", "lib.so.tmp"]
    os.utime(csrc / "c.cuh", (later + 5, later + 5))
    assert made() == ALL


@pytest.mark.parametrize("name", ["FLAGS", "ARCH"])
def test_other_commands(tree, monkeypatch, name):
    made, csrc = tree
    made()
    monkeypatch.setattr(build, name, getattr(build, name) + ["-DOTHER"])
    assert made() == ALL
    assert made() == []


def test_another_compiler(tree, monkeypatch):
    made, _ = tree
    made()
    monkeypatch.setenv("VERSION", "2")
    assert made() == ALL


def test_other_commands_and_one_source(tree, monkeypatch):
    """What happened before: one source newer, the other object linked as it was."""
    made, csrc = tree
    made()
    monkeypatch.setattr(build, "FLAGS", build.FLAGS + ["-DOTHER"])
    later = time.time() + 5
    os.utime(csrc / "b.cu", (later, later))
    assert made() == ALL


def test_a_compilation_cut_short(tree, monkeypatch):
    made, csrc = tree
    made()
    past = time.time() - 50  # the source was changed between the library and the half-written object
    os.utime(build.LIB, (past - 10, past - 10))
    os.utime(csrc / "b.cu", (past, past))
    os.utime(os.path.join(build.BUILD_DIR, "b.cu.o"), (past - 5, past - 5))
    monkeypatch.setenv("FAIL", "1")
    with pytest.raises(RuntimeError):
        made()
    monkeypatch.delenv("FAIL")
    assert made() == ["b.cu.o", "lib.so.tmp"]


def test_without_a_compiler(tree, monkeypatch):
    """A library that came with the tree is taken as it is, unless a source is newer."""
    made, csrc = tree
    made()
    monkeypatch.setattr(build, "NVCC", str(csrc / "no-nvcc"))
    assert made() == []
    later = time.time() + 5
    os.utime(csrc / "b.cu", (later, later))
    with pytest.raises(OSError):
        made()
