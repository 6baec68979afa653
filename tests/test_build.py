"""What the build takes for done, with a compiler that notes its calls in place of nvcc."""
import os
import stat

import pytest

from test_memorization_recurrent_gb300 import build as B

FAKE = """#!/bin/sh
[ "$1" = --version ] && { cat "%(dir)s/version"; exit 0; }
out=; src=
for a in "$@"; do
  case "$prev" in -o) out=$a;; -c) src=$a;; esac
  prev=$a
done
echo "$(basename "${src:-link}") $*" >> "%(dir)s/log"
if [ -e "%(dir)s/cut" ] && [ -n "$src" ]; then echo half > "$out"; exit 1; fi
if [ -n "$src" ]; then echo "$*" > "$out"; cat "$src" >> "$out"; else shift; for o in "$@"; do case "$o" in *.o) cat "$o" >> "$out";; esac; done; fi
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """-> (directory, sources compiled since the last look, build)"""
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (tmp_path / "include").mkdir()
    (csrc / "a.cu").write_text('#include "a.cuh"\none\n')
    (csrc / "a.cuh").write_text("two\n")
    (csrc / "b.cu").write_text("three\n")
    (tmp_path / "version").write_text("13.0\n")
    nvcc = tmp_path / "nvcc"
    nvcc.write_text(FAKE % dict(dir=tmp_path))
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    for k, v in dict(ROOT=tmp_path, CSRC=csrc, OUT=tmp_path / "out", LIB=tmp_path / "out" / "lib.so", NVCC=nvcc).items():
        monkeypatch.setattr(B, k, str(v))
    B._tool.cache_clear()

    def compiled():
        log = tmp_path / "log"
        lines = log.read_text().split("\n")[:-1] if log.exists() else []
        log.write_text("")
        return sorted(line.split()[0] for line in lines)
    yield tmp_path, compiled
    B._tool.cache_clear()


def later(path, text):
    """Writes a file, of a time that tells nothing: that of the epoch's first day."""
    path.write_text(text)
    os.utime(path, (1, 1))


def test_only_what_changed_is_compiled(tree):
    root, compiled = tree
    lib = B.build()
    assert compiled() == ["a.cu", "b.cu", "link"]
    assert B.up_to_date() and B.build() == lib and compiled() == []
    later(root / "csrc" / "a.cuh", "four\n")
    B.build()
    assert compiled() == ["a.cu", "link"]
    later(root / "csrc" / "b.cu", "five\n")
    B.build()
    assert compiled() == ["b.cu", "link"] and "five" in open(lib).read()
    B.build(force=True)
    assert compiled() == ["a.cu", "b.cu", "link"]


def test_other_options_or_another_compiler_compile_all(tree, monkeypatch):
    root, compiled = tree
    B.build()
    compiled()
    lib = B.build(extra=["-DOTHER"])
    assert compiled() == ["a.cu", "b.cu", "link"] and open(lib).read().count("-DOTHER") == 2
    later(root / "csrc" / "b.cu", "six\n")  # a change of one source with yet other options
    lib = B.build()
    assert compiled() == ["a.cu", "b.cu", "link"] and "-DOTHER" not in open(lib).read()
    monkeypatch.setattr(B, "FLAGS", [*B.FLAGS, "-G"])
    B.build()
    assert compiled() == ["a.cu", "b.cu", "link"]
    (root / "version").write_text("13.1\n")
    B._tool.cache_clear()
    B.build()
    assert compiled() == ["a.cu", "b.cu", "link"]


def test_an_object_that_was_cut_off_is_compiled_again(tree):
    root, compiled = tree
    (root / "cut").write_text("")
    with pytest.raises(RuntimeError):
        B.build()
    (root / "cut").unlink()
    compiled()
    lib = B.build()
    assert compiled() == ["a.cu", "b.cu", "link"] and "half" not in open(lib).read()
    # and one that was there before keeps its place until the new one is whole
    later(root / "csrc" / "b.cu", "seven\n")
    (root / "cut").write_text("")
    with pytest.raises(RuntimeError):
        B.build()
    (root / "cut").unlink()
    compiled()
    lib = B.build()
    assert compiled() == ["b.cu", "link"]
    text = open(lib).read()
    assert "half" not in text and "seven" in text


def test_variants_have_objects_of_their_own(tree):
    root, compiled = tree
    plain = B.build()
    compiled()
    other = B.build_variant("v", ["X"])
    assert compiled() == ["a.cu", "b.cu", "link"]
    assert "-DX" in open(other).read() and "-DX" not in open(plain).read()
    assert B.build_variant("v", ["X"]) == other and compiled() == []
    B.build_variant("v", ["Y"])
    assert compiled() == ["a.cu", "b.cu", "link"]


def test_without_a_compiler_a_library_that_is_done_stays(tree, monkeypatch):
    root, compiled = tree
    lib = B.build()
    monkeypatch.setattr(B, "NVCC", str(root / "nvcc"))
    (root / "nvcc").unlink()
    B._tool.cache_clear()
    assert B.build() == lib


def test_builds_at_the_same_time(tree):
    import concurrent.futures as cf
    root, compiled = tree
    with cf.ThreadPoolExecutor(8) as ex:
        libs = list(ex.map(lambda _: B.build(force=True), range(8)))
    assert len(set(libs)) == 1 and B.up_to_date()
    text = open(libs[0]).read()
    assert text.count("one") == text.count("three") == 1
    assert not [p for p in os.listdir(root / "out") if ".tmp" in p]
