"""Build libatlasmem.so (sm_103a) in-tree with nvcc: one object per .cu file,
compiled in parallel, then linked into a shared library under _build/.

An object is used again if what it was made of is the same: the text of its source and the
headers it includes, the compiler and its options, of which it has a digest beside it.  Objects,
digests and the library are written under another name and then take their place, so that
a build that is cut off leaves none that looks done.

``build_variant`` builds a separately named copy with extra preprocessor
definitions (used by tests that need a test-only switch compiled in); the
library the package loads is always the plain one."""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import functools
import glob
import hashlib
import os
import platform
import re
import subprocess
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libatlasmem.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"),
         "-I", CSRC, "--expt-relaxed-constexpr"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _included(path: str, seen: set) -> set:
    """A source file and the project's headers that it includes, directly or not."""
    if path not in seen:
        seen.add(path)
        with open(path, encoding="utf-8") as f:
            names = re.findall(r'^#include "([^"]+)"', f.read(), flags=re.M)
        for name in names:
            for where in (CSRC, os.path.join(ROOT, "include")):
                if os.path.exists(os.path.join(where, name)):
                    _included(os.path.join(where, name), seen)
    return seen


@functools.lru_cache(maxsize=None)
def _tool() -> str:
    """The compiler's version and the machine; empty without a compiler."""
    try:
        r = subprocess.run([NVCC, "--version"], capture_output=True, text=True)
    except OSError:
        return ""
    return hashlib.sha256((platform.machine() + r.stdout).encode()).hexdigest()


def _key(src: str, extra) -> str:
    """Digest of what an object is made of."""
    h = hashlib.sha256("\0".join([NVCC, *ARCH, *FLAGS, *extra]).encode())
    for path in sorted(_included(src, set())):
        with open(path, "rb") as f:
            text = f.read()
        h.update(f"\0{os.path.basename(path)} {len(text)}\0".encode() + text)
    return h.hexdigest()


def _done(path: str, key: str) -> bool:
    """Whether a file was made of this (by this compiler, if there is one)."""
    try:
        with open(path + ".made", encoding="utf-8") as f:
            made = f.read().split()
    except OSError:
        return False
    return os.path.exists(path) and made[:1] == [key] and (not _tool() or made[1:] == [_tool()])


def _make(path: str, key: str, cmd, what: str) -> None:
    """Runs cmd, which writes the file that its last argument names, here path under another name."""
    tmp = f"{path}.tmp{os.getpid()}.{threading.get_ident()}"
    try:
        r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
        with contextlib.suppress(FileNotFoundError):  # (another build may be at the same place)
            os.remove(path + ".made")
        os.replace(tmp, path)
        with open(tmp, "w", encoding="utf-8") as f:
            f.write(f"{key} {_tool()}\n")
        os.replace(tmp, path + ".made")
    finally:
        if os.path.exists(tmp):
            os.remove(tmp)


def _compile(src: str, objdir: str, extra, key: str, force: bool = True) -> str:
    obj = os.path.join(objdir, os.path.basename(src)[:-3] + ".o")
    if force or not _done(obj, key):
        _make(obj, key, [NVCC, *ARCH, *FLAGS, *extra, "-c", src], f"nvcc failed on {src}")
    return obj


def _keys(extra):
    """Of the objects, and of a library of them."""
    keys = [_key(s, extra) for s in _sources()]
    return keys, hashlib.sha256("".join(keys).encode()).hexdigest()


def up_to_date(lib: str = "", extra=()) -> bool:
    return _done(lib or LIB, _keys(list(extra))[1])


def _build(lib: str, objdir: str, extra, force: bool) -> str:
    extra = list(extra)
    keys, whole = _keys(extra)
    if not force and _done(lib, whole):
        return lib
    os.makedirs(objdir, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=os.cpu_count() or 4) as ex:
        objs = list(ex.map(lambda s, k: _compile(s, objdir, extra, k, force), _sources(), keys))
    _make(lib, whole, [NVCC, *ARCH, "-shared", *objs, "-lcudart"], "link failed")
    return lib


def build(force: bool = False, extra=()) -> str:
    return _build(LIB, OUT, extra, force)


def build_variant(name: str, defines, force: bool = False) -> str:
    """Build lib<name>.so under _build/<name>/ with -D<define> for each entry."""
    objdir = os.path.join(OUT, name)
    lib = os.path.join(objdir, f"lib{name}.so")
    return _build(lib, objdir, [f"-D{d}" for d in defines], force)


if __name__ == "__main__":
    print(build(force=True))
