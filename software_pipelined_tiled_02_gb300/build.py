"""Build the CUDA library ``libtgemm.so`` in-tree for sm_103a (GB300).

One ``-gencode`` target, static CUDA runtime, the translation units compiled
side by side; the result sits next to this file and is what the Python binding
loads.
``build(debug=True)`` makes ``libtgemm_debug.so`` instead: the same kernel
with TGEMM_DEBUG_CHECKS=1, which checks every address it forms and reports
TGEMM_ERR_CHECK instead of touching memory outside its layout.  The tests
run a part of the parity suite against it (``TGEMM_LIB`` selects it).
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libtgemm.so")
LIB_DEBUG = os.path.join(HERE, "libtgemm_debug.so")
SOURCES = [os.path.join(CSRC, f) for f in ("tgemm.cu", "norm.cu", "dropout.cu", "ffn.cu", "ffn_rows.cu", "ffn_few.cu")]
HEADERS = ("ptx.cuh", "layout.h", "watchdog.cuh", "host.h", "elem.cuh", "ffn.cuh")
DEPS = SOURCES + [os.path.join(CSRC, f) for f in HEADERS] + [os.path.join(INCLUDE, "tgemm.h")]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libtgemm.so")


def compile_command(source: str, obj: str, verbose_ptxas: bool = False, debug: bool = False) -> list[str]:
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-c", "-Xcompiler", "-fPIC",
           "-I", INCLUDE, "-I", CSRC, "-o", obj, source]
    if debug:
        cmd.insert(1, "-DTGEMM_DEBUG_CHECKS=1")
    if verbose_ptxas:
        cmd.insert(1, "-Xptxas=-v")
    return cmd


def link_command(objects: list[str], out: str) -> list[str]:
    return [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", out, *objects]


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(d) <= t for d in DEPS)


def _build(variants: list[tuple[bool, str]], verbose: bool = False) -> None:
    """Compile every source of every (debug, library) variant side by side,
    then link each library and put it in place."""
    with tempfile.TemporaryDirectory(prefix="tgemm_build_") as tmp:
        jobs = []
        for debug, lib in variants:
            for src in SOURCES:
                obj = os.path.join(tmp, f"{os.path.basename(src)}.{'debug' if debug else 'release'}.o")
                jobs.append((lib, src, obj, subprocess.Popen(compile_command(src, obj, verbose, debug),
                                                             stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                                             text=True)))
        errors = []
        for lib, src, _, proc in jobs:
            out, _ = proc.communicate()
            if proc.returncode != 0:
                errors.append(f"nvcc failed for {os.path.basename(lib)}, {os.path.basename(src)}:\n{out}")
            elif verbose:
                sys.stderr.write(out)
        if errors:
            raise RuntimeError("\n".join(errors))
        for _, lib in variants:
            out = lib + f".{os.getpid()}.tmp"
            r = subprocess.run(link_command([obj for to, _, obj, _ in jobs if to == lib], out), capture_output=True,
                               text=True)
            if r.returncode != 0:
                raise RuntimeError(f"linking {os.path.basename(lib)} failed:\n" + r.stdout + r.stderr)
            os.replace(out, lib)


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Compile ``libtgemm.so`` (or, with ``debug``, ``libtgemm_debug.so``)
    unless it is newer than every source."""
    lib = LIB_DEBUG if debug else LIB
    if force or not up_to_date(lib):
        _build([(debug, lib)], verbose)
    return lib


def build_all(force: bool = False) -> list[str]:
    """Compile the release and the debug-check library, skipping whichever is up to date."""
    todo = [(debug, lib) for debug, lib in ((False, LIB), (True, LIB_DEBUG)) if force or not up_to_date(lib)]
    if todo:
        _build(todo)
    return [LIB, LIB_DEBUG]


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv))
