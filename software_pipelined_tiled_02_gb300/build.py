"""Build the CUDA library ``libtgemm.so`` in-tree for sm_103a (GB300).

One ``-gencode`` target, static CUDA runtime, the translation units compiled
side by side; the result sits next to this file and is what the Python package
loads.  ``_binding.so`` is the package's extension module for the operators on
torch tensors, compiled against the installed torch, and again when another
torch or Python is installed; without torch it is left out, and the library,
which needs neither, is still made.
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
BINDING = os.path.join(HERE, "_binding.so")
BINDING_MADE_FOR = os.path.join(HERE, "_binding.made_for")  # what the binding was compiled against
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
SOURCES = [os.path.join(CSRC, f) for f in ("tgemm.cu", "norm.cu", "dropout.cu", "ffn.cu", "ffn_rows.cu", "ffn_few.cu",
                                                 "route.cu", "w4.cu", "experts.cu", "experts_rows.cu",
                                                 "experts_few.cu")]
HEADERS = ("ptx.cuh", "layout.h", "watchdog.cuh", "host.h", "elem.cuh", "ffn.cuh", "experts.cuh", "pairs.cuh")
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


def binding_command(out: str) -> list[str]:
    import sysconfig

    import torch

    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-Wno-attributes",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
            "-isystem", os.path.join(home, "include"),
            "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"], "-o", out, BINDING_SOURCE,
            "-L", os.path.join(home, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python",
            "-Wl,-rpath," + os.path.join(home, "lib")]


def made_for() -> str:
    """What the binding depends on besides its sources: the installed torch and this Python.  Does not import torch."""
    from importlib import metadata

    try:
        torch = metadata.version("torch")
    except metadata.PackageNotFoundError:
        torch = "none"
    return f"torch {torch}, {sys.implementation.cache_tag}, {sys.prefix}"


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    if lib == BINDING:
        try:
            with open(BINDING_MADE_FOR) as f:
                if f.read() != made_for():
                    return False
        except OSError:
            return False
    deps = [BINDING_SOURCE, os.path.join(INCLUDE, "tgemm.h")] if lib == BINDING else DEPS
    return all(os.path.getmtime(d) <= t for d in deps)


def _have_torch() -> bool:
    try:
        import torch  # noqa: F401
    except ImportError as e:
        sys.stderr.write(f"torch does not load ({e}): {os.path.basename(BINDING)}, which the operators on torch "
                         "tensors need, is left out\n")
        return False
    return True


def _build(libraries: list[str], verbose: bool = False) -> None:
    """Compile every source of every library in ``libraries`` (and the binding,
    if it is among them) side by side, then link and put each in place: what
    succeeds also when another one fails."""
    if BINDING in libraries and not _have_torch():
        libraries = [lib for lib in libraries if lib != BINDING]
    with tempfile.TemporaryDirectory(prefix="tgemm_build_") as tmp:
        todo = []  # (library, source, object, command)
        for lib in libraries:
            if lib == BINDING:
                obj = lib + f".{os.getpid()}.tmp"
                todo.append((lib, BINDING_SOURCE, obj, binding_command(obj)))
            else:
                objs = [os.path.join(tmp, f"{os.path.basename(src)}.{os.path.basename(lib)}.o") for src in SOURCES]
                todo += [(lib, src, obj, compile_command(src, obj, verbose, lib == LIB_DEBUG)) for src, obj in zip(SOURCES, objs)]
        jobs, errors, failed = [], [], set()
        for lib, src, obj, cmd in todo:
            try:
                jobs.append((lib, src, obj, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
            except OSError as e:
                failed.add(lib)
                errors.append(f"{os.path.basename(lib)}: {cmd[0]} does not start: {e}")
        for lib, src, _, proc in jobs:
            out, _ = proc.communicate()
            if proc.returncode != 0:
                failed.add(lib)
                errors.append(f"compiling {os.path.basename(src)} for {os.path.basename(lib)} failed:\n{out}")
            elif verbose:
                sys.stderr.write(out)
        for lib in libraries:
            if lib in failed:
                continue
            objects = [obj for to, _, obj, _ in jobs if to == lib]
            out = objects[0]
            if lib != BINDING:
                out = lib + f".{os.getpid()}.tmp"
                r = subprocess.run(link_command(objects, out), capture_output=True, text=True)
                if r.returncode != 0:
                    errors.append(f"linking {os.path.basename(lib)} failed:\n" + r.stdout + r.stderr)
                    continue
            os.replace(out, lib)
            if lib == BINDING:
                with open(BINDING_MADE_FOR, "w") as f:
                    f.write(made_for())
        if errors:
            raise RuntimeError("\n".join(errors))


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Compile ``libtgemm.so`` (or, with ``debug``, ``libtgemm_debug.so``) and
    the binding unless they are newer than their sources."""
    lib = LIB_DEBUG if debug else LIB
    _build([out for out in (lib, BINDING) if force or not up_to_date(out)], verbose)
    return lib


def build_all(force: bool = False) -> list[str]:
    """Compile the release and the debug-check library and the binding, skipping whichever is up to date."""
    outs = [LIB, LIB_DEBUG, BINDING]
    _build([out for out in outs if force or not up_to_date(out)])
    return outs


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv))
