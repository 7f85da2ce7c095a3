"""Builds the in-tree CUDA library ``libfp8mqa.so`` for sm_103a with nvcc, and with the host
compiler the paged operators' binding ``_paged_binding.so`` against the installed torch.

Usage: ``python -m fp8_mqa_logits_02_gb300.nvcc_build`` (also called by the package's
``build()`` helper).  The outputs (``libfp8mqa.so``, its bounds-checking variant
``libfp8mqa_debug.so`` and the binding) land next to this file and are git-ignored.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SOURCES = [os.path.join(CSRC, "fp8_mqa_logits.cu"), os.path.join(CSRC, "paged.cu")]
LIB = os.path.join(HERE, "libfp8mqa.so")
# The same library built with FP8MQA_DEBUG_BOUNDS: every global access and TMA coordinate of the
# prefill logits' kernel and of the paged operators' kernels is checked first, and a violation is
# recorded in the status word (fp8_mqa_logits_check_error then returns FP8MQA_ERR_BOUNDS) instead
# of being made.  (The top-k kernels are the same in both.)
DEBUG_LIB = os.path.join(HERE, "libfp8mqa_debug.so")
BINDING_SOURCE = os.path.join(CSRC, "paged_binding.cpp")
BINDING = os.path.join(HERE, "_paged_binding.so")
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libfp8mqa.so")
    return cand


def deps() -> list:
    """Every file the library is compiled from: all of csrc/, the public header and this
    script (a change to any of them triggers a rebuild)."""
    files = [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC))
             if f.endswith((".cu", ".cuh", ".h"))]
    return files + [os.path.join(ROOT, "include", "fp8_mqa_logits.h"), os.path.abspath(__file__)]


def torch_dir() -> str:
    import torch
    return os.path.dirname(os.path.abspath(torch.__file__))


def binding_deps() -> list:
    """What the binding is compiled from; another torch has other headers and needs a new one."""
    return [BINDING_SOURCE, os.path.join(ROOT, "include", "fp8_mqa_logits.h"), os.path.abspath(__file__),
            os.path.join(torch_dir(), "version.py")]


def up_to_date(lib: str) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(d) <= t for d in (binding_deps() if lib == BINDING else deps()))


def _compile(source: str, out: str, debug: bool, verbose: bool) -> list:
    cmd = [nvcc_path(), *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "-c",
           "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
           "-I", os.path.join(ROOT, "include"), "-o", out, source]
    if debug:
        cmd.insert(1, "-DFP8MQA_DEBUG_BOUNDS")
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    return cmd


def _binding(out: str) -> list:
    t, cuda = torch_dir(), os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    lib = os.path.join(t, "lib")
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            "-I", os.path.join(t, "include"), "-I", os.path.join(t, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"],
            "-o", out, BINDING_SOURCE, "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def _run(jobs: dict) -> dict:
    """Runs the commands side by side; their output by name, and whether each succeeded."""
    running, done = {}, {}
    for what, cmd in jobs.items():
        try:
            running[what] = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
        except OSError as e:  # no such compiler
            done[what] = (False, str(e))
    for what, proc in running.items():
        out, _ = proc.communicate()
        done[what] = (proc.returncode == 0, out)
    return done


def build(force: bool = False, verbose: bool = False, debug: bool | None = None) -> str:
    """Build the library (debug=False), its bounds-checking variant (debug=True), or both
    at once (debug=None, the default; returns the regular library's path), and the binding.
    Each is rebuilt only when a source is newer, unless `force`.  All translation units
    compile at the same time.

    Each output stands for itself: what compiles is put in place.  A library that does not build
    raises RuntimeError; the binding needs the host compiler and torch's headers as well, and where it
    cannot be built there is a warning, the rest of the library works, and the paged operators raise."""
    targets = [False, True] if debug is None else [bool(debug)]
    tag = f".tmp{os.getpid()}"
    jobs, objects = {}, {}  # name: command; library: {name: object}
    for dbg in targets:
        lib = DEBUG_LIB if dbg else LIB
        if not force and up_to_date(lib):
            continue
        objects[lib] = {}
        for source in SOURCES:
            what = f"{os.path.basename(lib)} ({os.path.basename(source)})"
            objects[lib][what] = f"{lib}.{os.path.basename(source)}{tag}.o"
            jobs[what] = _compile(source, objects[lib][what], dbg, verbose)
    binding, no_binding = os.path.basename(BINDING), ""
    try:
        if force or not up_to_date(BINDING):
            jobs[binding] = _binding(BINDING + tag)
    except ImportError as e:  # no torch
        no_binding = str(e)
    done = _run(jobs)
    if verbose:
        sys.stderr.write("".join(out for ok, out in done.values() if ok))
    failed = []
    for lib, parts in objects.items():
        wrong = [f"compiling {what} failed:\n{done[what][1]}" for what in parts if not done[what][0]]
        if not wrong:
            ok, out = _run({lib: [nvcc_path(), *ARCH_FLAGS, "-shared", "-o", lib + tag, *parts.values()]})[lib]
            if ok:
                os.replace(lib + tag, lib)
            else:
                wrong = [f"linking {os.path.basename(lib)} failed:\n{out}"]
        failed += wrong
        for path in [lib + tag, *parts.values()]:
            if os.path.exists(path):
                os.remove(path)
    if binding in done:
        if done[binding][0]:
            os.replace(BINDING + tag, BINDING)
        else:
            no_binding = done[binding][1]
    if no_binding:
        for path in (BINDING + tag, BINDING):  # one from other sources would not go with the library
            if os.path.exists(path):
                os.remove(path)
    if failed:
        raise RuntimeError("\n".join(failed))
    if no_binding:
        warnings.warn(f"the paged operators are not available: building {binding} failed:\n{no_binding}", stacklevel=2)
    return DEBUG_LIB if debug else LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
