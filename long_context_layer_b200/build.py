"""Build the in-tree shared libraries with nvcc for sm_100a.

    python long_context_layer_b200/build.py [--force]

(Run it by path: importing the package loads the library this script builds.)

Produces long_context_layer_b200/libdelta_attn.so (the C ABI of include/delta_attn.h),
long_context_layer_b200/_fastcall.<tag>.so (the binding's call module, named for the interpreter it is built for
and left out where Python's headers are missing), synth/libsynth_fill.so (the device-side input generator used by
tests and the benchmark) and synth/libsynth_host.so (the same generator on the host, for fast oracle inputs).
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
COMMON = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC"]

CSRC = os.path.join(ROOT, "long_context_layer_b200", "csrc")
# (sources, library, extra flags); the sources of one library compile side by side
TARGETS = [
    ([os.path.join(CSRC, f) for f in ("delta_attn.cu", "window_attn.cu", "attn_q8.cu", "attn_q8_e4m3.cu",
                                      "attn_q8_int8.cu", "cache_q8.cu", "rope.cu")],
     os.path.join(ROOT, "long_context_layer_b200", "libdelta_attn.so"),
     ["-I" + os.path.join(ROOT, "include")]),
    ([os.path.join(ROOT, "synth", "csrc", "synth_fill.cu")],
     os.path.join(ROOT, "synth", "libsynth_fill.so"), []),
]
# host (CPU) libraries built with gcc: the input generator's host copy and the binding's call module
HOST_TARGETS = [
    (os.path.join(ROOT, "synth", "csrc", "synth_host.c"), os.path.join(ROOT, "synth", "libsynth_host.so"), []),
]
PACKAGE = os.path.join(ROOT, "long_context_layer_b200")
PYTHON_INCLUDE = sysconfig.get_paths()["include"]
FASTCALL = (os.path.join(CSRC, "fastcall.c"), os.path.join(PACKAGE, "_fastcall" + sysconfig.get_config_var("EXT_SUFFIX")),
            ["-I" + PYTHON_INCLUDE])


def nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found")
    return p


def build(force: bool = False, verbose: bool = False) -> list:
    built = []
    for srcs, out, extra in TARGETS:
        csrc = os.path.dirname(srcs[0])
        deps = [os.path.join(csrc, f) for f in os.listdir(csrc) if f.endswith((".cu", ".cuh", ".h"))]
        deps += [os.path.join(ROOT, "include", f) for f in os.listdir(os.path.join(ROOT, "include"))]
        if not force and os.path.exists(out) and os.path.getmtime(out) >= max(os.path.getmtime(d) for d in deps):
            continue
        with tempfile.TemporaryDirectory() as tmp:
            objs = [os.path.join(tmp, os.path.basename(src) + ".o") for src in srcs]
            cmds = [[nvcc()] + ARCH + COMMON + extra + ["-c", src, "-o", obj] for src, obj in zip(srcs, objs)]
            link = [nvcc()] + ARCH + ["-shared"] + objs + ["-o", out]
            if verbose:
                print("\n".join(" ".join(c) for c in cmds + [link]), file=sys.stderr)
            with concurrent.futures.ThreadPoolExecutor(os.cpu_count()) as pool:
                list(pool.map(lambda c: subprocess.run(c, check=True), cmds))
            subprocess.run(link, check=True)
        built.append(out)
    host = list(HOST_TARGETS)
    if os.path.exists(os.path.join(PYTHON_INCLUDE, "Python.h")):
        host.append(FASTCALL)
    elif verbose:
        print("Python.h is missing: the binding calls through ctypes", file=sys.stderr)
    untagged = os.path.join(PACKAGE, "_fastcall.so")     # an earlier build's, which any interpreter would load
    if os.path.exists(untagged):
        os.remove(untagged)
    for src, out, extra in host:
        if not force and os.path.exists(out) and os.path.getmtime(out) >= os.path.getmtime(src):
            continue
        cmd = ["gcc", "-O3", "-ffp-contract=off", "-fno-fast-math", "-fPIC", "-shared"] + extra + [src, "-o", out]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
        built.append(out)
    return built


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
