"""Builds libkvp.so (sm_100a) and _torch_calls.so, the Python extension that passes
torch tensors to it, in place with nvcc.

Usage: ``python -m paged_kv_cache_319_b200.build [--force] [--verbose]``.
They land next to this file so the package loads them from the source
tree; intermediate output (the ptxas report) goes to ``_build/``.

libkvp.so needs nvcc alone. The extension also needs Python's headers and a torch whose
DLPack header has the C exchange table (2.11 has); without them it is left out, with a
note, and only the calls that pass through it are missing.
"""

from __future__ import annotations

import argparse
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libkvp.so")
CALLS = os.path.join(PKG, "_torch_calls.so")
CALLS_SOURCE = os.path.join(CSRC, "host", "torch_calls.cpp")
BUILD_DIR = os.path.join(PKG, "_build")

SOURCES = [
    os.path.join(CSRC, "host", "block_pool.cpp"),
    os.path.join(CSRC, "host", "group_plan.cpp"),
    os.path.join(CSRC, "host", "vcache.cpp"),
    os.path.join(CSRC, "kvp_device.cu"),
]


def _inputs():
    files = list(SOURCES)
    for d in (CSRC, INCLUDE):
        for dp, _, fs in os.walk(d):
            files += [os.path.join(dp, f) for f in fs if f.endswith((".h", ".cuh", ".cu", ".cpp"))]
    files.append(os.path.abspath(__file__))
    return files


def _calls_includes() -> list[str]:
    """Include folders of the extension; raises FileNotFoundError, naming what is missing."""
    python = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(python, "Python.h")):
        raise FileNotFoundError("Python's headers are not installed")
    spec = importlib.util.find_spec("torch")  # for one header, DLPack's
    if spec is None or not spec.submodule_search_locations:
        raise FileNotFoundError("torch is not installed")
    torch = os.path.join(spec.submodule_search_locations[0], "include")
    header = os.path.join(torch, "ATen", "dlpack.h")
    if not os.path.exists(header):
        raise FileNotFoundError("torch has no ATen/dlpack.h")
    with open(header) as f:
        if "DLPackExchangeAPI" not in f.read():
            raise FileNotFoundError("torch's DLPack header has no exchange table")
    return [torch, python]


def up_to_date() -> bool:
    built = [LIB]
    try:
        _calls_includes()
        built.append(CALLS)
    except FileNotFoundError:
        pass
    if not all(os.path.exists(f) for f in built):
        return False
    t = min(os.path.getmtime(f) for f in built)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    tmp = LIB + ".tmp"
    cmds = [[
        nvcc(), "-std=c++17", "-O3", "-lineinfo", "-DNDEBUG",
        "-gencode", "arch=compute_100a,code=sm_100a",
        "-Xcompiler", "-fPIC,-O3,-fvisibility=hidden",
        "-Xptxas", "-v",
        "-I", INCLUDE, "-I", CSRC,
        "-shared", "-o", tmp,
    ] + SOURCES]
    res = subprocess.run(cmds[0], capture_output=True, text=True)
    out, failed = res.stdout + res.stderr, res.returncode != 0
    calls = False
    if not failed:
        os.replace(tmp, LIB)
        try:
            torch_include, python_include = _calls_includes()
            calls = True
        except FileNotFoundError as e:
            sys.stderr.write(f"_torch_calls.so is not built, the block-sparse calls need it: {e}\n")
            if os.path.exists(CALLS):  # made for another libkvp.so
                os.remove(CALLS)
    if calls:
        cmds.append([
            nvcc(), "-std=c++17", "-O3", "-gencode", "arch=compute_100a,code=sm_100a",
            "-Xcompiler", "-fPIC,-O3,-fvisibility=hidden", "-I", INCLUDE,
            "-I", torch_include, "-I", python_include,
            "-shared", "-o", CALLS + ".tmp", CALLS_SOURCE, "-L", PKG, "-l:libkvp.so",
            "-Xlinker", "-rpath", "-Xlinker", "$ORIGIN",
        ])
        res = subprocess.run(cmds[1], capture_output=True, text=True)
        out, failed = out + res.stdout + res.stderr, res.returncode != 0
    with open(os.path.join(BUILD_DIR, "nvcc.log"), "w") as f:
        f.write("\n".join(" ".join(c) for c in cmds) + "\n\n" + out)
    if failed:
        sys.stderr.write(out)
        raise RuntimeError("nvcc failed; see " + os.path.join(BUILD_DIR, "nvcc.log"))
    if calls:
        os.replace(CALLS + ".tmp", CALLS)
    if verbose:
        sys.stdout.write(out)
    return LIB


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose))


if __name__ == "__main__":
    main()
