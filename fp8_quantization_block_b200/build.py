"""Build libmx.so (sm_100a) in-tree with nvcc.

    python -m fp8_quantization_block_b200.build [--force]
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmx.so")
UNITS = [os.path.join(CSRC, f) for f in ("mx_api.cu", "mx_experts.cu")]
OBJ = os.path.join(PKG, "_build")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
]


def _headers():
    out = [os.path.join(ROOT, "include", "mx.h")]
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".cuh", ".h")):
            out.append(os.path.join(CSRC, f))
    return out


def _sources():
    return _headers() + UNITS


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in _sources())


def _included(path: str, seen: set) -> set:
    """Files of this repository that a source includes, directly or not."""
    for line in open(path, encoding="utf-8"):
        if line.startswith('#include "'):
            name = line.split('"')[1]
            for d in (CSRC, os.path.join(ROOT, "include")):
                f = os.path.join(d, name)
                if os.path.exists(f) and f not in seen:
                    seen.add(f)
                    _included(f, seen)
    return seen


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the translation units (those whose sources changed, side by side), then link libmx.so."""
    if force or needs_build():
        nvcc = os.environ.get("NVCC", "nvcc")
        os.makedirs(OBJ, exist_ok=True)
        running = []
        objects = []
        for unit in UNITS:
            obj = os.path.join(OBJ, os.path.basename(unit) + ".o")
            objects.append(obj)
            if not force and os.path.exists(obj) and os.path.getmtime(obj) > max(
                    os.path.getmtime(f) for f in {unit, *_included(unit, set())}):
                continue
            cmd = [nvcc, *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-c", unit, "-o", obj + ".tmp"]
            if verbose:
                print(" ".join(cmd), flush=True)
            running.append((cmd, obj, subprocess.Popen(cmd)))
        failed = [cmd for cmd, _, p in running if p.wait() != 0]
        if failed:
            raise subprocess.CalledProcessError(1, failed[0])
        for _, obj, _ in running:
            os.replace(obj + ".tmp", obj)
        cmd = [nvcc, *NVCC_FLAGS, "-shared", *objects, "-o", LIB + ".tmp"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
