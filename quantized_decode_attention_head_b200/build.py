"""Build librq.so in-tree with nvcc for sm_100a.

Usage: python -m quantized_decode_attention_head_b200.build [--verbose-ptxas]
"""

from __future__ import annotations

import os
import re
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "librq.so")
# the decode kernel is instantiated once per (head_dim, GQA group) pair in its
# own translation unit, so the units compile in parallel
SOURCES = ["rq_alloc.cpp", "rq_host.cpp", "rq_quantize.cu", "rq_decode.cu", "rq_paged_host.cpp",
           "rq_paged_append.cu", "rq_paged_decode.cu", "rq_paged_prompt.cu"] + [
    f"rq_decode_{d}x{g}.cu" for d in (128, 64) for g in (1, 2, 4, 8)]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _flags(ptxas_verbose=False):
    f = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    f += ARCH
    if ptxas_verbose:
        f += ["-Xptxas", "-v"]
    return f


def _deps(path, seen):
    """path and the headers of this repository that it includes, all levels."""
    if path not in seen:
        seen.append(path)
        with open(path) as f:
            for name in re.findall(r'^#include "([^"]+)"', f.read(), re.M):
                for folder in (CSRC, os.path.join(ROOT, "include")):
                    if os.path.exists(os.path.join(folder, name)):
                        _deps(os.path.join(folder, name), seen)
    return seen


def _compile(src, ptxas_verbose):
    obj = os.path.join(OBJ, src + ".o")
    path = os.path.join(CSRC, src)
    deps = _deps(path, [])
    if not ptxas_verbose and os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(d) for d in deps):
        return obj, ""
    cmd = [_nvcc(), "-c", path, "-o", obj] + _flags(ptxas_verbose)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def build(ptxas_verbose: bool = False, quiet: bool = True) -> str:
    os.makedirs(OBJ, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 4)) as ex:
        results = list(ex.map(lambda s: _compile(s, ptxas_verbose), SOURCES))
    objs = [o for o, _ in results]
    logs = "".join(l for _, l in results)
    if ptxas_verbose or not quiet:
        sys.stderr.write(logs)
    newest = max(os.path.getmtime(o) for o in objs)
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < newest:
        cmd = [_nvcc(), "-shared", "-o", LIB] + objs + ARCH + ["-Xcompiler", "-fPIC", "-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    return LIB


if __name__ == "__main__":
    print(build(ptxas_verbose="--verbose-ptxas" in sys.argv, quiet=False))
