"""Build libpagedattn.so (hand-written CUDA for sm_103a) and the Python
extension that calls it (pa_binding.so) in-tree.

    python -m paged_kv_cache_174_gb300.build [--force] [--verbose]

Each translation unit is compiled with nvcc in parallel, then linked into a
shared library with the CUDA runtime linked statically, so the library needs
only the NVIDIA driver at run time.  The extension is host code on torch's and
Python's headers, linked to the library beside it.  Output: paged_kv_cache_174_gb300/_build/.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libpagedattn.so"
LIB = os.path.join(OUT_DIR, LIB_NAME)

SOURCES = ["pa_api.cu", "pa_cache.cu", "pa_decode.cu", "pa_decode_fp8.cu", "pa_decode_fused.cu",
           "pa_prefill.cu", "pa_prefill_fp8.cu", "pa_graph.cu", "pa_step.cu", "pa_rotary.cu",
           "pa_decode_window.cu", "pa_decode_window_fp8.cu", "pa_prefill_window.cu",
           "pa_prefill_window_fp8.cu", "pa_long_api.cu", "pa_blocks.cu", "pa_sparse.cu",
           "pa_weights.cu", "pa_weights_chunk.cu", "pa_evict.cu"]
BINDING_SOURCE = "pa_binding.cpp"
BINDING_NAME = "pa_binding.so"
BINDING = os.path.join(OUT_DIR, BINDING_NAME)
STAMP_NAME = "pa_binding.made_for"  # the torch and the Python of the last extension
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    env = os.environ.get("NVCC")
    if env:
        return env
    found = shutil.which("nvcc")
    if found:
        return found
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found (set NVCC or put CUDA's bin on PATH)")


def _headers():
    hs = [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    hs += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    return hs


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_dir() -> Optional[str]:
    """torch's folder, found without importing it; None where there is no torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    return list(spec.submodule_search_locations)[0]


def _made_for(torch_dir: str) -> str:
    """What the extension's headers and ABI come from."""
    with open(os.path.join(torch_dir, "version.py")) as f:
        return "\n".join([sys.version, torch_dir, f.read()])


def _read(path: str) -> Optional[str]:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return None


def _run(cmd, verbose: bool):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"command failed ({r.returncode}): {' '.join(cmd)}\n{r.stderr}")
    return r


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile and link; returns the path of the shared library.  Where there is no
    torch, the library alone (the Python package cannot be used there)."""
    os.makedirs(OUT_DIR, exist_ok=True)
    cc = nvcc()
    headers = _headers()
    objs, jobs = [], []
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
        objs.append(obj)
        if force or ptxas_verbose or _stale(obj, [path] + headers):
            cmd = [cc] + ARCH + CFLAGS + (["-Xptxas", "-v"] if ptxas_verbose else []) + [
                "-c", path, "-o", obj]
            jobs.append(cmd)
    binding_src = os.path.join(CSRC, BINDING_SOURCE)
    binding_obj = os.path.join(OUT_DIR, BINDING_SOURCE.replace(".cpp", ".o"))
    torch_dir = _torch_dir()
    stamp = os.path.join(OUT_DIR, STAMP_NAME)
    made_for = _made_for(torch_dir) if torch_dir else None
    if not torch_dir:
        sys.stderr.write(f"torch not found: {LIB_NAME} is built without {BINDING_NAME}\n")
    elif force or _stale(binding_obj, [binding_src, os.path.join(INCLUDE, "pagedattn.h")]) or \
            _read(stamp) != made_for:
        inc = os.path.join(torch_dir, "include")
        jobs.append(["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE, "-isystem", inc,
                     "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem",
                     os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))),
                                  "include"),
                     "-isystem", sysconfig.get_paths()["include"], "-c", binding_src, "-o",
                     binding_obj])
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            list(ex.map(lambda c: _run(c, verbose or ptxas_verbose), jobs))
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp"
        _run([cc] + ARCH + ["-shared", "-Xlinker", "-soname=" + LIB_NAME, "-o", tmp] + objs,
             verbose)
        os.replace(tmp, LIB)
    if torch_dir and (force or jobs or _stale(BINDING, [binding_obj, LIB])):
        tmp = BINDING + ".tmp"
        torch_lib = os.path.join(torch_dir, "lib")
        _run(["g++", "-shared", "-o", tmp, binding_obj, LIB, "-L", torch_lib, "-ltorch_python",
              "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN",
              "-Wl,-rpath," + torch_lib], verbose)
        os.replace(tmp, BINDING)
        with open(stamp, "w") as f:
            f.write(made_for)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv,
                ptxas_verbose="--ptxas" in sys.argv))
