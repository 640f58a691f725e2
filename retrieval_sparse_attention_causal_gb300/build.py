"""Builds libgca.so (the CUDA library behind include/gca.h) for sm_103a, in-tree, and the
Python extension that binds its decoding operators to PyTorch tensors.

Each translation unit is compiled by its own process (in parallel), then linked into the
two shared libraries under retrieval_sparse_attention_causal_gb300/_build/.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libgca.so")
EXT = os.path.join(BUILD, "_gca_decoding.so")
SOURCES = ["api.cu", "retrieve.cu", "gca_fwd.cu", "gca_bwd.cu", "scores_bwd.cu", "noalloc.cu", "tmap.cu", "gca_bwd_tc.cu",
           "gather.cu", "block_attn.cu", "window_bwd.cu", "encoder.cu", "retrieve_tc.cu", "rotary.cu", "tree_attn.cu",
           "tree_rows.cu", "tree_tc.cu", "cache.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the GCA library needs the CUDA toolkit to build")


def _stale(obj, src):
    if not os.path.exists(obj):
        return True
    deps = [src] + [os.path.join(CSRC, h) for h in os.listdir(CSRC) if h.endswith((".cuh", ".h"))]
    deps.append(os.path.join(ROOT, "include", "gca.h"))
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_dir():
    """Where torch's headers and libraries are, found without importing it."""
    return list(importlib.util.find_spec("torch").submodule_search_locations)[0]


def _binding_made_for():
    """What the Python extension fits besides its source: this torch and this Python."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f"{_torch_dir()}\n{f.read()}\n{sys.version}\n"


def _read(path):
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def _binding(obj):
    """Compile command of the Python extension, and its link command."""
    torch = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [os.path.join(ROOT, "include"), os.path.join(torch, "include"),
           os.path.join(torch, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include"),
           sysconfig.get_paths()["include"]]
    cxx = os.environ.get("CXX", "g++")
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *(f"-I{d}" for d in inc), "-c",
                os.path.join(CSRC, "binding.cpp"), "-o", obj]
    link = [cxx, "-shared", "-o", EXT, obj, f"-L{os.path.join(torch, 'lib')}", "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-lc10", "-lc10_cuda", f"-L{BUILD}", "-lgca", "-Wl,-rpath,$ORIGIN"]
    return compile_, link


def build(verbose: bool = False, extra_flags=None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    flags = FLAGS + list(extra_flags or [])
    jobs = []
    for s in SOURCES:
        src = os.path.join(CSRC, s)
        obj = os.path.join(BUILD, s.replace(".cu", ".o"))
        if _stale(obj, src) or extra_flags:
            jobs.append([nvcc, *ARCH, *flags, "-c", src, "-o", obj])
    cuda_jobs = bool(jobs)
    bind_obj = os.path.join(BUILD, "binding.o")
    bind_for = os.path.join(BUILD, "binding.txt")
    compile_binding, link_binding = _binding(bind_obj)
    made_for = _binding_made_for()
    bind_job = _stale(bind_obj, os.path.join(CSRC, "binding.cpp")) or _read(bind_for) != made_for

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode:
            raise RuntimeError(f"compiler failed: {' '.join(cmd)}")
        return r

    if bind_job and os.path.exists(bind_for):
        os.remove(bind_for)  # written again when the extension is linked
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        bound = ex.submit(run, compile_binding) if bind_job else None
        list(ex.map(run, jobs))
    objs = [os.path.join(BUILD, s.replace(".cu", ".o")) for s in SOURCES]
    if cuda_jobs or not os.path.exists(LIB):
        run([nvcc, *ARCH, "-shared", "-o", LIB, *objs])
    if bound:
        bound.result()  # raised here: the C library is there without the extension too
    if bind_job or not os.path.exists(EXT):
        run(link_binding)
        with open(bind_for, "w") as f:
            f.write(made_for)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
