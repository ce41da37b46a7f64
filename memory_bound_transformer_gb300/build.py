"""Build libmbt.so in-tree for sm_103a with nvcc (one process per translation
unit, in parallel, then one link) and the native part of the Python binding. Usage: python -m memory_bound_transformer_gb300.build"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmbt.so")
BINDING = os.path.join(PKG, "_binding.so")
SOURCES = ["gemv.cu", "misc.cu", "attention.cu", "tc_gemm.cu", "tc_stream.cu", "sampling.cu", "runtime.cu", "ops.cu",
           "ops_noalloc.cu", "kv_fp4.cu", "attention_fp4.cu", "prompt_attention.cu",
           "ops_fp4.cu", "kv_extend.cu", "block_select.cu", "attention_blocks.cu", "ops_blocks.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(src: str, obj: str) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    deps = [src] + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    deps += [os.path.join(PKG, "..", "include", f) for f in os.listdir(os.path.join(PKG, "..", "include"))]
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_flags():
    """Compiler and linker flags of the Python extension, for the torch and the Python that run this."""
    import sysconfig
    import torch
    at = os.path.dirname(os.path.abspath(torch.__file__))
    lib, inc = os.path.join(at, "lib"), [os.path.join(at, "include"), os.path.join(at, "include/torch/csrc/api/include"),
                                         sysconfig.get_paths()["include"],
                                         os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    return (["-O2", "-std=c++17", "-fPIC", *(f"-I{i}" for i in inc)],
            [f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python", f"-L{PKG}", "-lmbt", "-Wl,-rpath,$ORIGIN"])


def build(verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    cc = nvcc()
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(OBJ, src.replace(".cu", ".o"))
        if _stale(s, o) or ptxas_info:
            cmd = [cc, *ARCH, *FLAGS, "-c", s, "-o", o]
            if ptxas_info:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)

    bsrc, bobj = os.path.join(CSRC, "binding.cpp"), os.path.join(OBJ, "binding.o")
    compile_flags, link_flags = _binding_flags()
    nvcc_jobs = len(jobs)
    if _stale(bsrc, bobj):
        jobs.insert(0, ["g++", *compile_flags, "-c", bsrc, "-o", bobj])
    rebind = len(jobs) > nvcc_jobs

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        results = list(ex.map(run, jobs))
    failed = False
    for cmd, r in results:
        if verbose or ptxas_info or r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode:
            failed = True
            sys.stderr.write("FAILED: " + " ".join(cmd) + "\n")
    if failed:
        raise RuntimeError("nvcc failed")
    objs = [os.path.join(OBJ, s.replace(".cu", ".o")) for s in SOURCES]
    if nvcc_jobs or not os.path.exists(LIB):
        link = [cc, *ARCH, "-shared", "-o", LIB, *objs, "-lcudart"]
        r = subprocess.run(link, capture_output=True, text=True)
        if r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed")
    if rebind or not os.path.exists(BINDING):
        r = subprocess.run(["g++", "-shared", bobj, "-o", BINDING, *link_flags], capture_output=True, text=True)
        if r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link of the binding failed")
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="--ptxas" in sys.argv))
