"""Build libmbt.so in-tree for sm_103a with nvcc (one process per translation
unit, in parallel, then one link) and the native part of the Python binding.
Usage: python -m memory_bound_transformer_gb300.build [--library]
The library needs nvcc alone. The extension also needs torch, Python's headers
and g++; --library leaves it out, and so does a Python without torch."""
from __future__ import annotations

import importlib.util
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


def _deps(src: str):
    """A source and every header it may include."""
    inc = os.path.join(os.path.dirname(PKG), "include")
    return [src] + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + [
        os.path.join(inc, f) for f in os.listdir(inc)]


def _older(target: str, deps) -> bool:
    """Whether a file is missing or older than one of those it is made from."""
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
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


def _binding_stamp(flags) -> str:
    """What the extension's binary interface hangs on besides its sources."""
    import torch
    return "\n".join([sys.version, torch.__version__, *flags[0], *flags[1]]) + "\n"


def _run(cmd):
    return cmd, subprocess.run(cmd, capture_output=True, text=True)


def _check(results, what: str, verbose: bool = False) -> None:
    bad = False
    for cmd, r in results:
        if verbose or r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode:
            bad = True
            sys.stderr.write("FAILED: " + " ".join(cmd) + "\n")
    if bad:
        raise RuntimeError(what + " failed")


def _link(cmd, out: str, what: str) -> None:
    """A linked file appears whole; where that fails the old one is gone."""
    if os.path.exists(out):
        os.remove(out)
    part = f"{out}.{os.getpid()}.part"
    try:
        _check([_run([*cmd, "-o", part])], what)
        os.replace(part, out)
    finally:
        if os.path.exists(part):
            os.remove(part)


def _compile_binding(flags, verbose: bool) -> str:
    """The extension's object, for this Python and this torch."""
    src, obj, stamp = os.path.join(CSRC, "binding.cpp"), os.path.join(OBJ, "binding.o"), os.path.join(OBJ, "binding.stamp")
    want = _binding_stamp(flags)
    same = os.path.exists(stamp) and open(stamp).read() == want
    if not same or _older(obj, _deps(src)):
        for f in (stamp, obj, BINDING):                    # what a failure leaves missing is made the next time
            if os.path.exists(f):
                os.remove(f)
        _check([_run(["g++", *flags[0], "-c", src, "-o", obj])], "g++", verbose)
        with open(stamp, "w") as f:
            f.write(want)
    return obj


def build(verbose: bool = False, ptxas_info: bool = False, library_only: bool = False) -> str:
    """Makes what is missing or out of date; the library's path. A failure of the extension leaves the library made."""
    os.makedirs(OBJ, exist_ok=True)
    cc = nvcc()
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(OBJ, src.replace(".cu", ".o"))
        if _older(o, _deps(s)) or ptxas_info:
            cmd = [cc, *ARCH, *FLAGS, "-c", s, "-o", o]
            if ptxas_info:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)
    flags = None
    if not library_only:
        if importlib.util.find_spec("torch"):
            flags = _binding_flags()
        else:
            sys.stderr.write("no torch: the Python extension is left out\n")
    with ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 4))) as ex:
        binding = ex.submit(_compile_binding, flags, verbose) if flags else None
        _check(list(ex.map(_run, jobs)), "nvcc", verbose or ptxas_info)
    objs = [os.path.join(OBJ, s.replace(".cu", ".o")) for s in SOURCES]
    if _older(LIB, objs):
        if os.path.exists(BINDING):                        # it calls the library by the old one's signatures
            os.remove(BINDING)
        _link([cc, *ARCH, "-shared", *objs, "-lcudart"], LIB, "link")
    if binding:
        bobj = binding.result()
        if _older(BINDING, [bobj, LIB]):
            _link(["g++", "-shared", bobj, *flags[1]], BINDING, "link of the binding")
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="--ptxas" in sys.argv, library_only="--library" in sys.argv))
