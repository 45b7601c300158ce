"""Build libmsa.so (the CUDA library) in-tree with nvcc for sm_103a, and
_paged_binding.so (the paged calls' Python binding) with the host compiler.

Each .cu under csrc/ compiles to an object in parallel; the objects link
into block_sparse_gqa_causal_gb300/libmsa.so, without torch.  The binding is
compiled against the torch that is installed and linked with libmsa.so; where
there is no torch it is left out, and where it fails libmsa.so is there already.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmsa.so")
BINDING = os.path.join(HERE, "_paged_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _stale(out: str, deps: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_commands(out: str):
    """The binding's source, its object (named by the versions it is compiled for) and the commands that make and link it;
    None without torch."""
    try:
        import torch
    except ImportError:
        return None
    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = [os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include"), os.path.join(ROOT, "include")]
    src = os.path.join(CSRC, "paged_binding.cpp")
    obj = os.path.join(BUILD, f"paged_binding-{torch.__version__}-py{sysconfig.get_python_version()}.o")
    cxx = os.environ.get("CXX") or shutil.which("g++") or "c++"
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={abi}", *["-I" + i for i in inc], "-c", src, "-o", obj]
    libs = os.path.join(at, "lib")
    link = [cxx, "-shared", "-o", out, obj, LIB, "-Wl,-rpath,$ORIGIN", "-L" + libs, "-Wl,-rpath," + libs, "-ltorch_python", "-ltorch",
            "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    return src, obj, compile_, link


def build(verbose: bool = False, ptxas_info: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(ROOT, "include", "msa.h"))
    objs = []
    jobs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj]
            if ptxas_info:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0 or verbose or ptxas_info:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed for {cmd[-3]}")

    binding = _binding_commands(BINDING + ".tmp")
    with ThreadPoolExecutor(max(1, min(len(jobs) + 1, os.cpu_count() or 4))) as ex:
        bjob = None
        if binding and (force or _stale(binding[1], [binding[0], headers[-1]])):
            bjob = ex.submit(run, binding[2])
        list(ex.map(run, jobs))
        if force or jobs or _stale(LIB, objs):
            tmp = LIB + ".tmp"
            run([nvcc(), *ARCH, "-shared", "-Xlinker", "-soname", "-Xlinker", os.path.basename(LIB), "-o", tmp, *objs])
            os.replace(tmp, LIB)
        if bjob:
            bjob.result()
    if binding and (bjob or _stale(BINDING, [binding[1], LIB])):
        run(binding[3])
        os.replace(BINDING + ".tmp", BINDING)
    return LIB


if __name__ == "__main__":
    build(verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv, force="--force" in sys.argv)
    print(LIB)
