"""Build libloki.so in-tree with nvcc for sm_100a.

    python sparse_attention_decode_loki_b200/build.py [--verbose] [--force]

(Run it as a file, not as `-m`: importing the package loads libloki.so, which
is what this script produces.)

Each .cu under csrc/ compiles to an object in _build/ (in parallel), then the
objects link into sparse_attention_decode_loki_b200/libloki.so with the CUDA
runtime linked statically; csrc/binding.cpp compiles to the extension module _binding beside it, for the interpreter and
the torch that run this script. ptxas resource usage (registers, spills, shared memory) of every kernel goes to
_build/ptxas.log.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libloki.so")
# Python's calls of the decode step's entries; its name says which interpreter loads it
BINDING = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
         "-Xptxas", "-v", "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    deps = [src] + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    deps.append(os.path.join(ROOT, "include", "loki.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    srcs = sources()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(pair):
        src, obj = pair
        if not force and not _stale(obj, src):
            return src, ""
        cmd = [nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return src, r.stderr

    logs = []
    workers = min(len(srcs), os.cpu_count() or 4)
    with concurrent.futures.ThreadPoolExecutor(workers) as ex:
        for src, log in ex.map(compile_one, zip(srcs, objs)):
            if log:
                logs.append(f"==== {os.path.basename(src)}\n{log}")
    if logs:
        with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
            f.write("\n".join(logs))
    if force or not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs):
        cmd = [nvcc, *ARCH, "-shared", "-o", LIB, *objs, "-Xcompiler", "-fPIC"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    build_binding(force)
    if verbose:
        print("\n".join(logs))
    return LIB


def build_binding(force: bool = False) -> None:
    """csrc/binding.cpp against this interpreter and its torch, next to libloki.so. It uses torch's C++ classes, so
    it is built anew whenever the torch, its ABI, the interpreter or the command differ from the last build's."""
    import torch  # for its headers' place and its ABI
    src, stamp = os.path.join(CSRC, "binding.cpp"), os.path.join(BUILD, "binding.stamp")
    home, abi = os.path.dirname(torch.__file__), int(torch.compiled_with_cxx11_abi())
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={abi}", src, "-o", BINDING,
           "-I", os.path.join(ROOT, "include"), "-isystem", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(home, "include"),
           "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(shutil.which(_nvcc()) or _nvcc())), "include"),
           "-L", PKG, "-l:libloki.so", "-L", os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-Wl,-rpath,$ORIGIN"]
    made_by = "\n".join([torch.__version__, str(abi), sys.version, *cmd])
    deps = [src, os.path.join(ROOT, "include", "loki.h")]
    if not force and os.path.exists(BINDING) and os.path.exists(stamp):
        with open(stamp) as f:
            same = f.read() == made_by
        if same and all(os.path.getmtime(d) <= os.path.getmtime(BINDING) for d in deps):
            return
    os.makedirs(BUILD, exist_ok=True)
    for old in (stamp, os.path.join(PKG, "_binding.so")):
        if os.path.exists(old):
            os.remove(old)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {src}:\n{r.stdout}\n{r.stderr}")
    with open(stamp, "w") as f:
        f.write(made_by)


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force="--force" in sys.argv))
