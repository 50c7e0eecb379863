"""Build libfs_sampling.so in-tree for sm_103a, and the decode step's compiled binding.

Each CUDA source is compiled to an object in parallel with nvcc
(-gencode arch=compute_103a,code=sm_103a), then linked into a shared library with
the CUDA runtime linked statically, so the library loads on a machine without a
GPU and without a CUDA runtime on the loader path.  It needs nothing but nvcc.  _decode.so, the
argument checks and marshalling of torch tensors for the decode step, is host C++ against torch's
headers; it is left out where torch is not installed.

    python -m min_sampling_gb300.build [--debug]
"""
from __future__ import annotations

import argparse
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
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfs_sampling.so")
DECODE = os.path.join(PKG, "_decode.so")
SOURCES = ["sampling.cu", "renorm.cu", "speculative.cu", "uniforms.cu", "paged_kv.cu", "prefix_attention.cu",
           "prefix_tensor.cu", "api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found (CUDA toolkit required to build libfs_sampling.so)")
    return path


def flags(debug: bool) -> list[str]:
    f = ARCH + ["-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
                "--expt-relaxed-constexpr"]
    f += ["-O0", "-G"] if debug else ["-O3"]
    return f


def run(cmd: list[str], what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")
    return None if spec is None else os.path.dirname(spec.origin)


def compile_binding() -> str | None:
    if torch_dir() is None:
        return None
    obj = os.path.join(BUILD, "decode_binding.o")
    include = [INCLUDE, os.path.join(torch_dir(), "include"), os.path.join(torch_dir(), "include/torch/csrc/api/include"),
               sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    run(["g++", "-O2", "-std=c++17", "-fPIC", "-c", os.path.join(CSRC, "decode_binding.cpp"), "-o", obj]
        + [f for i in include for f in ("-isystem" if "torch" in i else "-I", i)], "g++ on decode_binding.cpp")
    return obj


def link_binding(obj: str) -> None:
    """_decode.so finds libfs_sampling.so beside itself; torch's libraries are loaded by then."""
    lib = os.path.join(torch_dir(), "lib")
    run(["g++", "-shared", "-o", DECODE + ".tmp", obj, "-L", PKG, "-l:libfs_sampling.so", "-L", lib, "-ltorch_python",
         "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", "-Wl,--as-needed"], "linking _decode.so")
    os.replace(DECODE + ".tmp", DECODE)


def build(debug: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    objs = []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, "-c", os.path.join(CSRC, src), "-o", obj] + flags(debug)
        if ptxas_info:
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(compile_binding)
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [cc, "-shared", "-o", tmp] + objs + ARCH + ["-cudart", "static", "-Xcompiler", "-fPIC"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    obj = binding.result()   # the library is there whatever becomes of the binding
    if obj is None:
        sys.stderr.write("torch is not installed: _decode.so is left out\n")
    else:
        link_binding(obj)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--debug", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers / spills / shared memory")
    args = ap.parse_args()
    print(build(debug=args.debug, verbose=True, ptxas_info=args.ptxas_info))
