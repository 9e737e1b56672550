"""Build the CUDA library (csrc/*.cu -> _build/libigconv.so) in-tree with nvcc
for sm_103a.  Only the C-ABI symbols (conv_*) are exported; the CUDA runtime is
linked statically and kept local to the library.  Beside it the native binding
of train.py (csrc/native.cpp -> _build/_igconv_native.so, g++ against torch's
headers)."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
SO = os.path.join(BUILD, "libigconv.so")
NATIVE_SRC = os.path.join(CSRC, "native.cpp")
NATIVE = os.path.join(BUILD, "_igconv_native.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + [NATIVE_SRC] + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def up_to_date() -> bool:
    if not os.path.exists(SO) or not os.path.exists(NATIVE):
        return False
    t = min(os.path.getmtime(SO), os.path.getmtime(NATIVE))
    return all(os.path.getmtime(d) <= t for d in _deps())


def compile_native(cc: str) -> str:
    """csrc/native.cpp (host C++ against torch's headers and Python's) -> an object file."""
    import sysconfig

    import torch

    obj = os.path.join(BUILD, "native.cpp.o")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", INCLUDE]
    for d in (inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"], cuda):
        cmd += ["-isystem", d]
    r = subprocess.run(cmd + ["-c", NATIVE_SRC, "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on native.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def link_native(obj: str) -> None:
    import torch

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = NATIVE + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", BUILD, "-l:libigconv.so", "-L", libs,
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the native binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, NATIVE)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and up_to_date():
        return SO
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                    "-I", CSRC, "--expt-relaxed-constexpr"]
    if ptxas_info:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc] + flags + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        native = ex.submit(compile_native, cc)
        results = list(ex.map(compile_one, srcs))
        native_obj = native.result()
    if verbose or ptxas_info:
        for _, err in results:
            if err:
                sys.stderr.write(err)
    vers = os.path.join(BUILD, "exports.map")
    with open(vers, "w") as f:
        f.write("{ global: conv_*; local: *; };\n")
    tmp = SO + f".tmp{os.getpid()}"
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results] + [
        "-Xlinker", f"--version-script={vers}", "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, SO)
    link_native(native_obj)
    return SO


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas-info" in sys.argv))
