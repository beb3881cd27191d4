"""Build libmx.so (HIP, gfx950) and the binding _bind.so in-tree.

Every .hip source under csrc/ is compiled with hipcc to its own object (in
parallel) and linked into ``mx_block_scaled_quantize_amd/libmx.so``.  hipcc
cross-compiles for gfx950 without a GPU present.  csrc/bind.cpp is host code
against Python's and torch's headers, compiled with g++ into ``_bind.so``.
"""

import concurrent.futures
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmx.so")
BIND = os.path.join(PKG, "_bind.so")
ARCH = "gfx950"

# Device code keeps FP32 denormals (the default) and never contracts a*b+c into
# an FMA, so every FP32 step rounds exactly where the algorithm says.  Packed
# FP32 instructions are disabled for the device target.
FLAGS = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def _hipcc():
    for c in ("/opt/rocm/bin/hipcc", "hipcc"):
        if os.path.exists(c) or c == "hipcc":
            return c
    raise RuntimeError("hipcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))


def _compile(src):
    obj = os.path.join(BUILD, os.path.basename(src)[:-4] + ".o")
    cmd = [_hipcc(), *FLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_bind():
    import torch
    root = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD, "bind.o")
    _run(["g++", "-std=c++17", "-O2", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          f"-I{root}/include", f"-I{root}/include/torch/csrc/api/include", "-I/opt/rocm/include",
          f"-I{sysconfig.get_paths()['include']}", "-c", os.path.join(CSRC, "bind.cpp"), "-o", obj], "g++ bind.cpp")
    return obj, os.path.join(root, "lib")


def build(verbose=False):
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        bind = ex.submit(_compile_bind)
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + ".tmp"
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    # libmx is there even if the binding cannot be built.  torch's libraries are loaded before the binding is; libmx
    # lies beside it
    bind_obj, torch_lib = bind.result()
    tmp = BIND + ".tmp"
    _run(["g++", "-shared", "-o", tmp, bind_obj, f"-L{PKG}", "-lmx", f"-L{torch_lib}", "-ltorch_python", "-ltorch_cpu",
          "-lc10", "-lc10_hip", "-lamdhip64", "-Wl,-rpath,$ORIGIN"], "link of _bind.so")
    os.replace(tmp, BIND)
    if verbose:
        print(f"built {LIB} and {BIND}", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
