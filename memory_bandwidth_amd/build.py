"""Compile the HIP library libq4gemv.so in-tree for gfx950, and the CPython
module _bind_i8, which calls its 8-bit entry points.

Each source under csrc/ is compiled with hipcc to an object in _build/, in
parallel, and the objects are linked into memory_bandwidth_amd/libq4gemv.so.
The module is host code against torch's headers, compiled with the host
compiler, and works with the Python and the torch it was built for: its name
has the one's tag, and it knows the other's version.
Run as ``python -m memory_bandwidth_amd.build`` (or through
``__graft_entry__.build()``).  Compiles every time it is called.
"""

from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libq4gemv.so")
BIND = os.path.join(HERE, "_bind_i8" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ["api.cpp", "gemv_q4.hip", "gemv_f32.hip", "dequant_q4.hip", "probes.hip", "gemv_blocks.hip",
           "scan2.hip", "quant_i8.hip", "gemm_i8.hip"]
ARCH = "gfx950"

# Packed-FP32 instructions stay off: the code never asks for them and the
# compiler must not form them on its own.
HIP_FLAGS = [
    "-O3", "-std=c++17", f"--offload-arch={ARCH}", "-fPIC", "-Wall",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    path = os.path.join(rocm, "bin", "hipcc")
    return path if os.path.exists(path) else "hipcc"


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), *HIP_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _compile_bind() -> str:
    import torch
    out = os.path.join(BUILD, os.path.basename(BIND))
    top = os.path.dirname(torch.__file__)
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DBUILT_FOR_TORCH="{torch.__version__}"',
           "-I", os.path.join(ROOT, "include"), "-I", os.path.join(top, "include"),
           "-I", os.path.join(top, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], os.path.join(CSRC, "bind_i8.cpp"), "-o", out,
           "-L", os.path.join(top, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
           f"-Wl,-rpath,{os.path.join(top, 'lib')}"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except FileNotFoundError as e:
        raise RuntimeError("g++, which compiles bind_i8.cpp, is not installed") from e
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for bind_i8.cpp:\n{r.stdout}\n{r.stderr}")
    return out


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    jobs = min(len(SOURCES) + 1, max(1, min(8, os.cpu_count() or 1)))
    with concurrent.futures.ThreadPoolExecutor(jobs) as ex:
        bind = ex.submit(_compile_bind)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    # The library and every call but the 8-bit ones need no module: a machine
    # that cannot compile it has them all the same.  A module built for another
    # library could call it wrongly, so an older one goes.
    try:
        os.replace(bind.result(), BIND)
    except Exception:
        if os.path.exists(BIND):
            os.remove(BIND)
        raise
    if verbose:
        print(f"built {BIND}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
