"""Compile the HIP library libfp4w4a16.so for gfx950, in place (hipcc; no GPU needed), the native half of the
Python binding (_fp4bind.so) and the benchmark's measurement probes, libfp4probe.so (a separate library outside the C ABI)."""
from __future__ import annotations

import os
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libfp4w4a16.so")
BIND_LIB = os.path.join(HERE, "_fp4bind.so")
PROBE_LIB = os.path.join(HERE, "libfp4probe.so")
PROBE_SOURCES = ["probe.hip"]
BUILD_DIR = os.path.join(HERE, "_build")
SOURCES = ["api.hip", "layout.hip", "gemv.hip", "gemm.hip", "quantize.hip",
           "mx_quant.hip", "mx_gemv.hip", "mx_gemm.hip"]
ARCH = os.environ.get("FP4_OFFLOAD_ARCH", "gfx950")

FLAGS = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-I", INCLUDE, "-I", CSRC,
    # no packed FP32 instructions anywhere in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # the GEMV and mid-M kernels take their leading 8 arguments (at most 12 dwords) in preloaded
    # scalar registers, so that a wave's first loads do not wait on the kernel-argument memory
    "-mllvm", "-amdgpu-kernarg-preload-count=8",
    "-Wno-unused-command-line-argument",
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, src + ".o")
    cmd = ["hipcc", "-c", os.path.join(CSRC, src), "-o", obj] + FLAGS
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def _link(objs: list[str], lib: str) -> None:
    tmp = lib + f".tmp{os.getpid()}"
    r = subprocess.run(["hipcc", "-shared", "-fPIC", f"--offload-arch={ARCH}", "-o", tmp] + objs,
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib)


def _compile_binding() -> str:
    """The native half of the Python binding (host code only): links the installed torch and, by name, LIB."""
    import torch
    base = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD_DIR, "bind.cpp.o")
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], INCLUDE, os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include")]
    cmd = ["g++", "-c", os.path.join(CSRC, "bind.cpp"), "-o", obj, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1", "-DTORCH_EXTENSION_NAME=_fp4bind",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [a for i in inc for a in ("-isystem" if i != INCLUDE else "-I", i)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for bind.cpp:\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BIND_LIB + f".tmp{os.getpid()}"
    r = subprocess.run(["g++", "-shared", "-o", tmp, obj, "-L", HERE, "-lfp4w4a16", "-Wl,-rpath,$ORIGIN", "-L", libs, "-lc10",
                        "-lc10_hip", "-ltorch_cpu", "-ltorch", "-ltorch_python"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, BIND_LIB)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = SOURCES + PROBE_SOURCES
    with ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        bind = ex.submit(_compile_binding)
        objs = dict(zip(srcs, ex.map(_compile, srcs)))
        bind_obj = bind.result()
    _link([objs[s] for s in SOURCES], LIB)
    _link([objs[s] for s in PROBE_SOURCES], PROBE_LIB)
    _link_binding(bind_obj)
    if verbose:
        print(LIB)
        print(PROBE_LIB)
        print(BIND_LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
