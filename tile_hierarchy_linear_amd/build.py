"""Build libthl.so (HIP kernels for gfx950 + host C++) in-tree with hipcc, and
_torch_ops.so (host C++ only) where a torch with its HIP libraries is."""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(os.path.dirname(HERE), "_build")
LIB = os.path.join(HERE, "libthl.so")
TORCH_OPS = os.path.join(HERE, "_torch_ops.so")
PROBE_LIB = os.path.join(HERE, "libthl_probe.so")
SOURCES = ["gemm.hip", "layout.cpp", "gemm_inst_bf16.hip", "gemm_inst_f16.hip", "gemm_inst_i8.hip",
           "gemm_inst_e4m3.hip", "gemm_inst_e2m1.hip", "gemm_inst_bf16_ops.hip", "gemm_inst_f16_ops.hip",
           "gemm_inst_skinny.hip", "gemm_inst_e5m2.hip",
           "gemm_inst_mx8.hip", "gemm_inst_mx8e5.hip", "gemm_inst_mx8mix.hip", "gemm_inst_e4e5.hip",
           "gemm_inst_e5e4.hip", "gemm_inst_mxout16.hip", "gemm_inst_mxout8.hip", "convert.hip",
           "norm.hip", "moe.hip", "w4.hip"]
HEADERS = ["convert.hpp", "gemm_args.hpp", "gemm_kernels.hpp", "gemm_launch.hpp", "gemm_skinny.hpp", "host_checks.hpp",
           "index_maps.hpp", "layout.hpp", "rows.hpp"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
# Packed fp32 VALU instructions are switched off for every HIP compile.
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-result",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def build_torch_ops() -> None:
    """The torch-tensor forms: links torch's Python and C++ libraries and libthl.so beside it."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return
    torch = list(spec.submodule_search_locations)[0]
    if not os.path.exists(os.path.join(torch, "lib", "libc10_hip.so")):  # a torch without GPUs: no tensors to take
        if os.path.exists(TORCH_OPS):  # built for another torch
            os.remove(TORCH_OPS)
        return
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(HIPCC)))
    tmp = TORCH_OPS + ".tmp"
    subprocess.check_call(
        [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1",
         "-DUSE_ROCM=1", "-isystem", os.path.join(torch, "include"), "-isystem", os.path.join(rocm, "include"),
         "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "torch_ops.cpp"), "-o", tmp,
         "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip", "-L" + HERE,
         "-l:libthl.so", "-Wl,-rpath,$ORIGIN"])
    # a symbol that torch does not export shows here, not at a user's first call
    load = f"import ctypes, os, torch; ctypes.CDLL({os.path.abspath(tmp)!r}, os.RTLD_NOW)"
    subprocess.check_call([sys.executable, "-c", load])
    os.replace(tmp, TORCH_OPS)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, src + ".o")
        objs.append(obj)
        lang = ["-x", "hip"] if src.endswith(".hip") else []
        cmd = [HIPCC] + FLAGS + lang + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                            text=True)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        lines = [l for l in out.splitlines() if "not a recognized feature" not in l]
        if lines and (verbose or p.returncode):
            print("\n".join(lines), file=sys.stderr)
        if p.returncode:
            failed.append(src)
    if failed:
        raise RuntimeError(f"hipcc failed on {failed}")
    tmp = LIB + ".tmp"
    subprocess.check_call([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC"] + objs + ["-o", tmp])
    os.replace(tmp, LIB)
    build_torch_ops()
    # the measurement probe, a library of its own outside the GEMM boundary
    tmp = PROBE_LIB + ".tmp"
    subprocess.check_call([HIPCC] + FLAGS + ["-shared", "-x", "hip", os.path.join(CSRC, "mfma_probe.hip"), "-o", tmp],
                          stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)
    os.replace(tmp, PROBE_LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
