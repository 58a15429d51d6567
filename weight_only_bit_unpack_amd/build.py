"""Build libw4.so (gfx950) in-tree with hipcc.

    python weight_only_bit_unpack_amd/build.py

Every source of the library under csrc/ is compiled for gfx950 only; the objects
go to csrc/_build/ and the shared library to this package directory, where the
binding loads it from.  The MX operators' part of the binding, _w4mx, is host
code and is built beside it.
"""

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(CSRC, "_build")
LIB = os.path.join(PKG, "libw4.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

SOURCES = ["w4_api.cpp", "w4_quantize.hip", "w4_dequant.hip", "w4_gemv.hip", "w4_gemm.hip",
           "w4_workspace.cpp", "w4_fit.hip", "w4_noalloc.hip", "w4_mx_api.cpp", "w4_mx_quant.hip",
           "w4_mx_gemm.hip", "w4_mx_skinny.hip", "w4_mx_bf16_api.cpp", "w4_mx_bf16.hip",
           "w4_mx_bf16_gemm.hip", "w4_mx_bf16_skinny.hip", "w4_mx_bf16_narrow.hip",
           "w4_counters.cpp"]

CFLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # IEEE arithmetic: no contraction of separate multiplies and adds
    "-ffp-contract=off",
    # keep packed-fp32 instructions out of the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
    "-I", os.path.join(ROOT, "include"),
    "-I", CSRC,
]


def _compile(src):
    obj = os.path.join(OBJ, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *CFLAGS]
    if src.endswith(".cpp"):
        cmd += ["-x", "hip"]
    cmd += ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


# Measurement context for the benchmark only (a plain streaming read); its
# own library so that nothing of it is in libw4.
CTX_SOURCES = ["ctx_read.hip"]
CTX_LIB = os.path.join(PKG, "libw4ctx.so")


# The MX operators' Python binding: host code against torch's C++ headers,
# linked to libw4.so beside it.
BINDING = "w4_mx_binding.cpp"
BINDING_LIB = os.path.join(PKG, "_w4mx.so")
CXX = os.environ.get("CXX", "g++")


def _build_binding():
    import sysconfig
    import torch
    base = os.path.dirname(torch.__file__)
    inc = [sysconfig.get_paths()["include"], os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include"),
           os.path.join(ROOT, "include")]
    lib = os.path.join(base, "lib")
    tmp = BINDING_LIB + ".tmp"
    cmd = [CXX, "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *[f"-isystem{i}" for i in inc], os.path.join(CSRC, BINDING), "-o", tmp,
           LIB, f"-L{lib}", "-lc10", "-ltorch_cpu", "-ltorch", "-ltorch_python",
           "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        error = r.stderr if r.returncode != 0 else None
    except OSError as e:  # no such compiler
        error = str(e)
    if error is not None:
        raise RuntimeError(f"{CXX} failed for {BINDING}, without which the MX operators' calls fail (the "
                           f"codecs work: {os.path.basename(LIB)} is built):\n{error}")
    os.replace(tmp, BINDING_LIB)


def _link(objs, lib):
    tmp = lib + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp,
           f"-Wl,-soname,{os.path.basename(lib)}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib)


def build(verbose=False):
    os.makedirs(OBJ, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(8, len(SOURCES) + len(CTX_SOURCES))) as ex:
        objs = list(ex.map(_compile, SOURCES + CTX_SOURCES))
    _link(objs[:len(SOURCES)], LIB)
    _link(objs[len(SOURCES):], CTX_LIB)
    _build_binding()
    if verbose:
        print(f"built {LIB}, {CTX_LIB} and {BINDING_LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
