"""Build step: compile the gfx950 HIP sources into the in-tree libfp8bs.so.

Run ``python -m fp8_block_scaled_05_amd.build`` (or ``__graft_entry__.build()``).
hipcc cross-compiles for gfx950 without a GPU present.
"""
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libfp8bs.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
MARSHAL_PATH = os.path.join(PKG, "_marshal.so")
SOURCES = ["status.cpp", "quant.hip", "dequant.hip", "tensor_quant.hip", "gemm.hip", "kv_append.hip", "kv_attention.hip", "moe.hip"]

# -packed-fp32-ops: no v_pk_{add,mul,fma}_f32 in the generated code.
# Division and sqrt stay correctly rounded (hipcc's default); no fast-math.
HIP_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def hipcc():
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libfp8bs)")


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    msgs = "\n".join(l for l in (res.stdout + res.stderr).splitlines()
                     if "packed-fp32-ops" not in l)
    if res.returncode != 0:
        raise RuntimeError(f"libfp8bs build failed:\n{msgs}")
    if verbose and msgs.strip():
        print(msgs, flush=True)


def build(verbose=False, extra_flags=()):
    """Each source is compiled by itself, a few at a time, and the objects are linked."""
    out_tmp = LIB_PATH + ".tmp"
    flags = [hipcc(), *HIP_FLAGS, *extra_flags]
    with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
        objs = [os.path.join(tmp, s + ".o") for s in SOURCES]
        list(pool.map(lambda so: _run([*flags, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, so[0]), "-o", so[1]], verbose),
                      zip(SOURCES, objs)))
        _run([*flags, "-shared", *objs, "-o", out_tmp], verbose)
    os.replace(out_tmp, LIB_PATH)
    _build_marshal(verbose)
    return LIB_PATH


def _build_marshal(verbose):
    """The CPython module that marshals PyTorch tensors onto the decoder layer's entry points (host code only).
    Callers of the C library need none of what it is built with: where that is missing, it is left out."""
    headers = sysconfig.get_paths()["include"]
    missing = [name for name, there in (("torch", importlib.util.find_spec("torch")), ("g++", shutil.which("g++")),
                                        ("Python.h", os.path.exists(os.path.join(headers, "Python.h")))) if not there]
    if missing:
        if os.path.exists(MARSHAL_PATH):       # of an earlier build: it need not fit the new library
            os.remove(MARSHAL_PATH)
        print(f"{MARSHAL_PATH} (the decoder layer's operators in Python) is not built: {', '.join(missing)} not found", flush=True)
        return
    import torch
    root = os.path.dirname(torch.__file__)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    out_tmp = MARSHAL_PATH + ".tmp"
    _run(["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-isystem", os.path.join(root, "include"),
          "-isystem", headers, "-isystem", os.path.join(rocm, "include"), "-I", INCLUDE,
          os.path.join(CSRC, "marshal.cpp"), "-o", out_tmp, "-L", PKG, "-lfp8bs", "-L", os.path.join(root, "lib"),
          "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN"], verbose)
    os.replace(out_tmp, MARSHAL_PATH)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
