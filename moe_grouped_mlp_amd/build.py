"""Build libmoe_gmlp.so (gfx950) in-tree with hipcc.

    python -m moe_grouped_mlp_amd.build      # or __graft_entry__.build()

Every HIP source is compiled for gfx950 only, with packed-fp32 instruction
selection switched off, then linked into one shared library next to this
file, and with it, where torch is installed, _call.so, the compiled part of the
Python binding.  Objects go to moe_grouped_mlp_amd/_build/.  The library itself
needs no torch: `python moe_grouped_mlp_amd/build.py` builds it without.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmoe_gmlp.so")
CALL = os.path.join(HERE, "_call.so")   # Python's way into the smaller calls

SOURCES = ["api.cpp", "route.hip", "router.hip", "unfused.hip", "permute.hip", "quant.hip", "gemm.hip", "gemm_store.hip",
           "gemm_glu_bf16.hip", "gemm_glu_mx.hip", "gemm_dglu_bf16.hip", "gemm_dglu_mx.hip", "gemm_wgrad.hip",
           "gemm_store_mx4.hip", "gemm_glu_mx4.hip", "gemm_dglu_mx4.hip", "gemm_wgrad_mx4.hip",
           "noalloc.hip",
           "api_step.cpp", "fp8_quant.hip", "fp8_gemm.hip", "fp8_wgrad.hip", "fp8_gemm_rows.hip",
           "router_loss.hip", "grad.hip",
           "gate.hip", "adamw.hip", "int8_quant.hip", "int8_gemm.hip", "int8_gemm_rows.hip",
           "router_route.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
COMMON = [
    f"--offload-arch={ARCH}", "-O3", "-fPIC", "-std=c++17",
    "-Wall", "-Wno-unused-function",
    # never select packed fp32 VALU instructions (v_pk_{add,mul,fma}_f32)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *COMMON, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass does not know the device-only feature: drop that note
    err = "\n".join(l for l in r.stderr.splitlines()
                    if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{err}")
    if err.strip():
        sys.stderr.write(err + "\n")
    return obj


def _compile_call() -> str | None:
    """csrc/py_call.cpp, host code on CPython's and torch's headers; None
    where torch is not installed."""
    import sysconfig

    try:
        import torch  # noqa: F401
    except ModuleNotFoundError:
        return None
    from torch.utils import cpp_extension
    obj = os.path.join(BUILD, "py_call.o")
    cmd = [HIPCC, "-x", "c++", "-O2", "-fPIC", "-std=c++17", "-Wall", "-fvisibility=hidden",
           *(f"-I{p}" for p in (sysconfig.get_paths()["include"], *cpp_extension.include_paths())),
           "-c", os.path.join(CSRC, "py_call.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling py_call.cpp failed:\n{r.stderr}")
    return obj


def _link_call(obj: str) -> None:
    from torch.utils import cpp_extension
    libs = cpp_extension.library_paths()
    tmp = CALL + ".tmp"
    cmd = [HIPCC, "-no-hip-rt", "-shared", "-fPIC", "-o", tmp, obj, f"-L{HERE}",
           f"-l:{os.path.basename(LIB)}", "-Wl,-rpath,$ORIGIN",
           *(f"-L{p}" for p in libs), *(f"-Wl,-rpath,{p}" for p in libs),
           "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, CALL)


def build(verbose: bool = True) -> str:
    if shutil.which(HIPCC) is None and not os.path.exists(HIPCC):
        raise RuntimeError(f"hipcc not found ({HIPCC})")
    os.makedirs(BUILD, exist_ok=True)
    jobs = min(len(SOURCES), int(os.environ.get("MAX_JOBS", "8")))
    with cf.ThreadPoolExecutor(jobs) as ex:
        call = ex.submit(_compile_call)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    obj = call.result()
    if obj is not None:
        _link_call(obj)
    elif os.path.exists(CALL):
        os.remove(CALL)   # of an older library
    if verbose:
        print(f"built {LIB}\n" + (f"built {CALL}" if obj else "no _call.so: torch, which the Python binding needs, is not installed"))
    return LIB


if __name__ == "__main__":
    build()
