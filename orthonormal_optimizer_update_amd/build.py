"""Build libortho.so in-tree with hipcc for gfx950, and with the host compiler the
binding of its calls over many tensors.

    python -m orthonormal_optimizer_update_amd.build

Every call recompiles all sources.  Both land next to this file, where ``api``
loads them from.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libortho.so")
BINDING = os.path.join(HERE, "_binding.so")

SOURCES = ["kernels_gemm.hip", "kernels_aux.hip", "kernels_stream.hip", "kernels_gram_ns.hip",
           "kernels_sweep.hip", "kernels_dion2.hip", "kernels_fp8_gemm.hip", "kernels_fp8_exact.hip",
           "kernels_fp8_few.hip", "kernels_fp8_rows.hip", "kernels_adamw.hip", "kernels_experts.hip",
           "noalloc.hip", "abi.cpp", "abi_fp8.cpp", "abi_adamw.cpp", "abi_experts.cpp", "plan.cpp"]

COMMON_FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-function",
    "--offload-arch=gfx950",
    # never emit packed-fp32 VALU instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # the unrolled epilogues index the accumulator arrays with constants only if
    # every loop over them is fully unrolled; the default size limit is too low
    "-mllvm", "-pragma-unroll-threshold=200000",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), *COMMON_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in res.stderr.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{err}")
    if err.strip():
        sys.stderr.write(err + "\n")
    return obj


def _run(what: str, cmd) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed: {' '.join(cmd)}\n{res.stderr}")


def _compile_binding() -> str:
    import torch
    root = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD, "binding.o")
    _run("compile", [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-Wno-attributes",
                     f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                     "-isystem", os.path.join(root, "include"),
                     "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
                     "-isystem", sysconfig.get_paths()["include"],
                     "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj])
    return obj


def _link_binding(obj: str) -> None:
    import torch
    tmp = BINDING + ".tmp"
    _run("link", [shutil.which("g++") or "g++", "-shared", "-o", tmp, obj,
                  "-L" + HERE, "-lortho", "-Wl,-rpath,$ORIGIN",
                  "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"])
    os.replace(tmp, BINDING)


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), "-shared", "-fPIC", "--offload-arch=gfx950", "-o", tmp, *objs]
    _run("link", cmd)
    os.replace(tmp, LIB)
    # (callers of the C-ABI need neither torch nor Python's headers nor the host compiler)
    try:
        _link_binding(binding.result())
    except Exception as e:
        if os.path.exists(BINDING):   # an older one may not fit this library
            os.remove(BINDING)
        raise RuntimeError(f"built {LIB}, but not its binding for Python: {e}") from e
    if verbose:
        print(f"built {LIB} and {BINDING}")
    return LIB


if __name__ == "__main__":
    build()
