"""Builds libfp8opt.so in-tree (bit_optimizer_gb300/_build) with nvcc for
sm_103a: one object per .cu file, compiled in parallel, then linked.  Beside
it, fp8opt_binding.so: the PyTorch binding of the training operators (g++,
against the installed torch).

Flags that matter for results: ``-fmad=false`` (no multiply-add contraction
in device code, so each product and sum is rounded on its own) and
``-ffp-contract=off`` for the host compiler (the per-call scalars).  Division
and square root keep nvcc's IEEE defaults (``-prec-div=true
-prec-sqrt=true``), and denormals are kept (``-ftz=false``).
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libfp8opt.so")
BINDING = os.path.join(OUT_DIR, "fp8opt_binding.so")
BINDING_STAMP = BINDING + ".torch"
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
SOURCES = ["api.cu", "cast_kernels.cu", "step_kernels.cu", "fused_kernels.cu",
           "noalloc.cu", "reduce_kernels.cu", "norm_kernels.cu", "train_api.cu",
           "act_kernels.cu", "layer_norm_fwd.cu", "layer_norm_bwd.cu",
           "linear_xent.cu", "embedding.cu", "policy_loss.cu"]
DEPS = ["fp8opt_internal.cuh", "ops_internal.cuh", "layer_norm.cuh",
        "tensor_core.cuh", "teacher.cuh", os.path.join("..", "..", "include", "fp8opt.h")]

NVCC = os.environ.get("NVCC", "nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-fmad=false", "-ftz=false",
         "-prec-div=true", "-prec-sqrt=true", "-Xcompiler",
         "-fPIC,-ffp-contract=off,-fvisibility=hidden", "-Xptxas",
         "-warn-spills"]


def _stale(out, sources) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(p) > t for p in [*sources, __file__])


def _torch() -> str:
    """The torch and Python that a binding is built against."""
    return f"{importlib.metadata.version('torch')} {sys.version}"


def _binding_stale() -> bool:
    if _stale(BINDING, [BINDING_SOURCE]) or not os.path.exists(BINDING_STAMP):
        return True
    with open(BINDING_STAMP) as f:
        return f.read() != _torch()


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        sys.stderr.write(r.stdout + r.stderr)
    return obj


def _compile_binding() -> None:
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(NVCC))))
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
           "-fvisibility=hidden", "-I" + sysconfig.get_paths()["include"],
           "-I" + os.path.join(torch_dir, "include"),
           "-I" + os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           "-I" + os.path.join(cuda, "include"), BINDING_SOURCE, "-o", tmp,
           "-L" + os.path.join(torch_dir, "lib"), "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling binding.cpp failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING_STAMP, "w") as f:
        f.write(_torch())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libfp8opt.so and the binding where a source is newer,
    the binding also where it was built against another torch; return the
    library's path."""
    lib = force or _stale(LIB, [os.path.join(CSRC, s) for s in SOURCES + DEPS])
    binding = force or _binding_stale()
    os.makedirs(OUT_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        other = ex.submit(_compile_binding) if binding else None
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES)) if lib else []
        if other is not None:
            other.result()
    if lib:
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
