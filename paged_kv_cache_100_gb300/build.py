"""Builds ``_build/libpagedkv.so`` in-tree: the CUDA kernels for sm_103a and the host
block manager, linked against the static CUDA runtime (no libcuda link-time
dependency; the driver is reached at run time)."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libpagedkv.so")
BINDING_MODULE = "_pagedkv_torch.so"

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CU_SOURCES = ["pa_decode.cu", "pa_cache.cu", "pa_decode_noalloc.cu", "pa_prefill.cu", "pa_plan.cu",
              "pa_rope.cu", "pa_block8_decode.cu", "pa_block8_prefill.cu", "pa_fp4_cache.cu", "pa_fp4_decode.cu"]
CPP_SOURCES = ["block_manager.cpp"]
BINDING = "torch_binding.cpp"     # its own module: it follows the installed torch, the library does not
HEADERS = ["pa_device.cuh", "pa_internal.h", "pa_tc.cuh", "pa_block8.cuh", "pa_rope.cuh", "pa_fp4.cuh"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _no_binding() -> str:
    """Why the tensor binding cannot be built here ("" when it can): the C ABI needs neither torch nor
    its headers, so a machine without them gets the library alone."""
    import importlib.util
    import sysconfig
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return "torch is not installed"
    for header in (os.path.join(os.path.dirname(spec.origin), "include", "ATen", "core", "Tensor.h"),
                   os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(header):
            return f"{header} is missing"
    return ""


def _stale(lib: str) -> bool:
    binding = os.path.join(os.path.dirname(lib), BINDING_MODULE)
    if not os.path.exists(lib) or (lib == LIB and not os.path.exists(binding) and not _no_binding()):
        return True
    t = os.path.getmtime(lib)
    deps = [os.path.join(CSRC, f) for f in CU_SOURCES + CPP_SOURCES + HEADERS + [BINDING]]
    deps += [os.path.join(INCLUDE, "pagedkv.h"), os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_command(out: str) -> list:
    """The compiled tensor binding: a CPython module linked against the installed torch."""
    import sysconfig
    import torch
    tdir = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(tdir, "include"),
           os.path.join(tdir, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    libs = os.path.join(tdir, "lib")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[f"-I{d}" for d in inc], os.path.join(CSRC, BINDING), "-o", out, f"-L{libs}", f"-Wl,-rpath,{libs}",
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def build(force: bool = False, verbose_ptxas: bool = False, defines=(), build_dir=None) -> str:
    """Compile and link the library; returns its path.

    ``defines`` (e.g. ``["PA_DECODE_STAGES=2"]``) and ``build_dir`` produce a
    variant build elsewhere; the default build is ``_build/libpagedkv.so``, and
    beside it the tensor binding where torch and its headers are there.
    """
    bdir = build_dir or BUILD
    lib = os.path.join(bdir, "libpagedkv.so")
    if not force and not _stale(lib):
        return lib
    os.makedirs(bdir, exist_ok=True)
    nvcc = _nvcc()
    common = ["-O3", "-std=c++17", "-I", INCLUDE, "-I", CSRC] + [f"-D{d}" for d in defines]
    jobs = []
    objs = []
    for src in CU_SOURCES:
        obj = os.path.join(bdir, src + ".o")
        cmd = [nvcc, *ARCH, *common, "-lineinfo", "-Xcompiler", "-fPIC", "-c",
               os.path.join(CSRC, src), "-o", obj]
        if verbose_ptxas:
            cmd[1:1] = ["-Xptxas", "-v"]
        jobs.append((cmd, src))
        objs.append(obj)
    for src in CPP_SOURCES:
        obj = os.path.join(bdir, src + ".o")
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE, "-c",
               os.path.join(CSRC, src), "-o", obj]
        jobs.append((cmd, src))
        objs.append(obj)
    binding, bound = os.path.join(bdir, BINDING_MODULE), False
    if build_dir is None:
        reason = _no_binding()
        if reason:
            sys.stderr.write(f"--- {BINDING}: not built, {reason}\n")
        else:
            bound = True
            jobs.append((_binding_command(binding + f".tmp{os.getpid()}"), BINDING))
    procs = [(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT), src)
             for cmd, src in jobs]
    failed = []
    for p, src in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if text.strip():
            sys.stderr.write(f"--- {src}\n{text}")
        if p.returncode != 0:
            failed.append(src)
    if [f for f in failed if f != BINDING]:
        raise RuntimeError(f"compilation failed: {', '.join(failed)}")
    if bound and not failed:
        os.replace(binding + f".tmp{os.getpid()}", binding)
    elif build_dir is None and os.path.exists(binding):
        os.remove(binding)                # one made for another build of the library
    tmp = lib + f".tmp{os.getpid()}"
    subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], check=True)
    os.replace(tmp, lib)
    if failed:                            # the library itself is there
        raise RuntimeError(f"compilation failed: {', '.join(failed)}")
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
