"""Builds the CUDA library ``libcompfp32.so`` in place (nvcc, sm_103a only).

Each ``csrc/*.cu`` is compiled in parallel to an object under ``_build/`` and
the objects are linked into one shared library next to this file.
``csrc/attn_binding.cpp`` is compiled with the host compiler at the same time
and becomes ``_attn_binding.so``, the torch binding of the attention calls, for
the torch that is there; without one, or with one without CUDA, the C library is
all that is built.  The CUDA
runtime is linked statically, so the library needs only the NVIDIA driver at
run time (and loads, without running anything, on a machine with no GPU).

No fast-math and no flush-to-zero: the split and merge must be bit-exact.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libcompfp32.so")
BINDING = os.path.join(PKG, "_attn_binding.so")
BINDING_SRC = os.path.join(CSRC, "attn_binding.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3",
    "-lineinfo",
    "-std=c++17",
    "-Xcompiler",
    "-fPIC",
    "-Xptxas",
    "-v",
    "-I",
    INCLUDE,
    "-I",
    CSRC,
]


def nvcc() -> str:
    env = os.environ.get("NVCC")
    if env:
        return env
    found = shutil.which("nvcc")
    if found:
        return found
    return "/usr/local/cuda/bin/nvcc"


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    return _sources() + [BINDING_SRC] + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + [
        os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)
    ] + [os.path.abspath(__file__)]


def _torch_dir() -> str | None:
    """The folder of a torch with CUDA, found without importing it."""
    spec = importlib.util.find_spec("torch")
    for d in (spec.submodule_search_locations or []) if spec else []:
        if os.path.exists(os.path.join(d, "lib", "libc10_cuda.so")):
            return d
    return None


def _torch_stamp(torch: str) -> str:
    """What the binding's ABI depends on: this torch's place and version."""
    with open(os.path.join(torch, "version.py")) as f:
        version = re.search(r"__version__\s*=\s*['\"]([^'\"]+)", f.read())
    return f"{torch} {version.group(1) if version else ''}\n"


def _stamp_path() -> str:
    return os.path.join(BUILD, "attn_binding.torch")


def _built_for() -> str:
    try:
        with open(_stamp_path()) as f:
            return f.read()
    except OSError:
        return ""


def up_to_date() -> bool:
    torch = _torch_dir()
    made = [LIB] if torch is None else [LIB, BINDING]
    if not all(os.path.exists(m) for m in made) or (torch is not None and _built_for() != _torch_stamp(torch)):
        return False
    t = min(os.path.getmtime(m) for m in made)
    return all(os.path.getmtime(d) <= t for d in _deps())


def _compile(src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *NVCC_FLAGS, "-c", src, "-o", obj]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{p.stdout}\n{p.stderr}")
    return obj, p.stderr


def _cuda_include() -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")


def _compile_binding(torch: str) -> str:
    """The binding's object, with the headers of the torch in this folder."""
    obj = os.path.join(BUILD, "attn_binding.o")
    inc = [INCLUDE, os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], _cuda_include()]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-c", BINDING_SRC, "-o", obj,
           *[a for d in inc for a in ("-isystem" if d != INCLUDE else "-I", d)]]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {BINDING_SRC}:\n{' '.join(cmd)}\n{p.stdout}\n{p.stderr}")
    return obj


def _link_binding(obj: str, torch: str) -> None:
    lib = os.path.join(torch, "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-shared", obj, "-o", tmp, "-L", PKG, "-l:libcompfp32.so", "-L", lib,
           "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{p.stdout}\n{p.stderr}")
    os.replace(tmp, BINDING)
    with open(_stamp_path(), "w") as f:
        f.write(_torch_stamp(torch))


# Kernels that move registers between warpgroups with setmaxnreg assume this
# launch register count; a different count could make setmaxnreg.inc wait
# forever, so the build refuses it.
SETMAXNREG_KERNELS = {"comp_gemm_kernel": 96, "comp_f16x2_kernel": 168, "comp_f16x2_pair_kernel": 168,
                      "comp_f16x2_splitk_kernel": 168, "comp_f32x16_pair_kernel": 128, "attn_tc_kernel": 168}


def _check_register_budget(ptxas_log: str) -> None:
    current = None
    for line in ptxas_log.splitlines():
        if "Compiling entry function" in line:
            current = next((k for k in SETMAXNREG_KERNELS if k in line), None)
        elif current and "Used" in line and "registers" in line:
            used = int(line.split("Used")[1].split("registers")[0])
            if used != SETMAXNREG_KERNELS[current]:
                raise RuntimeError(f"{current}: ptxas reports {used} registers, the register split assumes "
                                   f"{SETMAXNREG_KERNELS[current]}")
            current = None


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the library if any source, or the torch of its binding,
    changed; returns its path.  A binding that cannot be built is an error, raised
    once the library is in place."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs, torch = _sources(), _torch_dir()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        binding = ex.submit(_compile_binding, torch) if torch is not None else None
        results = list(ex.map(_compile, srcs))
    with open(os.path.join(BUILD, "ptxas.txt"), "w") as f:
        for (obj, log), src in zip(results, srcs):
            f.write(f"== {os.path.basename(src)}\n{log}\n")
    _check_register_budget("\n".join(log for _, log in results))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{p.stdout}\n{p.stderr}")
    os.replace(tmp, LIB)
    if binding is not None:
        _link_binding(binding.result(), torch)
    if verbose:
        print(open(os.path.join(BUILD, "ptxas.txt")).read())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
