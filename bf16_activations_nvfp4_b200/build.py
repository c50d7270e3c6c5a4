"""Build libfi_nvfp4.so in-tree with nvcc for sm_100a (B200), and the Python module _binding.so.

    python -m bf16_activations_nvfp4_b200.build [--force]

Each csrc/*.cu is compiled to an object under _build/ (skipped when up to date), then
linked into bf16_activations_nvfp4_b200/libfi_nvfp4.so with the CUDA runtime linked
statically, so the library loads without a CUDA install path and without a GPU. csrc/binding.cpp
is compiled by the host compiler against the installed torch.
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfi_nvfp4.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_RECORD = os.path.join(BUILD, "binding.command")  # what BINDING was built with

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libfi_nvfp4.so")


def _deps() -> list[str]:
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(CSRC, "*.inc")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(target: str, sources: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in sources)


def _binding_command(nvcc: str, target: str) -> list[str]:
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    paths = [INCLUDE, inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"], cuda]
    # torch's libraries are in the process before the module is: no run path
    return [shutil.which("g++") or "g++", "-O2", "-std=c++20", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f'-DFI_TORCH_VERSION="{torch.__version__}"', *["-isystem" + p for p in paths],
            os.path.join(CSRC, "binding.cpp"), "-L" + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
            "-ltorch_python", "-o", target]


def _binding_stale(record: str) -> bool:
    """The module uses torch's C++ interface: another torch, Python or compiler call needs another one."""
    sources = [os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "fi_nvfp4.h"), __file__]
    if _stale(BINDING, sources) or not os.path.exists(BINDING_RECORD):
        return True
    with open(BINDING_RECORD) as f:
        return f.read() != record


def build(force: bool = False, verbose: bool = False) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = _deps()
    jobs = []
    objs = []
    for src in sources:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + deps + [__file__]):
            jobs.append([nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj])
    link = force or bool(jobs)
    binding_tmp = BINDING + f".tmp{os.getpid()}"
    record = " ".join(_binding_command(nvcc, BINDING))
    binding = force or _binding_stale(record)
    if binding:
        jobs.append(_binding_command(nvcc, binding_tmp))

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed for {cmd[-3]}:\n{r.stdout}\n{r.stderr}")
        return r

    with ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        list(ex.map(run, jobs))
    if binding:
        os.replace(binding_tmp, BINDING)
        with open(BINDING_RECORD, "w") as f:
            f.write(record)
    if link or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    return LIB


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    args = ap.parse_args(argv)
    print(build(force=args.force, verbose=args.verbose))
    return 0


if __name__ == "__main__":
    sys.exit(main())
