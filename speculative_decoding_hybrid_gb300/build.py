"""Builds libgdnspec.so in-tree with nvcc for sm_103a.

Each translation unit is compiled in parallel, then linked into one shared
library next to this file.  Usage: ``python -m speculative_decoding_hybrid_gb300.build``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import re
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(HERE, "libgdnspec.so")
BUILD_DIR = os.path.join(HERE, "_build")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# Kernels whose warps share out the registers of their launch: with another number of them (the assembler's choice, up to
# the launch bound's) the shares would not add up, and the library refuses to launch them.
LAUNCH_REGISTERS = {"prompt_attend_kernel": 168}


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgdnspec.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps_mtime():
    files = _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return max(os.path.getmtime(f) for f in files)


def up_to_date() -> bool:
    return os.path.exists(OUT) and os.path.getmtime(OUT) >= _deps_mtime()


def check_registers(info: str) -> None:
    """Raises unless every kernel of LAUNCH_REGISTERS in the assembler's report has its number of registers."""
    for name, used in re.findall(r"Compiling entry function '(\S+)'.*?Used (\d+) registers", info, re.S):
        for kernel, wanted in LAUNCH_REGISTERS.items():
            if kernel in name and int(used) != wanted:
                raise RuntimeError("%s has %s registers where its warps share out %d: its shares (setmaxnreg) have to be "
                                   "set for this compiler" % (name, used, wanted))


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and not ptxas_info and up_to_date():
        return OUT
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    common = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE, "-I", CSRC]

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [cc, "-c", *ARCH, *common, "-Xptxas", "-v", "-o", obj, src]
        if src.endswith(".cpp"):
            cmd = [cc, "-c", "-x", "c++", *common, "-o", obj, src]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        check_registers(r.stderr)
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 2)) as ex:
        results = list(ex.map(compile_one, _sources()))
    if verbose or ptxas_info:
        for _, err in results:
            if not ptxas_info:
                err = re.sub(r"^(ptxas info|    \d+ bytes stack frame).*\n", "", err, flags=re.M)
            sys.stderr.write(err)
    objs = [o for o, _ in results]
    tmp = OUT + ".tmp%d" % os.getpid()
    cudalib = os.path.join(os.path.dirname(os.path.dirname(cc)), "lib64")
    link = [cc, "-shared", *ARCH, "-cudart", "shared", "-o", tmp, *objs,
            "-Xlinker", "-rpath," + cudalib]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
