"""Build libqk.so (the CUDA library behind include/qk.h) in-tree with nvcc, and
_block_calls (csrc/block_calls.cpp, calls of it for binding.py) with g++, for this
Python and this torch.

Every .cu under csrc/ is compiled for sm_100a only
(``-gencode arch=compute_100a,code=sm_100a``), objects go to ``_build/``, and
the shared library lands next to this file.  The CUDA runtime is linked
statically, so loading the library needs no GPU; only the driver is required
at call time.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
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
LIB = os.path.join(PKG, "libqk.so")
CALLS = os.path.join(PKG, "_block_calls" + sysconfig.get_config_var("EXT_SUFFIX"))
CALLS_ABI = os.path.join(BUILD, "block_calls.abi")  # what CALLS was built against

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC, *ARCH]

# Kernels that share out the registers they are launched with (setmaxnreg): their sources' kRegsLaunch is
# what the split adds up to, and a launch with another count is refused, so the compiler has to have chosen it.
SPLITS = {"sage_attn.cu": "sage_attn_kernel", "gemm_w4a8.cu": "w4a8_gemm_kernel", "kv4_chunk.cu": "kv4_chunk_kernel"}


def launch_registers(ptxas: str, kernel: str) -> list:
    """The registers per thread of each instance of the kernel, from what ptxas -v printed."""
    name = re.compile(rf"Compiling entry function '\S*{len(kernel)}{kernel}[IE]\S*'")
    counts, mine = [], False
    for line in ptxas.splitlines():
        if "Compiling entry function" in line:
            mine = name.search(line) is not None
        used = re.search(r"Used (\d+) registers", line)
        if used and mine:
            counts.append(int(used.group(1)))
    return counts


def check_split(src: str, ptxas: str) -> str:
    """What is wrong with the registers of the source's kernel, or nothing."""
    kernel = SPLITS[os.path.basename(src)]
    with open(src) as f:
        want = int(re.search(r"constexpr int kRegsLaunch = (\d+);", f.read()).group(1))
    counts = launch_registers(ptxas, kernel)
    if not counts or set(counts) != {want}:
        return f"{kernel}: compiled to {counts} registers per thread, its split is of {want}\n"
    return ""


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libqk.so")


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, ptxas_verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    objs = []
    jobs = []
    for src in sources:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if _newer(obj, [src, *headers]) or ptxas_verbose:
            cmd = [nvcc(), *NVCC_FLAGS, "-c", src, "-o", obj]
            if ptxas_verbose or os.path.basename(src) in SPLITS:
                cmd += ["-Xptxas", "-v"]
            jobs.append((cmd, src, obj))
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        results = list(ex.map(lambda c: subprocess.run(c[0], capture_output=True, text=True), jobs))
    failed = False
    for (cmd, src, obj), r in zip(jobs, results):
        wrong = ""
        if r.returncode == 0 and os.path.basename(src) in SPLITS:
            wrong = check_split(src, r.stdout + r.stderr)
            if wrong:
                os.remove(obj)
        if verbose or ptxas_verbose or r.returncode != 0 or wrong:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr + wrong)
        failed |= r.returncode != 0 or wrong != ""
    if failed:
        raise RuntimeError("nvcc failed building libqk.so")
    if _newer(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.run([nvcc(), "-shared", *ARCH, "-o", tmp, *objs], check=True)
        os.replace(tmp, LIB)
    _build_calls(verbose)
    return LIB


def _build_calls(verbose: bool) -> None:
    src = os.path.join(CSRC, "block_calls.cpp")
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    abi = f"Python {sys.version}\ntorch {importlib.metadata.version('torch')} in {torch_dir}\n"
    built = None
    if os.path.exists(CALLS_ABI):
        with open(CALLS_ABI) as f:
            built = f.read()
    if built == abi and not _newer(CALLS, [src, os.path.join(INCLUDE, "qk.h")]):
        return
    inc = os.path.join(torch_dir, "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = CALLS + f".tmp{os.getpid()}"
    # (torch's libraries are in the process by the time this one is loaded)
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], "-isystem", inc,
           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), src, "-o", tmp, "-L", PKG, "-l:libqk.so",
           "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
           "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError("g++ failed building _block_calls")
    os.replace(tmp, CALLS)
    with open(CALLS_ABI, "w") as f:
        f.write(abi)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, ptxas_verbose="--ptxas" in sys.argv))
