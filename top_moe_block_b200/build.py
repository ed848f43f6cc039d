"""Build libzaya.so in-tree: every CUDA source of csrc/ for sm_100a; and _fast.so,
the paged operators' Python calls (csrc/binding.cpp), which links it.

    python -m top_moe_block_b200.build
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
OUT = os.path.join(HERE, "libzaya.so")
FAST = os.path.join(HERE, "_fast.so")
FAST_STAMP = os.path.join(HERE, "_fast.stamp")   # what _fast.so was built against
BINDING = os.path.join(HERE, "csrc", "binding.cpp")


def sources():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(HERE, "csrc", "*.cuh")) + glob.glob(
        os.path.join(HERE, "csrc", "*.h")) + glob.glob(os.path.join(ROOT, "include", "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(OUT):
        return False
    t = os.path.getmtime(OUT)
    return all(os.path.getmtime(f) <= t for f in _deps())


def _fast_flags() -> list[str]:
    import torch
    return ["-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]


def _fast_stamp() -> str:
    """The interpreter and the torch whose C++ interfaces _fast.so is compiled against, and the flags."""
    import sysconfig

    import torch
    return "\n".join([sysconfig.get_config_var("SOABI") or sys.version, "torch " + torch.__version__,
                      str(torch.version.git_version), " ".join(_fast_flags())]) + "\n"


def _fast_up_to_date() -> bool:
    if not os.path.exists(FAST) or not os.path.exists(FAST_STAMP):
        return False
    with open(FAST_STAMP) as f:
        if f.read() != _fast_stamp():
            return False
    t = os.path.getmtime(FAST)
    return all(os.path.getmtime(f) <= t for f in [BINDING] + glob.glob(os.path.join(ROOT, "include", "*.h")))


def build_fast(verbose: bool = False) -> str:
    """_fast.so against this interpreter and its torch."""
    import sysconfig

    import torch
    torch_dir = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"))
    tmp = FAST + ".tmp"
    cmd = [shutil.which("g++") or "g++"] + _fast_flags()
    for d in (os.path.join(ROOT, "include"), os.path.join(torch_dir, "include"), os.path.join(cuda, "include"),
              sysconfig.get_paths()["include"]):
        cmd += ["-I", d]
    cmd += ["-o", tmp, BINDING, "-L", HERE, "-l:libzaya.so", "-L", os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, FAST)
    with open(FAST_STAMP, "w") as f:
        f.write(_fast_stamp())
    return FAST


def build(force: bool = False, verbose: bool = False) -> str:
    if force or not up_to_date():
        _build_lib(verbose)
    if force or not _fast_up_to_date():
        build_fast(verbose)
    return OUT


def _build_lib(verbose: bool) -> None:
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    tmp = OUT + ".tmp"
    cmd = [nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
           "-Xcompiler", "-fPIC", "-shared", "-I", os.path.join(ROOT, "include"), "-o", tmp] + sources()
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, OUT)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
