"""Build librd.so (the HIP kernels and their C ABI) for gfx950 and _rd.so (the routed
layer's calls from PyTorch, host code), in-tree.

Usage: ``python -m expert_ffn_ragged_amd.build`` (or ``__graft_entry__.build()``).
Always recompiles.  Flags: -O3 for gfx950 only; packed-FP32 instructions are
disabled (``-packed-fp32-ops``); no fast-math; the GLU units (plain
and with an 8-bit residual) additionally get ``-ffp-contract=off`` so their float32 op order is exactly the
source's.
"""

import concurrent.futures
import os
import shlex
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "librd.so")
MODULE = os.path.join(HERE, "_rd.so")
BUILD_DIR = os.path.join(ROOT, "_build")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CXX = os.environ.get("CXX", "g++")
ARCH = "gfx950"
COMMON = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE, "-I", CSRC, "-Wall", "-Wno-unused-result",
]
SOURCES = [
    ("rd_gemm.hip", []),
    ("rd_glu.hip", ["-ffp-contract=off"]),
    ("rd_unsort.hip", []),
    ("rd_rows.hip", []),
    ("rd_route.hip", []),
    ("rd_combine.hip", []),
    ("rd_mx.hip", ["-ffp-contract=off"]),
    ("rd_gemm_mx.hip", []),
    ("rd_api.cpp", ["-x", "hip"]),
]
MODULE_SOURCE = "rd_torch.cpp"


def _run(cmd):
    proc = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    # hipcc's host pass does not know the packed-fp32 feature and says so; drop that line
    lines = [ln for ln in proc.stdout.splitlines() if "packed-fp32-ops' is not a recognized feature" not in ln]
    if proc.returncode != 0:
        sys.stderr.write("\n".join(lines) + "\n")
        raise RuntimeError("command failed: " + " ".join(shlex.quote(c) for c in cmd))
    return "\n".join(lines)


def _torch_flags():
    """Compile and link flags of a host module that takes torch tensors."""
    import torch

    root = os.path.dirname(torch.__file__)
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    include = ["-I", os.path.join(root, "include"), "-I",
               os.path.join(root, "include", "torch", "csrc", "api", "include"),
               "-isystem", sysconfig.get_paths()["include"], f"-D_GLIBCXX_USE_CXX11_ABI={abi}"]
    return include, ["-L", os.path.join(root, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python"]


def _obj(src):
    return os.path.join(BUILD_DIR, src + ".o")


def _compile_module():
    """The host module's object; returns the flags to link it with, or None where torch is not installed."""
    try:
        include, libs = _torch_flags()
    except ImportError as e:
        sys.stderr.write(f"{e}: _rd.so (the routed layer's calls from PyTorch) is not built\n")
        return None
    _run([CXX, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-I", INCLUDE, *include, "-c",
          os.path.join(CSRC, MODULE_SOURCE), "-o", _obj(MODULE_SOURCE)])
    return libs


def build(verbose=False):
    """Compile every source for gfx950 and link librd.so and _rd.so next to this file.

    librd.so needs hipcc alone and is there before a failure of the host module, which needs torch, a C++ compiler
    and Python's headers, is raised.
    """
    os.makedirs(BUILD_DIR, exist_ok=True)
    steps = [[HIPCC, *COMMON, *extra, "-c", os.path.join(CSRC, src), "-o", _obj(src)] for src, extra in SOURCES]
    # each is linked beside its place and moved there whole; _rd.so finds librd.so in its own folder
    with concurrent.futures.ThreadPoolExecutor(4) as pool:
        outs = pool.map(_run, steps)
        module = pool.submit(_compile_module)
        for out in outs:
            if verbose and out.strip():
                print(out)
        _run([HIPCC, "-shared", f"--offload-arch={ARCH}", "-fPIC", "-Wl,-soname,librd.so",
              *(_obj(src) for src, _ in SOURCES), "-o", LIB + ".tmp"])
        os.replace(LIB + ".tmp", LIB)
        libs = module.result()
    if libs is not None:
        _run([CXX, "-shared", _obj(MODULE_SOURCE), LIB, *libs, "-Wl,-rpath,$ORIGIN", "-o", MODULE + ".tmp"])
        os.replace(MODULE + ".tmp", MODULE)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
