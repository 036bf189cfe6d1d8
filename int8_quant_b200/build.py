"""Builds libssd.so (nvcc, sm_100a) and its Python binding _binding.so in-tree."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libssd.so")
BINDING = os.path.join(HERE, "_binding.so")
SOURCES = ["api.cu", "quantize.cu", "cumsum.cu", "chunk_state.cu", "state_passing.cu", "chunk_scan.cu",
           "noalloc.cu", "tmap.cu", "chunk_state_tc.cu", "chunk_scan_tc.cu", "selftest.cu",
           "decode.cu", "out_proj.cu", "fused_i8.cu", "chunk_bmm.cu", "rmsnorm_i8.cu", "matmul_i8.cu", "conv.cu"]
NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
              "-Xcompiler", "-fPIC", "-shared"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def needs_build() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps.append(os.path.join(HERE, "..", "include", "ssd.h"))
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    cmd = [_nvcc(), *NVCC_FLAGS, "-o", LIB + ".tmp", *[os.path.join(CSRC, s) for s in SOURCES]]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True, cwd=CSRC)
    os.replace(LIB + ".tmp", LIB)
    build_binding(verbose)
    return LIB


def build_binding(verbose: bool = False) -> str:
    """_binding.so: linked to libssd.so beside it and to torch's libraries (loaded by `import torch`)."""
    import sysconfig

    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"]]
    # nvcc hands a .cpp to its host compiler: the library's own toolchain and C++ runtime
    cmd = [_nvcc(), "-Wno-deprecated-gpu-targets", "-O2", "-std=c++17", "-Xcompiler", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *[f for i in inc for f in ("-isystem", i)], "-o", BINDING + ".tmp", os.path.join(CSRC, "binding.cpp"),
           "-L" + HERE, "-l:libssd.so", "-Xlinker", "-rpath", "-Xlinker", "$ORIGIN",
           "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True, cwd=CSRC)
    os.replace(BINDING + ".tmp", BINDING)
    return BINDING


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
