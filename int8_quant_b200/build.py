"""Builds libssd.so (nvcc, sm_100a) and, where torch is installed, its Python binding _binding.so in-tree."""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libssd.so")
BINDING = os.path.join(HERE, "_binding.so")
STAMP = os.path.join(HERE, "_binding.torch")          # the torch that it was built for
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


def _torch_version() -> str | None:
    """The torch that a binding is for, or None where there is none: the library alone is built then."""
    if importlib.util.find_spec("torch") is None:
        return None
    import torch
    return torch.__version__


def _binding_is_for() -> str:
    """The torch that _binding.so was built for."""
    try:
        with open(STAMP) as f:
            return f.read().strip()
    except OSError:
        return ""


def needs_build() -> bool:
    version = _torch_version()
    built = [LIB] if version is None else [LIB, BINDING]
    if not all(os.path.exists(p) for p in built) or (version is not None and _binding_is_for() != version):
        return True
    t = min(os.path.getmtime(p) for p in built)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps.append(os.path.join(HERE, "..", "include", "ssd.h"))
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True, cwd=CSRC)


def build(force: bool = False, verbose: bool = False) -> str:
    """The library and, where torch is installed, its binding; both are put in place once both are there."""
    if not force and not needs_build():
        return LIB
    with tempfile.TemporaryDirectory(dir=HERE, prefix=".build-") as tmp:
        lib, binding = os.path.join(tmp, os.path.basename(LIB)), os.path.join(tmp, os.path.basename(BINDING))
        _run([_nvcc(), *NVCC_FLAGS, "-o", lib, *[os.path.join(CSRC, s) for s in SOURCES]], verbose)
        version = _torch_version()
        if version is not None:
            _link_binding(binding, tmp, version, verbose)
        os.replace(lib, LIB)
        if version is not None:
            _place_binding(binding, version)
    return LIB


def build_binding(verbose: bool = False) -> str:
    """_binding.so alone, for the library that is there."""
    with tempfile.TemporaryDirectory(dir=HERE, prefix=".build-") as tmp:
        binding, version = os.path.join(tmp, os.path.basename(BINDING)), _torch_version()
        _link_binding(binding, HERE, version, verbose)
        _place_binding(binding, version)
    return BINDING


def _link_binding(out: str, lib_dir: str, version: str, verbose: bool):
    """The binding, linked to the libssd.so that will lie beside it and to torch's libraries (loaded by `import torch`)."""
    import sysconfig

    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"]]
    # nvcc hands a .cpp to its host compiler: the library's own toolchain and C++ runtime
    _run([_nvcc(), "-Wno-deprecated-gpu-targets", "-O2", "-std=c++17", "-Xcompiler", "-fPIC", "-shared",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", f'-DSSD_TORCH_VERSION="{version}"',
          *[f for i in inc for f in ("-isystem", i)], "-o", out, os.path.join(CSRC, "binding.cpp"),
          "-L" + lib_dir, "-l:libssd.so", "-Xlinker", "-rpath", "-Xlinker", "$ORIGIN",
          "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"], verbose)


def _place_binding(binding: str, version: str):
    os.replace(binding, BINDING)
    with open(STAMP, "w") as f:
        f.write(version + "\n")


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
