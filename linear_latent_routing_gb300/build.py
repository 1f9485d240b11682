"""Build ``libgma.so`` in-tree from the CUDA sources in ``csrc/`` for sm_103a, and ``_block.so``, the Python
binding of ``include/gma_block.h`` (``csrc/block_binding.cpp``, against the installed torch's headers).

Each translation unit compiles in parallel with nvcc (the binding with the host compiler), then one
link step produces the shared library next to this file.  No CMake; a rebuild happens only when a
source or header is newer than what it goes into.
"""
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgma.so")
BINDING_SRC = os.path.join(CSRC, "block_binding.cpp")
BINDING = os.path.join(PKG, "_block.so")

NVCC = os.environ.get("NVCC", "nvcc")
CXX = os.environ.get("CXX", "g++")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def _stale():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _deps())


def _compile(src, verbose_ptxas=False):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [NVCC] + ARCH + FLAGS + (["-Xptxas", "-v"] if verbose_ptxas else []) + ["-c", src,
                                                                                   "-o", obj]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{p.stdout}\n{p.stderr}")
    return obj, p.stderr


def _binding_stale():
    deps = [BINDING_SRC, os.path.abspath(__file__)] + glob.glob(os.path.join(INCLUDE, "*.h"))
    return not os.path.exists(BINDING) or any(os.path.getmtime(p) > os.path.getmtime(BINDING) for p in deps)


def _compile_binding():
    """The binding's object file; it is linked once libgma.so is there."""
    import sysconfig

    import torch
    torch_dir = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(NVCC) or "/usr/local/cuda/bin/nvcc")))
    includes = [INCLUDE, os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(cuda, "include"), "/usr/local/cuda/include"]
    obj = os.path.join(BUILD, "block_binding.o")
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
    for i in includes:
        cmd += ["-I", i]
    p = subprocess.run(cmd + ["-c", BINDING_SRC, "-o", obj], capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"{CXX} failed for {BINDING_SRC}:\n{p.stdout}\n{p.stderr}")
    return obj, os.path.join(torch_dir, "lib")


def _link_binding(obj, torch_lib):
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [CXX, "-shared", "-o", tmp, obj, "-L", PKG, "-l:libgma.so", "-Wl,-rpath,$ORIGIN", "-L", torch_lib, "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"link failed:\n{p.stdout}\n{p.stderr}")
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile and link libgma.so and its binding if needed; return the library's path."""
    lib_stale, binding_stale = force or _stale(), force or _binding_stale()
    if not lib_stale and not binding_stale:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=8) as ex:
        binding = ex.submit(_compile_binding) if binding_stale else None
        if lib_stale:
            _build_library(ex, verbose_ptxas)
        if binding:
            _link_binding(*binding.result())
    return LIB


def _build_library(ex, verbose_ptxas):
    results = list(ex.map(lambda s: _compile(s, verbose_ptxas), _sources()))
    if verbose_ptxas:
        for _, log in results:
            print(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"link failed:\n{p.stdout}\n{p.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose_ptxas="-v" in sys.argv))
