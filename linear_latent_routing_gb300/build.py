"""Build ``libgma.so`` in-tree from the CUDA sources in ``csrc/`` for sm_103a, and ``_block.so``, the Python
binding of ``include/gma_block.h`` (``csrc/block_binding.cpp``, against the installed torch's headers).

Each translation unit compiles in parallel with nvcc (the binding with the host compiler), then one
link step produces the shared library next to this file.  No CMake; a rebuild happens only when a
source or header is newer than what it goes into, or the binding was made for another torch.  Where no torch
with CUDA is installed, libgma.so is built alone.
"""
import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgma.so")
BINDING_SRC = os.path.join(CSRC, "block_binding.cpp")
BINDING = os.path.join(PKG, "_block.so")
BINDING_STAMP = os.path.join(BUILD, "block_binding.for")

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


def _torch_dir():
    """Where the installed torch lies, without importing it; None if there is none, or one without CUDA."""
    spec = importlib.util.find_spec("torch")
    where = os.path.dirname(spec.origin) if spec and spec.origin else ""
    return where if os.path.exists(os.path.join(where, "lib", "libc10_cuda.so")) else None


def _binding_for(torch_dir):
    """What the binding's object code depends on beside the sources: this interpreter and that torch."""
    with open(os.path.join(torch_dir, "version.py")) as f:
        return "\n".join([sysconfig.get_config_var("EXT_SUFFIX"), torch_dir, f.read()])


def _binding_stale(torch_dir):
    deps = [BINDING_SRC, os.path.abspath(__file__)] + glob.glob(os.path.join(INCLUDE, "*.h"))
    if not os.path.exists(BINDING) or any(os.path.getmtime(p) > os.path.getmtime(BINDING) for p in deps):
        return True
    if not os.path.exists(BINDING_STAMP):
        return True
    with open(BINDING_STAMP) as f:
        return f.read() != _binding_for(torch_dir)


def _compile_binding(torch_dir):
    """The binding's object file; it is linked once libgma.so is there."""
    import torch
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
    return obj


def _link_binding(obj, torch_dir):
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [CXX, "-shared", "-o", tmp, obj, "-L", PKG, "-l:libgma.so", "-Wl,-rpath,$ORIGIN", "-L", os.path.join(torch_dir, "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"link failed:\n{p.stdout}\n{p.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING_STAMP, "w") as f:
        f.write(_binding_for(torch_dir))


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile and link libgma.so and, where torch is installed, its binding if needed; return the library's path.

    Without torch the C ABI is all there is to use, and nvcc all that it needs.
    """
    torch_dir = _torch_dir()
    lib_stale, binding_stale = force or _stale(), torch_dir is not None and (force or _binding_stale(torch_dir))
    if not lib_stale and not binding_stale:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=8) as ex:
        binding = ex.submit(_compile_binding, torch_dir) if binding_stale else None
        if lib_stale:
            _build_library(ex, verbose_ptxas)
        if binding:
            _link_binding(binding.result(), torch_dir)
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
