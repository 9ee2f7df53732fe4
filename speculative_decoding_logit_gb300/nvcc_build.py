"""Build step for libasv.so: compile every CUDA source under csrc/ for sm_103a with nvcc
(in parallel, one -gencode) and link the shared library in-tree under _build/."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libasv.so")
# The checked build: the same sources with -DASV_CHECKED (every kernel index tested against its
# buffer, failures counted in the workspace's check log, the access skipped).
LIB_CHECKED = os.path.join(BUILD, "libasv_checked.so")
# The binding's compiled part (a CPython module over PyTorch's C++ tensors, no device code).
TORCH_EXT = os.path.join(BUILD, "asv_torch.so")
TORCH_EXT_SRC = os.path.join(CSRC, "asv_torch.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
              "-Xptxas", "-warn-spills", f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _deps():
    return (glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.inc")) +
            [os.path.join(INCLUDE, "asv.h"), os.path.abspath(__file__)])


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(d) <= t for d in _deps())


def build_checked(force: bool = False, verbose: bool = False) -> str:
    """Compile the checked library (_build/libasv_checked.so, -DASV_CHECKED)."""
    return build(force=force, verbose=verbose, extra_flags=("-DASV_CHECKED",), lib=LIB_CHECKED)


def torch_ext_fits() -> bool:
    """Whether the binding's module was built for the PyTorch and the Python that run (noted beside it)."""
    try:
        with open(TORCH_EXT + ".for") as f:
            return f.read() == _running()
    except OSError:
        return False


def _running() -> str:
    import sysconfig

    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def build_torch_ext(force: bool = False) -> str:
    """Compile the binding's module (_build/asv_torch.so) with the host compiler, for the PyTorch that runs."""
    deps = [TORCH_EXT_SRC, os.path.join(INCLUDE, "asv.h"), os.path.abspath(__file__)]
    if not force and torch_ext_fits() and os.path.exists(TORCH_EXT) and all(
            os.path.getmtime(d) <= os.path.getmtime(TORCH_EXT) for d in deps):
        return TORCH_EXT
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), INCLUDE]
    os.makedirs(BUILD, exist_ok=True)
    tmp = TORCH_EXT + f".{os.getpid()}.tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++20", "-fPIC", "-shared", *[f"-I{i}" for i in inc],
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", TORCH_EXT_SRC, "-o", tmp,
           f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", f"-Wl,-rpath,{lib}"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        failed = r.returncode != 0 and f"{r.stdout}\n{r.stderr}"
    except OSError as e:
        failed = str(e)
    if failed:
        if os.path.exists(TORCH_EXT):   # of older sources, or for another PyTorch
            os.remove(TORCH_EXT)
        raise RuntimeError(f"the binding's module failed to compile:\n{failed}")
    os.replace(tmp, TORCH_EXT)
    with open(tmp, "w") as f:
        f.write(_running())
    os.replace(tmp, TORCH_EXT + ".for")
    return TORCH_EXT


def build(force: bool = False, verbose: bool = False, extra_flags=(), lib: str = LIB) -> str:
    """Compile csrc/*.cu and link `lib` (default _build/libasv.so), and with the default library the
    binding's module; returns the library path.  Only the paged calls and the sampling need the module: where
    it does not compile that is a warning here, and they refuse."""
    if lib != LIB:
        return _build_library(force, verbose, extra_flags, lib)
    with cf.ThreadPoolExecutor(1) as ex:
        ext = ex.submit(build_torch_ext, force)
        path = _build_library(force, verbose, extra_flags, lib)
    try:
        ext.result()
    except RuntimeError as e:
        warnings.warn(f"the paged calls and sample_tokens are not available: {e}", RuntimeWarning, stacklevel=2)
    return path


def _build_library(force: bool, verbose: bool, extra_flags, lib: str) -> str:
    if not force and up_to_date(lib):
        return lib
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    tag = f"{os.getpid()}{'c' if extra_flags else ''}"

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + f".{tag}.o")
        cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = lib + f".{tag}.tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs, "-lcudart_static", "-ldl", "-lpthread", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    for o in objs:
        os.remove(o)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
    print(build_checked(force="--force" in sys.argv, verbose=True))
