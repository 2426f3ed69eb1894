"""Build the CUDA library (libqhl_stage.so) in-tree for sm_100a with nvcc.

Every source under csrc/ is compiled with
``-gencode arch=compute_100a,code=sm_100a -O3 -lineinfo`` (no fast-math) and
linked into one shared object beside this file, with the CUDA runtime linked
statically so the library is self-contained.  The native marshalling of the
tree-verification calls (csrc/marshal.cpp, host code against PyTorch's headers)
becomes an extension module of its own, so the library stays free of PyTorch.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libqhl_stage.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
SOURCES = ["gemv.cu", "pass.cu", "mixers.cu", "stage.cu", "kernel_abi.cu", "noalloc.cu",
           "norm_rope.cu", "tree_attention.cu", "deltanet_tree.cu", "pages.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(out: str, marshal: bool) -> bool:
    """Whether `out` is older than a source of it: marshal.cpp, or all the others, and the header."""
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if (f == "marshal.cpp") == marshal]
    paths.append(os.path.join(os.path.dirname(HERE), "include", "qhl_stage.h"))
    return not os.path.exists(out) or os.path.getmtime(out) < max(os.path.getmtime(p) for p in paths)


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, src.replace(".cu", ".o"))
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stderr)
    return obj


def _torch_root() -> str | None:
    """Where PyTorch is installed, if it is (it is not imported: that takes seconds)."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _built_for() -> str:
    """What the marshalling module is built against; its docstring holds it, so that a module for another is known as one."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:      # on the path, but not installed as a package
        version = "of unknown version"
    return f"built for torch {version}, {sysconfig.get_config_var('SOABI')}"


def _marshal_stale() -> bool:
    if _stale(MARSHAL, True):
        return True
    with open(MARSHAL, "rb") as f:
        return _built_for().encode() not in f.read()


def _build_marshal(root: str):
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-DNDEBUG", f'-DQHL_BUILT_FOR="{_built_for()}"', *[f"-I{p}" for p in include],
           os.path.join(CSRC, "marshal.cpp"), "-o", tmp, f"-L{root}/lib", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{root}/lib"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on marshal.cpp:\n{r.stderr}")
    os.replace(tmp, MARSHAL)


def _build_lib(verbose: bool):
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    """The library, and the marshalling module beside it.  The library needs nvcc alone: it is there even where the module
    cannot be built, which is left out where PyTorch or g++ is missing."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        marshal = None
        root = _torch_root()
        if force or not root or _marshal_stale():
            if root and shutil.which("g++"):
                marshal = ex.submit(_build_marshal, root)
            else:
                sys.stderr.write(f"{'g++' if root else 'PyTorch'} is missing: the Python binding's tree-verification calls are not built\n")
        if force or _stale(LIB, False):
            _build_lib(verbose)
        if marshal:
            marshal.result()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
