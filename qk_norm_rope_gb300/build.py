"""Builds libst_rope_attn.so in-tree with nvcc for sm_103a (GB300), and
st_bind.*.so, the Python binding of the serving calls, with g++ against torch.

The translation units compile in parallel; the shared objects land in
``qk_norm_rope_gb300/_build/``. Rebuilds only when a source is newer than the
library.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libst_rope_attn.so")
BIND_SRC = os.path.join(CSRC, "st_bind.cpp")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         f"-I{os.path.join(ROOT, 'include')}"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OUT, exist_ok=True)
    srcs = _sources()
    objs = [os.path.join(OUT, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(pair):
        src, obj = pair
        cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, r

    with ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        results = list(ex.map(compile_one, zip(srcs, objs)))
    for src, r in results:
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [NVCC, *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def _bind_name() -> str:
    """Path without suffix of the binding's object and library: the torch and the Python (version and machine) whose
    headers it is compiled against are in it, as neither takes what another's layouts were compiled into."""
    import sysconfig

    import torch
    return os.path.join(OUT, f"st_bind.{torch.__version__}.{sysconfig.get_config_var('SOABI')}")


def _bind_object() -> str:
    """Compiles st_bind.cpp against the running Python and the installed torch."""
    import sysconfig

    import torch
    t = os.path.dirname(os.path.abspath(torch.__file__))
    obj = _bind_name() + ".o"
    head = os.path.join(ROOT, "include", "st_rope_attn.h")
    if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(BIND_SRC), os.path.getmtime(head)):
        return obj
    cuda = os.path.dirname(os.path.dirname(NVCC))
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{os.path.join(ROOT, 'include')}",
           f"-I{sysconfig.get_paths()['include']}", f"-isystem{t}/include", f"-isystem{t}/include/torch/csrc/api/include",
           f"-isystem{cuda}/include", "-c", BIND_SRC, "-o", obj + f".{os.getpid()}.tmp"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for st_bind.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(obj + f".{os.getpid()}.tmp", obj)
    return obj


def build_bind(obj: str | None = None) -> str:
    """The Python binding of the serving calls, linked to libst_rope_attn.so beside it."""
    import torch
    build_lib = build()
    obj = obj or _bind_object()
    so = _bind_name() + ".so"
    if os.path.exists(so) and os.path.getmtime(so) >= os.path.getmtime(obj):
        return so
    t = os.path.join(os.path.dirname(os.path.abspath(torch.__file__)), "lib")
    tmp = so + f".{os.getpid()}.tmp"
    cmd = ["g++", "-shared", obj, "-o", tmp, f"-L{t}", "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           f"-L{os.path.dirname(build_lib)}", "-l:libst_rope_attn.so", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{t}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed for st_bind.so:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, so)
    return so


def build_all(force: bool = False, verbose: bool = False) -> None:
    """The library and the binding, their compilers side by side."""
    os.makedirs(OUT, exist_ok=True)
    with ThreadPoolExecutor(max_workers=1) as ex:
        obj = ex.submit(_bind_object)
        build(force=force, verbose=verbose)
        build_bind(obj.result())


if __name__ == "__main__":
    build_all(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
