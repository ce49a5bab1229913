"""Build ``libpagedkv.so`` in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` translation unit (and the host-only ``csrc/*.cpp``) is
compiled in parallel (one nvcc process each), then linked into a shared library with the CUDA runtime linked
statically, so the library loads without a GPU driver present.  Objects go to
``_build/`` beside this file.  The host compiler builds ``binding/marshal.cpp``,
the argument marshalling of the calls whose GPU time is a few microseconds, as
the CPython module ``_marshal.so`` next to it, against the installed PyTorch; only
those calls need it.  Usage: ``python -m paged_kv_cache_52_gb300.build``.
"""

from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libpagedkv.so")
MARSHAL_SRC = os.path.join(HERE, "binding", "marshal.cpp")
MARSHAL_PATH = os.path.join(HERE, "_marshal.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden", "-Xptxas", "-v"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpagedkv.so")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def _compile(nvcc: str, src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
    if src.endswith(".cpp"):   # host-only code: the host compiler, through nvcc
        cmd = [nvcc, "-O3", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden,-Wall",
               "-c", src, "-o", obj]
    else:
        cmd = [nvcc, *ARCH, *CFLAGS, "-c", src, "-o", obj]
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{proc.stdout}{proc.stderr}")
    return obj, proc.stderr


def _run(cmd):
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"{' '.join(cmd)}\n{proc.stdout}{proc.stderr}")


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("PyTorch is required to build the Python binding")
    return list(spec.submodule_search_locations)[0]


def _compile_marshal(nvcc: str) -> str:
    obj = os.path.join(BUILD_DIR, "marshal.o")
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall",
          f"-I{sysconfig.get_paths()['include']}", f"-isystem{inc}",
          f"-isystem{os.path.join(inc, 'torch', 'csrc', 'api', 'include')}", f"-isystem{cuda}",
          "-c", MARSHAL_SRC, "-o", obj])
    return obj


def _link_marshal(obj: str) -> None:
    lib = os.path.join(_torch_dir(), "lib")
    tmp = MARSHAL_PATH + ".tmp"
    _run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, f"-L{HERE}", "-l:libpagedkv.so",
          f"-L{lib}", "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10",
          "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"])
    os.replace(tmp, MARSHAL_PATH)


def build(verbose: bool = False) -> str:
    """Compile every source and link ``libpagedkv.so`` and ``_marshal.so``;
    returns the library's path."""
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        marshal = ex.submit(_compile_marshal, nvcc)
        results = list(ex.map(lambda s: _compile(nvcc, s), srcs))
    if verbose:
        for obj, log in results:
            sys.stderr.write(f"== {os.path.basename(obj)}\n{log}")
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{proc.stdout}{proc.stderr}")
    os.replace(tmp, LIB_PATH)
    try:
        _link_marshal(marshal.result())
    except RuntimeError as e:
        raise RuntimeError("libpagedkv.so is built; _marshal.so, which the speculative step's "
                           f"calls need, is not:\n{e}") from e
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
