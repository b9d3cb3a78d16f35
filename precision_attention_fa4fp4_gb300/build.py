"""Compile the CUDA library in-tree for sm_103a: every .cu under csrc/ with
nvcc in parallel, then one shared library ``libfa4fp4.so`` next to this file, and
beside it the native Python binding of the calls of every layer (cache, norm and
rotation, cross attention), ``_cache_binding`` with the running Python's suffix (g++, against the installed torch; left out, with a
note, where torch or Python's headers are not installed: the library itself needs
neither).
Run ``python -m precision_attention_fa4fp4_gb300.build`` or call ``build()``."""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfa4fp4.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
         "--expt-relaxed-constexpr"]


BINDING = os.path.join(HERE, "_cache_binding" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
STAMP = os.path.join(OUT_DIR, "cache_binding.torch")


def _cuda_home() -> str:
    return os.environ.get("CUDA_HOME", "/usr/local/cuda")


def _nvcc() -> str:
    p = os.path.join(_cuda_home(), "bin", "nvcc")
    return p if os.path.exists(p) else "nvcc"


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _stale(out: str, deps: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_commands(force: bool, header: str) -> tuple[list[str] | None, list[str] | None, str]:
    """The binding's compile and link commands where they are needed, and what it
    is built against."""
    include = sysconfig.get_paths()["include"]
    try:
        import torch
    except ImportError:
        torch = None
    if torch is None or not os.path.exists(os.path.join(include, "Python.h")):
        print("the native Python binding is left out: "
              + ("torch is not installed" if torch is None else f"no Python.h in {include}"), file=sys.stderr)
        return None, None, ""
    src = os.path.join(CSRC, "cache_binding.cpp")
    obj = os.path.join(OUT_DIR, "cache_binding.o")
    root = os.path.dirname(torch.__file__)
    against = f"torch {torch.__version__}, {os.path.basename(BINDING)}"
    built = ""
    if os.path.exists(STAMP):
        with open(STAMP) as f:
            built = f.read()
    parts = [os.path.join(CSRC, f) for f in ("binding.h", "cross_binding.h")]
    fresh = not force and built == against and not _stale(obj, [src, header, *parts])
    compile_ = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                "-I", include, "-isystem", os.path.join(root, "include"),
                "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
                "-isystem", os.path.join(_cuda_home(), "include"), "-c", src, "-o", obj]
    lib = os.path.join(root, "lib")
    link = ["g++", "-shared", "-o", BINDING + f".{os.getpid()}.tmp", obj, "-L" + HERE, "-lfa4fp4", "-L" + lib,
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]
    return (None if fresh else compile_), (None if fresh and not _stale(BINDING, [obj]) else link), against


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(os.path.dirname(HERE), "include", "fa4fp4.h"))
    nvcc = _nvcc()
    jobs = []
    objs = []
    for src in sources():
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            jobs.append([nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj])
    compile_binding, link_binding, against = _binding_commands(force, headers[-1])
    relink = force or bool(jobs)
    if compile_binding:
        jobs.insert(0, compile_binding)
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(12, len(jobs))) as ex:
            for res in ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs):
                if res.returncode != 0:
                    raise RuntimeError("compilation failed:\n" + " ".join(res.args) + "\n" + res.stderr)
                if verbose and res.stderr:
                    print(res.stderr)
    if relink or _stale(LIB, objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("link failed:\n" + res.stderr)
        os.replace(tmp, LIB)
    if link_binding:
        res = subprocess.run(link_binding, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("link failed:\n" + res.stderr)
        os.replace(link_binding[3], BINDING)
        with open(STAMP, "w") as f:
            f.write(against)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
