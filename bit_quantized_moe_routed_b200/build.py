"""Build libmoeq.so in-tree with nvcc for sm_100a.

``python -m bit_quantized_moe_routed_b200.build [--force] [-v]``.  Each
``csrc/*.cu`` compiles to ``_build/<name>.o`` (in parallel, skipped when up
to date), then they link into ``bit_quantized_moe_routed_b200/libmoeq.so``.
No GPU is needed: nvcc cross-compiles.  ``csrc/torch_calls.cpp`` (the torch
side of the dense operators' Python calls) compiles with g++ against the
installed torch into ``_torch_calls.so`` beside it, again where that torch or
Python is another one; without torch or the headers it is left out, and the
library and the rest of the binding build and load as they do with it.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import hashlib
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
SO = os.path.join(PKG, "libmoeq.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
CALLS_SRC = os.path.join(CSRC, "torch_calls.cpp")
CALLS_SO = os.path.join(PKG, "_torch_calls.so")
CALLS_STAMP = os.path.join(BUILD, "torch_calls.stamp")   # what CALLS_SO was built against

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
          "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _deps_mtime() -> float:
    hdrs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hdrs), default=0.0)


def _compile(src: str, force: bool, verbose: bool, extra: list) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    if (not force and os.path.exists(obj)
            and os.path.getmtime(obj) >= max(os.path.getmtime(src), _deps_mtime())):
        return obj
    cmd = [NVCC] + ARCH + CFLAGS + extra + ["-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, flush=True)
    return obj


def _torch_root():
    """The installed torch's directory (without importing it), or None."""
    try:
        spec = importlib.util.find_spec("torch")
    except (ImportError, ValueError):
        return None
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _build_calls(force: bool, verbose: bool) -> None:
    root = _torch_root()
    python_inc = sysconfig.get_paths()["include"]
    needed = [os.path.join(root, "include", "ATen", "ATen.h")] if root else []
    needed.append(os.path.join(python_inc, "Python.h"))
    missing = [h for h in needed if not os.path.exists(h)]
    if not root or missing:
        print(f"{os.path.basename(CALLS_SO)} is not built (the dense operators' Python calls need it): "
              f"{'torch is not installed' if not root else 'no ' + ', '.join(missing)}", file=sys.stderr)
        return
    with open(os.path.join(root, "version.py"), "rb") as f:   # version, CUDA version and commit
        key = hashlib.sha256(f.read() + f"{root}\n{sys.version}\n".encode()).hexdigest()
    deps = (CALLS_SRC, os.path.join(INCLUDE, "moeq.h"))
    if (not force and os.path.exists(CALLS_SO) and os.path.exists(CALLS_STAMP)
            and os.path.getmtime(CALLS_SO) >= max(os.path.getmtime(f) for f in deps)):
        with open(CALLS_STAMP) as f:
            if f.read().strip() == key:
                return
    import torch
    cuda = os.path.dirname(os.path.dirname(NVCC))
    tmp = CALLS_SO + f".tmp{os.getpid()}"
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), python_inc, INCLUDE]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-DUSE_CUDA",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for d in inc:
        cmd += ["-isystem" if d != INCLUDE else "-I", d]
    cmd += [CALLS_SRC, "-o", tmp, "-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu",
            "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {CALLS_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS_SO)
    with open(CALLS_STAMP + f".tmp{os.getpid()}", "w") as f:
        f.write(key + "\n")
    os.replace(f.name, CALLS_STAMP)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(s, force or ptxas_info, verbose or ptxas_info, extra), srcs))
    newest = max(os.path.getmtime(o) for o in objs)
    if force or not os.path.exists(SO) or os.path.getmtime(SO) < newest:
        tmp = SO + f".tmp{os.getpid()}"
        cmd = [NVCC] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        os.replace(tmp, SO)
    _build_calls(force, verbose)
    return SO


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="rebuild with -Xptxas -v (registers, spills)")
    a = ap.parse_args(argv)
    print(build(a.force, a.verbose, a.ptxas_info))


if __name__ == "__main__":
    sys.exit(main())
