"""Builds libdetffn.so in-tree for sm_103a (GB300), and where PyTorch is
installed the native binding.

Each ``csrc/*.cu`` file is compiled in parallel with nvcc and the objects are
linked into ``gemm_deterministic_bf16_gb300/libdetffn.so``; ``csrc/bind.cpp``
is compiled with the host compiler against PyTorch's headers and linked into
``_native.so`` beside it.  No cmake; the whole build takes well under two
minutes.
"""
import concurrent.futures as cf
import glob
import os
import importlib.util
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "libdetffn.so")
NATIVE = os.path.join(PKG, "_native.so")
BUILD = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall", "-Xcompiler", "-fvisibility=hidden",
           "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _nvcc():
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found; libdetffn needs the CUDA toolkit")
    return exe


def _torch():
    """PyTorch's folder, without importing it; None where it is not installed."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _stale(obj, src, deps):
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(p) > t for p in [src, *deps])


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compiles every source and links libdetffn.so and _native.so (without
    PyTorch the library alone); returns the former's path."""
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(ROOT, "include", "*.h")))
    jobs = []
    for src in srcs:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        if force or _stale(obj, src, deps):
            jobs.append([nvcc, *ARCH, *NVFLAGS, *extra, "-c", src, "-o", obj])

    torch_dir = _torch()
    bind_src, bind_obj = os.path.join(CSRC, "bind.cpp"), os.path.join(BUILD, "bind.o")
    bind = torch_dir is not None and (force or _stale(bind_obj, bind_src, deps + [os.path.join(torch_dir, "version.py")]))
    if bind:
        inc = [os.path.join(ROOT, "include"), sysconfig.get_paths()["include"], os.path.join(torch_dir, "include"),
               os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")]
        jobs.append(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *("-I" + i for i in inc), "-c",
                     bind_src, "-o", bind_obj])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("build failed:\n%s\n%s%s" % (" ".join(cmd), r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        list(ex.map(run, jobs))
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    if force or jobs or not os.path.exists(OUT):
        tmp = OUT + ".tmp.%d" % os.getpid()
        run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-ldl", "-lrt", "-lpthread"])
        os.replace(tmp, OUT)
    if torch_dir is not None and (bind or not os.path.exists(NATIVE)):
        lib = os.path.join(torch_dir, "lib")
        tmp = NATIVE + ".tmp.%d" % os.getpid()
        run(["g++", "-shared", "-o", tmp, bind_obj, "-L" + PKG, "-l:libdetffn.so", "-Wl,-rpath,$ORIGIN", "-L" + lib,
             "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath," + lib])
        os.replace(tmp, NATIVE)
    return OUT


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
