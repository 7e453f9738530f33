"""Builds libkda.so in-tree (linear_attention_state_kda_gb300/_build/) for sm_103a, and the
compiled half of the Python binding (_kda_native.so) that calls it.

Each csrc/*.cu file compiles to an object in parallel with one -gencode
(compute_103a -> sm_103a), then the objects link into one shared library with the CUDA
runtime linked statically. No cmake, no torch extension machinery.
"""
import concurrent.futures as cf
import glob
import hashlib
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libkda.so")
NATIVE = os.path.join(OUT_DIR, "_kda_native.so")
NATIVE_SRC = os.path.join(CSRC, "kda_binding.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler",
              "-fvisibility=hidden", "--expt-relaxed-constexpr", "-I", INCLUDE]


def _nvcc():
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found")
    return p


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stamp(extra=()):
    h = hashlib.sha256()
    for f in _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
            [os.path.join(INCLUDE, "kda.h")]:
        with open(f, "rb") as fh:
            h.update(f.encode() + fh.read())
    h.update(" ".join(ARCH + NVCC_FLAGS + list(extra)).encode())
    return h.hexdigest()


def _native_commands():
    """Compile and link commands of the binding module, against the installed torch's headers."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    inc = os.path.join(root, "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    obj = os.path.join(OUT_DIR, "kda_binding.o")
    cxx = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wno-deprecated",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_path("include"), "-isystem", os.path.join(cuda, "include"),
           "-c", NATIVE_SRC, "-o", obj]
    link = ["g++", "-shared", obj, "-L", OUT_DIR, "-lkda", "-Wl,-rpath,$ORIGIN", "-L",
            os.path.join(root, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
            "-lc10_cuda"]
    return cxx, link


def _native_stamp():
    import sysconfig

    import torch
    h = hashlib.sha256()
    for f in (NATIVE_SRC, os.path.join(INCLUDE, "kda.h")):
        with open(f, "rb") as fh:
            h.update(f.encode() + fh.read())
    h.update(f"{torch.__version__} {sysconfig.get_config_var('SOABI')}".encode())
    return h.hexdigest()


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def build(force=False, verbose=False, extra_flags=()):
    """Builds both; the binding's object compiles while the CUDA files do."""
    os.makedirs(OUT_DIR, exist_ok=True)
    stamp, stamp_file = _native_stamp(), os.path.join(OUT_DIR, "native_stamp")
    if not force and os.path.exists(NATIVE) and os.path.exists(stamp_file):
        with open(stamp_file) as f:
            if f.read() == stamp:
                return _build_lib(force, verbose, extra_flags)
    cxx, link = _native_commands()
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        obj = ex.submit(_run, cxx, "g++ (binding)")
        lib = _build_lib(force, verbose, extra_flags)
        obj.result()
    tmp = NATIVE + f".tmp{os.getpid()}"
    _run([*link, "-o", tmp], "link of the binding")
    os.replace(tmp, NATIVE)
    with open(stamp_file, "w") as f:
        f.write(stamp)
    return lib


def _build_lib(force, verbose, extra_flags):
    stamp_file = os.path.join(OUT_DIR, "stamp")
    stamp = _stamp(extra_flags)
    if not force and os.path.exists(LIB) and os.path.exists(stamp_file):
        with open(stamp_file) as f:
            if f.read() == stamp:
                return LIB
    nvcc = _nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    with open(stamp_file, "w") as f:
        f.write(stamp)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=("-Xptxas", "-v") if "--ptxas" in sys.argv else ()))
