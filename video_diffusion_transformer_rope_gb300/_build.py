"""Build libvdx.so in-tree with nvcc for sm_103a (GB300), and with the host compiler the Python entry of
the streaming calls (_streaming_py.so, where a PyTorch with CUDA and the interpreter's headers are installed;
the library itself needs neither).

Each .cu file is compiled to an object in parallel, then linked into one shared library with
the CUDA runtime linked statically (so the library loads on machines without the NVIDIA driver;
libcuda is reached only when a call is made).  Run `python -m
video_diffusion_transformer_rope_gb300._build` or call build().
"""
import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import platform
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libvdx.so")
SOURCES = ["vdx_capi.cu", "attn_fwd_sm103.cu", "attn_fwd_f32.cu", "vdx_noalloc.cu", "kv_capi.cu",
           "kv_append.cu", "attn_rows.cu", "attn_tiles_sm103.cu"]
EXT = os.path.join(PKG, "_streaming_py.so")
EXT_STAMP = os.path.join(OUT_DIR, "streaming_py.torch")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
         "-I", INCLUDE, "-I", CSRC]


def _nvcc():
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libvdx.so")
    return exe


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "vdx.h"), __file__]
    return files


def _ext_lacks(base):
    """What the Python entry would need and does not find, PyTorch being installed in `base` (None: not at all)."""
    if base is None:
        return "PyTorch is not installed"
    for name in ("lib/libc10_cuda.so", "include/c10/cuda/CUDAStream.h"):
        if not os.path.exists(os.path.join(base, name)):
            return f"this PyTorch has no CUDA part ({name})"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "this Python has no headers (Python.h)"
    return None


def _torch_base():
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _torch():
    """PyTorch's folder and version, without importing it; None where the Python entry cannot be built with it."""
    base = _torch_base()
    return None if _ext_lacks(base) else (base, importlib.metadata.version("torch"))


def _ext_stamp(version):
    """What the Python entry is bound to: the PyTorch and interpreter it was compiled against, the machine."""
    return f"{version} {sys.version} {platform.machine()}"


def _ext_stale(torch):
    if torch is None:
        return False
    if not os.path.exists(EXT) or not os.path.exists(EXT_STAMP):
        return True
    return open(EXT_STAMP).read() != _ext_stamp(torch[1])


def _stale():
    if not os.path.exists(LIB) or _ext_stale(_torch()):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in _deps())


def _build_ext(torch):
    base, version = torch
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        raise RuntimeError("g++ not found: a C++ compiler is required to build the Python entry of the streaming calls")
    include = [INCLUDE, base + "/include", base + "/include/torch/csrc/api/include", sysconfig.get_paths()["include"],
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")]
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", *("-I" + i for i in include),
           os.path.join(CSRC, "streaming_py.cpp"), "-o", EXT + ".tmp", "-L" + base + "/lib", "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on streaming_py.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(EXT + ".tmp", EXT)
    with open(EXT_STAMP, "w") as f:
        f.write(_ext_stamp(version))
    return EXT


def build(force=False, verbose=False):
    """Compile and link libvdx.so, and the Python entry of the streaming calls, if any source is newer.
    Returns the library path.  Where the Python entry cannot be built (no PyTorch with CUDA, no headers) the
    library is built alone and the streaming calls say why; where its compilation fails, the library is linked
    all the same before that is raised."""
    if not force and not _stale():
        return LIB
    nvcc = _nvcc()
    os.makedirs(OUT_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        with open(os.path.join(OUT_DIR, src + ".ptxas.txt"), "w") as f:
            f.write(r.stderr)
        return obj

    torch = _torch()
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        ext = ex.submit(_build_ext, torch) if torch else None
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if ext:
        ext.result()
    if verbose:
        for src in SOURCES:
            print(open(os.path.join(OUT_DIR, src + ".ptxas.txt")).read())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
