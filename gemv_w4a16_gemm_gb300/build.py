"""Build libw4q.so in-tree: one nvcc per translation unit (in parallel) for
sm_103a, then one shared-library link; and _w4q_binding.so, the Python module
that marshals the decode-step operators' arguments, by g++ against the
installed torch's headers.  No cmake."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libw4q.so")
BINDING = os.path.join(PKG, "_w4q_binding.so")
SOURCES = ("api.cu", "pack.cu", "pack_compact.cu", "gemv_w4.cu", "gemv_w4_cluster.cu",
           "gemv_w4_umma.cu", "w8.cu", "gemv_w8_umma.cu", "noalloc.cu", "selftest.cu",
           "api_decode.cu", "kv8_append.cu", "kv8_attention.cu", "moe_w4.cu")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags(extra=()):
    return ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                   "-I", INCLUDE, "-I", CSRC, *extra]


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s\n%s" % (cmd[0], r.stdout, r.stderr))


def _torch_dir() -> str:
    import importlib.util
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("_w4q_binding.so needs torch's headers: torch is not installed")
    return os.path.dirname(spec.origin)


def _torch_id() -> str:
    """The installed torch that the Python module is compiled against."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return _torch_dir() + "\n" + f.read()


def _compile_binding(force: bool) -> str:
    """The Python module of binding.cpp, compiled against the torch headers (no torch import)."""
    src, obj, stamp = os.path.join(CSRC, "binding.cpp"), os.path.join(BUILD, "binding.o"), os.path.join(BUILD, "binding.torch")
    torch_id, was = _torch_id(), None
    if os.path.exists(stamp):
        with open(stamp) as f:
            was = f.read()
    if force or was != torch_id or _stale(obj, [src, os.path.join(INCLUDE, "w4q.h")]):
        inc = os.path.join(_torch_dir(), "include")
        cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
        _run(["g++", "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE, "-isystem", inc,
              "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
              "-isystem", sysconfig.get_paths()["include"], "-c", src, "-o", obj])
        with open(stamp, "w") as f:
            f.write(torch_id)
    return obj


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every CUDA translation unit and link libw4q.so; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(os.path.join(INCLUDE, "w4q.h"))
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        path = os.path.join(CSRC, src)
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        if force or ptxas_info or _stale(obj, [path, *headers]):
            cmd = [cc, *_flags(extra), "-c", path, "-o", obj]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
            if verbose or ptxas_info:
                sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding, force)
        objs = list(ex.map(compile_one, SOURCES))
        # the library needs neither torch nor its headers, and is there without them
        if force or _stale(LIB, [*objs, os.path.abspath(__file__)]):
            tmp = LIB + ".tmp%d" % os.getpid()
            cmd = [cc, *ARCH, "-shared", "-Xlinker", "-soname=" + os.path.basename(LIB), "-o", tmp, *objs, "-cudart", "static"]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
            os.replace(tmp, LIB)
        binding_obj = binding.result()
    if force or _stale(BINDING, [binding_obj, LIB]):
        tmp = BINDING + ".tmp%d" % os.getpid()
        lib = os.path.join(_torch_dir(), "lib")
        # the library is needed by its name, and found beside the module: a copied or moved package uses its own
        _run(["g++", "-shared", "-o", tmp, binding_obj, LIB, "-L" + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu",
              "-ltorch_python", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib])
        os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
