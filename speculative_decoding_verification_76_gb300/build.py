"""Build libspecverify.so in-tree with nvcc for sm_103a (no cmake).

Each CUDA source is compiled in parallel to an object file, then linked into
one shared library beside this file.  _native.so, the native part of the Python
binding (csrc/binding.cpp, host code against the installed PyTorch), is linked to
it; the library does not need it, and where PyTorch is not installed the library
alone is built.  Each is built again when one of its sources or headers is newer,
the binding also for another PyTorch or Python.
"""
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libspecverify.so")
NATIVE = os.path.join(HERE, "_native.so")
BINDING = os.path.join(CSRC, "binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libspecverify")
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)]


def _older(path, deps) -> bool:
    return not os.path.exists(path) or \
        any(os.path.getmtime(d) > os.path.getmtime(path) for d in deps)


def _lib_stale() -> bool:
    return _older(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + _headers())


def _torch():
    """The installed PyTorch, or None."""
    try:
        import torch
        return torch
    except ImportError:
        return None


def _built_for(torch) -> str:
    return f"torch {torch.__version__}, python {sys.version}"


def _record():
    return os.path.join(BUILD, "native.txt")  # what _native.so was built for


def _native_stale(torch) -> bool:
    if _older(NATIVE, [BINDING] + _headers()) or not os.path.exists(_record()):
        return True
    with open(_record()) as f:
        return f.read() != _built_for(torch)


def build(force: bool = False, verbose: bool = False) -> str:
    torch = _torch()
    lib = force or _lib_stale()
    native = torch is not None and (force or _native_stale(torch))
    if not lib and not native:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    def compile_binding():
        root = os.path.dirname(torch.__file__)
        obj = os.path.join(BUILD, "binding.cpp.o")
        cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")
        inc = [os.path.join(root, "include"), sysconfig.get_paths()["include"], cuda]
        r = subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC",
                            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                            *(x for d in inc for x in ("-isystem", d)), "-c", BINDING, "-o", obj],
                           capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for {BINDING}:\n{r.stderr}")
        return obj, os.path.join(root, "lib")

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        binding = ex.submit(compile_binding) if native else None
        if lib:
            objs = list(ex.map(compile_one, sources()))
            tmp = LIB + ".tmp"
            r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, "-Xlinker",
                                "-soname=libspecverify.so", *objs], capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stderr}")
            os.replace(tmp, LIB)
    if native:
        obj, torch_lib = binding.result()   # (a failure leaves the library in place)
        tmp = NATIVE + ".tmp"
        r = subprocess.run(["g++", "-shared", "-o", tmp, obj, LIB, "-L" + torch_lib,
                            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
                            "-Wl,-rpath,$ORIGIN"], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, NATIVE)
        with open(_record(), "w") as f:
            f.write(_built_for(torch))
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
