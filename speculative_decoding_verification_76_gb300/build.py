"""Build libspecverify.so in-tree with nvcc for sm_103a (no cmake).

Each CUDA source is compiled in parallel to an object file, then linked into
one shared library beside this file; _native.so, the native part of the Python
binding (csrc/binding.cpp, host code against the installed PyTorch), is linked to
it.  Rebuilds only when a source or header is newer than the two.
"""
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
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


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(NATIVE):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(NATIVE))
    deps = sources() + [BINDING] + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
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
        import torch
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
        native = ex.submit(compile_binding)
        objs = list(ex.map(compile_one, sources()))
        native = native.result()
    tmp = LIB + ".tmp"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, "-Xlinker", "-soname=libspecverify.so",
                        *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    obj, torch_lib = native
    tmp = NATIVE + ".tmp"
    r = subprocess.run(["g++", "-shared", "-o", tmp, obj, LIB, "-L" + torch_lib, "-ltorch_python",
                        "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, NATIVE)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
