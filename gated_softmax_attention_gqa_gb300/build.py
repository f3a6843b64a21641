"""Build libgattn.so (the CUDA kernels and the C ABI) for sm_103a, in-tree.

Each .cu file compiles in parallel with nvcc, then one shared library is linked
with the CUDA runtime statically, so loading it needs no GPU and no libcudart
of a particular version.  Set GATTN_PTXAS_VERBOSE=1 to print register and
shared-memory usage per kernel.  Beside it the CPython module _qcache.so (the
4-bit cache's tensor checks and calls) compiles with g++ against the installed
torch and links to the library.
"""
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libgattn.so")
SOURCES = ["api.cu", "prologue.cu", "prefill_tc.cu", "prefill_pair.cu", "prefill_fp32.cu", "decode.cu", "decode_noalloc.cu",
           "oproj.cu", "qcache.cu", "decode_qcache.cu", "qcache_api.cu"]
BINDING = "qcache_binding.cpp"
MODULE = os.path.join(HERE, "_qcache.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags():
    f = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
    if os.environ.get("GATTN_PTXAS_VERBOSE"):
        f += ["-Xptxas", "-v"]
    return f


def _binding_compile(obj):
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    dirs = [inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"], INCLUDE,
            os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-c", os.path.join(CSRC, BINDING), "-o", obj] + [
        f"-I{d}" for d in dirs]


def _binding_link(obj, to):
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ["g++", "-shared", "-o", to, obj, f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda",
            f"-L{HERE}", "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(MODULE):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(MODULE))
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "gattn.h"), __file__]
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    exe = nvcc()
    procs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [exe] + _flags() + ["-c", os.path.join(CSRC, src), "-o", obj]
        procs.append((src, obj, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    binding = os.path.join(BUILD, BINDING.replace(".cpp", ".o"))
    procs.append((BINDING, binding, subprocess.Popen(_binding_compile(binding), stdout=subprocess.PIPE,
                                                     stderr=subprocess.STDOUT, text=True)))
    objs, failed = [], []
    for src, obj, p in procs:
        out, _ = p.communicate()
        if out and (verbose or p.returncode != 0 or os.environ.get("GATTN_PTXAS_VERBOSE")):
            sys.stderr.write(f"--- {src}\n{out}")
        if p.returncode != 0:
            failed.append(src)
        objs.append(obj)
    if failed:
        raise RuntimeError("the compiler failed for: " + ", ".join(failed))
    objs.remove(binding)
    tmp = LIB + ".tmp%d" % os.getpid()
    subprocess.run([exe] + ARCH + ["-shared", "-cudart", "static", "-Xlinker", "-soname=" + os.path.basename(LIB), "-o",
                    tmp] + objs, check=True)
    os.replace(tmp, LIB)
    tmp = MODULE + ".tmp%d" % os.getpid()
    subprocess.run(_binding_link(binding, tmp), check=True)
    os.replace(tmp, MODULE)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
