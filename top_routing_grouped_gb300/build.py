"""Build libmoe.so (the CUDA library behind include/moe.h) in-tree, for sm_103a only.

Each .cu in csrc/ is compiled to an object in parallel, then linked with the CUDA runtime
into ``top_routing_grouped_gb300/libmoe.so``; csrc/binding.cpp becomes the Python module
``_fp8`` beside it.  The results are git-ignored; they are rebuilt wherever they are used (the GPU
host is a different architecture from the build host).
"""
import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libmoe.so")
BINDING = os.path.join(HERE, "_fp8.so")
BUILD_DIR = os.path.join(HERE, "_build")
GENCODE = "arch=compute_103a,code=sm_103a"


def nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def common_flags(extra=()):
    return ["-gencode", GENCODE, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
            "-Xcompiler", "-Wall", "--expt-relaxed-constexpr", *extra]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  [os.path.join(os.path.dirname(HERE), "include", h) for h in ("moe.h", "moe_fp8.h")])


def binding_source():
    return os.path.join(CSRC, "binding.cpp")


def binding_lacks():
    """What this machine lacks for the binding of the 8-bit operators, or None.  The library needs none of it."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return "torch"
    root = os.path.dirname(spec.origin)
    if not shutil.which("g++"):
        return "g++"
    for f in (os.path.join(sysconfig.get_paths()["include"], "Python.h"), os.path.join(root, "include", "ATen", "core", "Tensor.h"),
              os.path.join(root, "lib", "libc10_cuda.so")):
        if not os.path.exists(f):
            return f
    return None


def up_to_date(out=OUT):
    outs = [out, BINDING] if out == OUT and not binding_lacks() else [out]
    if not all(os.path.exists(o) for o in outs):
        return False
    t = min(os.path.getmtime(o) for o in outs)
    return all(os.path.getmtime(f) <= t for f in sources() + headers() + [binding_source()])


def run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def compile_binding(obj):
    """csrc/binding.cpp against the torch that imports it; links in link_binding."""
    import torch
    t = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    run(["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
         *(f"-I{d}" for d in (t, os.path.join(t, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"], cuda)),
         "-c", binding_source(), "-o", obj], "g++ on binding.cpp")
    return obj


def link_binding(obj):
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    run(["g++", "-shared", obj, "-o", BINDING + ".tmp", f"-L{lib}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
         "-lc10_cuda", f"-L{HERE}", "-l:libmoe.so", "-Wl,-rpath,$ORIGIN"], "linking binding.cpp")
    os.replace(BINDING + ".tmp", BINDING)


def build(out=OUT, verbose=False, extra=(), jobs=None):
    """Compile every csrc/*.cu and link ``out``, and for the package's own library the binding of the
    8-bit operators (where the machine has what that needs; else a warning says what it lacks, and importing
    ``fp8`` fails).  Returns the library path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    flags = common_flags(extra)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [cc, *flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    lacks = binding_lacks() if out == OUT else None
    if lacks:
        warnings.warn(f"the binding of the 8-bit operators is not built: {lacks} is missing")
        if os.path.exists(BINDING):
            os.remove(BINDING)  # of another library
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=jobs or min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(compile_binding, os.path.join(BUILD_DIR, "binding.o")) if out == OUT and not lacks else None
        objs = list(ex.map(compile_one, srcs))
    tmp = out + ".tmp"
    cmd = [cc, "-gencode", GENCODE, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", tmp, "-lcudart"]
    run(cmd, "link")
    os.replace(tmp, out)
    if binding:
        link_binding(binding.result())
    return out


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, extra=[a for a in sys.argv[1:] if a != "-v"]))
