"""Build librmsnorm.so (the C-ABI CUDA library) in-tree for sm_103a, and
_fp8_torch.so, the torch binding of its 8-bit entry points.

Each translation unit under csrc/ (and csrc/fp8/) is compiled by nvcc in parallel into
_build/, then linked into rmsnorm_fwd_bwd_02_gb300/librmsnorm.so. A unit is
rebuilt when it, any header under csrc/ or include/, or this file is newer
than its object. No cmake; plain nvcc with one -gencode.

    python -m rmsnorm_fwd_bwd_02_gb300.build [--force] [--ptxas-verbose]
"""
import glob
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
SOURCE_DIRS = (CSRC, os.path.join(CSRC, "fp8"))
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "librmsnorm.so")
TORCH_SRC = os.path.join(CSRC, "fp8", "fp8_torch.cpp")
TORCH_LIB = os.path.join(PKG, "_fp8_torch.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-I" + INCLUDE, "-I" + CSRC]


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _newest_dep_mtime():
    deps = glob.glob(os.path.join(INCLUDE, "*.h"))
    for d in SOURCE_DIRS:
        deps += glob.glob(os.path.join(d, "*.cuh")) + glob.glob(os.path.join(d, "*.h"))
    deps.append(os.path.abspath(__file__))
    return max(os.path.getmtime(d) for d in deps)


def _compile(src, obj, extra):
    cmd = [_nvcc()] + NVCC_FLAGS + extra + ["-c", src, "-o", obj + ".tmp"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n"
                           f"{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(obj + ".tmp", obj)
    return r.stdout + r.stderr


def build_torch(force: bool = False) -> str:
    """The torch binding, compiled by g++ against the torch that is installed."""
    import sysconfig

    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    os.makedirs(BUILD, exist_ok=True)
    stamp = os.path.join(BUILD, "fp8_torch.version")    # the torch it was built against
    made = ""
    if os.path.exists(stamp) and os.path.exists(TORCH_LIB):
        with open(stamp) as f:
            made = f.read()
    newest = max(os.path.getmtime(f) for f in (TORCH_SRC, os.path.join(INCLUDE, "rmsnorm.h"),
                                               os.path.abspath(__file__)))
    if not force and made == torch.__version__ and os.path.getmtime(TORCH_LIB) >= newest:
        return TORCH_LIB
    nvcc = _nvcc()
    cuda = (os.path.dirname(os.path.dirname(nvcc)) if os.path.sep in nvcc
            else os.environ.get("CUDA_HOME", "/usr/local/cuda"))
    tmp = TORCH_LIB + ".tmp.%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I" + INCLUDE,
           "-I" + sysconfig.get_paths()["include"], "-isystem" + os.path.join(cuda, "include"),
           "-isystem" + os.path.join(root, "include"),
           "-isystem" + os.path.join(root, "include", "torch", "csrc", "api", "include"),
           TORCH_SRC, "-o", tmp, "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {os.path.basename(TORCH_SRC)}:\n{' '.join(cmd)}\n"
                           f"{r.stdout}\n{r.stderr}")
    os.replace(tmp, TORCH_LIB)
    with open(stamp, "w") as f:
        f.write(torch.__version__)
    return TORCH_LIB


def build(force: bool = False, ptxas_verbose: bool = False, jobs: int = 0) -> str:
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(s for d in SOURCE_DIRS for s in glob.glob(os.path.join(d, "*.cu")))
    dep_t = _newest_dep_mtime()
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []
    binding = ThreadPoolExecutor(max_workers=1)
    torch_built = binding.submit(build_torch, force)
    todo = []
    objs = []
    for s in sources:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if (force or ptxas_verbose or not os.path.exists(o)
                or os.path.getmtime(o) < max(dep_t, os.path.getmtime(s))):
            todo.append((s, o))
    logs = []
    if todo:
        n = jobs or min(len(todo), os.cpu_count() or 4)
        with ThreadPoolExecutor(max_workers=n) as ex:
            for log in ex.map(lambda so: _compile(so[0], so[1], extra), todo):
                logs.append(log)
    if (todo or not os.path.exists(LIB)
            or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs)):
        tmp = LIB + ".tmp.%d" % os.getpid()
        cmd = [_nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    torch_built.result()
    binding.shutdown()
    if ptxas_verbose:
        sys.stdout.write("".join(logs))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv,
                ptxas_verbose="--ptxas-verbose" in sys.argv))
