"""Build librmsnorm.so (the C-ABI CUDA library) in-tree for sm_103a, and
_fp8_torch.so and _heads_torch.so, the torch bindings of its 8-bit entry
points and of those on attention heads.

Each translation unit under csrc/ (and csrc/fp8/, csrc/heads/) is compiled by nvcc in parallel into
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
SOURCE_DIRS = (CSRC, os.path.join(CSRC, "fp8"), os.path.join(CSRC, "heads"))
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "librmsnorm.so")
TORCH_MODULES = ("fp8", "heads")     # csrc/NAME/NAME_torch.cpp -> _NAME_torch.so

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


def build_torch(name: str, force: bool = False) -> str:
    """A torch binding, compiled by g++ against the torch that is installed."""
    import sysconfig

    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    src = os.path.join(CSRC, name, f"{name}_torch.cpp")
    lib = os.path.join(PKG, f"_{name}_torch.so")
    os.makedirs(BUILD, exist_ok=True)
    stamp = os.path.join(BUILD, f"{name}_torch.version")    # the torch it was built against
    made = ""
    if os.path.exists(stamp) and os.path.exists(lib):
        with open(stamp) as f:
            made = f.read()
    newest = max(os.path.getmtime(f) for f in (src, os.path.join(CSRC, "torch", "binding.h"),
                                               os.path.join(INCLUDE, "rmsnorm.h"),
                                               os.path.abspath(__file__)))
    if not force and made == torch.__version__ and os.path.getmtime(lib) >= newest:
        return lib
    nvcc = _nvcc()
    cuda = (os.path.dirname(os.path.dirname(nvcc)) if os.path.sep in nvcc
            else os.environ.get("CUDA_HOME", "/usr/local/cuda"))
    tmp = lib + ".tmp.%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I" + INCLUDE,
           "-I" + sysconfig.get_paths()["include"], "-isystem" + os.path.join(cuda, "include"),
           "-isystem" + os.path.join(root, "include"),
           "-isystem" + os.path.join(root, "include", "torch", "csrc", "api", "include"),
           src, "-o", tmp, "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {os.path.basename(src)}:\n{' '.join(cmd)}\n"
                           f"{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    with open(stamp, "w") as f:
        f.write(torch.__version__)
    return lib


def build(force: bool = False, ptxas_verbose: bool = False, jobs: int = 0) -> str:
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(s for d in SOURCE_DIRS for s in glob.glob(os.path.join(d, "*.cu")))
    dep_t = _newest_dep_mtime()
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []
    binding = ThreadPoolExecutor(max_workers=len(TORCH_MODULES))
    torch_built = [binding.submit(build_torch, name, force) for name in TORCH_MODULES]
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
    for f in torch_built:
        f.result()
    binding.shutdown()
    if ptxas_verbose:
        sys.stdout.write("".join(logs))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv,
                ptxas_verbose="--ptxas-verbose" in sys.argv))
