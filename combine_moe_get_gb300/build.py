"""Build ``libmoe_get.so`` in place: nvcc for sm_103a, one object per .cu
(compiled in parallel), linked against the shared CUDA runtime so that the
library and PyTorch share one runtime instance in a process. Also the Python
module ``_marshal`` (csrc/marshal.cpp), by the host compiler against torch."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmoe_get.so")
# the same library compiled with MOE_PROFILE: every kernel warp records its start and end (moe_trace_enable)
TRACE_LIB = os.path.join(HERE, "libmoe_get_trace.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe_get.so")


def _cuda_lib_dirs(nvcc: str) -> list[str]:
    root = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    dirs = [os.path.join(root, "lib64")] + glob.glob(os.path.join(root, "targets", "*", "lib"))
    return [d for d in dirs if os.path.isdir(d)]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def build(force: bool = False, verbose: bool = False, defines: tuple = (), lib: str = LIB,
          build_dir: str = BUILD_DIR) -> str:
    """Compile and link the library in place. `defines` (e.g. ("MOE_TUNE_X=4",))
    builds a variant with other compile-time settings; the default build has none."""
    if not force and up_to_date(lib):
        return lib
    nvcc = _nvcc()
    os.makedirs(build_dir, exist_ok=True)
    common = [nvcc, *ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "-I", INCLUDE, "--expt-relaxed-constexpr", *(f"-D{d}" for d in defines)]

    def compile_one(src: str) -> str:
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        cmd = common + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = lib + f".tmp{os.getpid()}"
    link = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs]
    for d in _cuda_lib_dirs(nvcc):
        link += ["-Xlinker", f"-rpath,{d}"]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


def build_trace(force: bool = False, verbose: bool = False) -> str:
    """libmoe_get_trace.so: the library compiled with MOE_PROFILE (per-warp timer records)."""
    return build(force, verbose, defines=("MOE_PROFILE=1",), lib=TRACE_LIB, build_dir=BUILD_DIR + "_trace")


def build_marshal(force: bool = False) -> str:
    """Argument marshalling of the small calls. The file's name has the versions of torch and Python in it, whose
    binary interfaces it is compiled against: another version's is never taken for it."""
    import torch

    path = os.path.join(HERE, f"_marshal-{torch.__version__}-{sysconfig.get_config_var('SOABI')}.so")
    src = os.path.join(CSRC, "marshal.cpp")
    inputs = [src, os.path.join(INCLUDE, "moe_get.h"), os.path.abspath(__file__)]
    if not force and os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in inputs):
        return path
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    includes = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(root, "include"),
                os.path.join(root, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    tmp = path + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *(f"-I{d}" for d in includes), src, "-o", tmp, f"-L{os.path.join(root, 'lib')}", "-ltorch_python",
           "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{os.path.join(root, 'lib')}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)
    return path


if __name__ == "__main__":
    print(build(force=True, verbose=True))
