"""Build libkda.so (the C-ABI CUDA library) in-tree for sm_100a, and the latent-attention
binding's extension module.

    python -m kimi_delta_attention_19_b200.build

Each .cu under csrc/ is compiled by nvcc in parallel into _build/, then linked
into kimi_delta_attention_19_b200/libkda.so; csrc/latent_host.cpp becomes
_latent_host.so beside it. Nothing is JIT-compiled at import.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libkda.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-Xptxas", "-v", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    cuda_home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    p = os.path.join(cuda_home, "bin", "nvcc")
    return p if os.path.exists(p) else (shutil.which("nvcc") or "nvcc")


def _compile(src: str, obj: str, extra: list[str] | None = None) -> str:
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, *(extra or []), "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return r.stderr  # ptxas -v report


# Test-only variants of the library. In one the first wait on the inputs in each tensor-core prefill
# kernel, and any wait in a latent-attention kernel, gives up after 64 clocks, so a test can
# watch the kernels' bail-out path (status word set, copies and products drained, tensor memory
# freed) run on the GPU and the context stay usable. The product never loads them.
SHORTWAIT_LIB = os.path.join(PKG, "libkda_shortwait.so")
SHORTWAIT_DEFINES = {"kda_prefill_tc.cu": ["-DKDA_FIRST_WAIT_LIMIT=64", "-DKDA_FIRST_WAIT_STUCK=1"],
                     **{f"kda_latent_{k}.cu": ["-DKDA_LATENT_WAIT_CYCLES=64"]
                        for k in ("fwd", "bwd", "decode")}}

# A second one, whose latent-attention kernels give up the wait for a unit's last products, when
# every other role is done or about to be.
LASTWAIT_LIB = os.path.join(PKG, "libkda_lastwait.so")
LASTWAIT_DEFINES = {f"kda_latent_{k}.cu": ["-DKDA_LATENT_RESULTS_GIVEN_UP"]
                    for k in ("fwd", "bwd", "decode")}

VARIANTS = {"shortwait": (SHORTWAIT_LIB, SHORTWAIT_DEFINES),
            "lastwait": (LASTWAIT_LIB, LASTWAIT_DEFINES)}


def _link(lib: str, objs: list[str]) -> None:
    if os.path.exists(lib) and os.path.getmtime(lib) >= max(os.path.getmtime(o) for o in objs):
        return
    cmd = [_nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", lib, *objs]
    subprocess.run(cmd, check=True)


# The latent-attention binding's extension module (csrc/latent_host.cpp), for this interpreter
# and this torch. Without it (no Python.h, no torch headers, another g++) the library is whole and
# the binding's calls take the host 5 to 11 us longer, so that it cannot be built is a warning.
HOST_MODULE = os.path.join(PKG, "_latent_host.so")


def _build_host(src: str) -> str:
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    libs = os.path.join(root, "lib")
    cuda_home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    inc = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda_home, "include")]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-isystem{i}" for i in inc), src, "-o", HOST_MODULE, f"-L{libs}",
           f"-Wl,-rpath,{libs}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}\n{r.stderr}")
    return r.stderr


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = sources + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        [os.path.join(ROOT, "include", "kda.h")]
    newest_dep = max(os.path.getmtime(p) for p in deps)
    objs, of_variant = [], {name: [] for name in VARIANTS}
    jobs = {}
    with cf.ThreadPoolExecutor(max_workers=min(8, 2 * len(sources))) as ex:
        for src in sources:
            name = os.path.basename(src)
            obj = os.path.join(BUILD, name + ".o")
            objs.append(obj)
            todo = [(obj, [])]
            for variant, (_, defines) in VARIANTS.items():
                vobj = obj
                if name in defines:
                    vobj = os.path.join(BUILD, f"{name}.{variant}.o")
                    todo.append((vobj, defines[name]))
                of_variant[variant].append(vobj)
            for o, extra in todo:
                if os.path.exists(o) and os.path.getmtime(o) >= newest_dep:
                    continue
                jobs[ex.submit(_compile, src, o, extra)] = (name, extra)
        host_src = os.path.join(CSRC, "latent_host.cpp")
        host = None
        if not os.path.exists(HOST_MODULE) or os.path.getmtime(HOST_MODULE) < max(
                os.path.getmtime(host_src), os.path.getmtime(os.path.join(ROOT, "include", "kda.h"))):
            if os.path.exists(HOST_MODULE):  # (not left behind for another kda.h, should this fail)
                os.unlink(HOST_MODULE)
            host = ex.submit(_build_host, host_src)
        for fut in cf.as_completed(jobs):
            report = fut.result()
            if verbose:
                print(f"== {jobs[fut][0]} {' '.join(jobs[fut][1])}\n{report}", file=sys.stderr)
    _link(LIB, objs)
    for variant, (path, _) in VARIANTS.items():
        _link(path, of_variant[variant])
    try:
        if host is not None and (report := host.result()) and verbose:
            print(f"== latent_host.cpp\n{report}", file=sys.stderr)
    except Exception as e:
        warnings.warn(f"the latent binding's extension module was not built, its calls go the "
                      f"slower way through latent.py: {e}")
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
