"""Build ``libhyb_attn.so`` (the C-ABI library) in-tree with nvcc for sm_100a.

Objects are compiled in parallel under ``_build/`` and linked with the static
CUDA runtime, so the library carries its own runtime and needs no JIT cache.
``_binding.so`` (the calls that take PyTorch tensors) is linked against it; it alone needs
PyTorch and Python's headers, and the library is there whether it can be built or not.
"""

from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libhyb_attn.so")
BINDING = os.path.join(HERE, "_binding.so")
BUILD_DIR = os.path.join(ROOT, "_build")
SOURCES = ["api.cu", "api_delta.cu", "api_paged.cu", "k_delta.cu", "k_fused.cu", "k_multi.cu", "k_paged.cu", "k_paged_append.cu", "k_paged_mma.cu", "k_select.cu", "k_state.cu"]
HEADERS = ["errors.h", "hyb_device.cuh", "hyb_internal.h", "k_common.cuh", "k_delta.h", "k_paged.cuh", "k_paged.h", "k_select.h", "k_tcgen05.cuh"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    return os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def compile_binding(force: bool) -> str:
    """The compiled calls from PyTorch tensors (host code only)."""
    import sysconfig

    from torch.utils import cpp_extension
    src, obj = os.path.join(CSRC, "binding.cpp"), os.path.join(BUILD_DIR, "binding.o")
    if force or _stale(obj, [src, os.path.join(ROOT, "include", "hyb_attn.h")]):
        includes = [f"-I{p}" for p in cpp_extension.include_paths()]
        includes.append(f"-I{sysconfig.get_paths()['include']}")
        r = subprocess.run([nvcc(), "-O2", "-std=c++17", "-Xcompiler", "-fPIC", "-DTORCH_API_INCLUDE_EXTENSION_H",
                            *includes, "-c", src, "-o", obj], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{src}:\n{r.stderr}")
    return obj


def link_binding(obj: str) -> None:
    from torch.utils import cpp_extension
    libs = [p for d in cpp_extension.library_paths() for p in (f"-L{d}", "-Xlinker", f"-rpath={d}")]
    r = subprocess.run([nvcc(), "-shared", "-o", BINDING + ".tmp", obj, f"-L{HERE}", "-l:libhyb_attn.so", "-Xlinker",
                        "-rpath=$ORIGIN", *libs, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python", "-cudart",
                        "none"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(BINDING + ".tmp", BINDING)


def build(force: bool = False, verbose: bool = False) -> str:
    headers = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "hyb_attn.h")]
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs = [os.path.join(BUILD_DIR, os.path.splitext(s)[0] + ".o") for s in SOURCES]

    def compile_one(src, obj):
        if not force and not _stale(obj, [src] + headers):
            return ""
        cmd = [nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        return r.stderr

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        binding = ex.submit(compile_binding, force)
        logs = list(ex.map(compile_one, srcs, objs))
    if verbose:
        for lg in logs:
            if lg:
                sys.stderr.write(lg)
    if force or _stale(LIB, objs):
        cmd = [nvcc(), *ARCH, "-shared", "-o", LIB + ".tmp", *objs, "-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(LIB + ".tmp", LIB)
    try:
        binding = binding.result()
    except Exception as e:
        raise RuntimeError(f"{LIB} is built; {os.path.basename(BINDING)} (PagedKVCache, GatedDeltaState) is not: {e}") from e
    if force or _stale(BINDING, [binding]):
        link_binding(binding)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
