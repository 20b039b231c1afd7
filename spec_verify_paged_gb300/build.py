"""Builds libsvp.so in place: nvcc for sm_103a, one object per translation
unit compiled in parallel, then one shared-library link.  No cmake."""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libsvp.so")
SOURCES = ["attention.cu", "attention_tc.cu", "attention_fp4.cu", "accept.cu",
           "attention_fp4_tc.cu", "kv_append.cu", "score.cu", "evict.cu", "api.cu", "noalloc.cu",
           "step.cu", "page_select.cu", "attention_sparse.cu", "assign.cu",
           "logprobs.cu"]
HEADERS = [os.path.join(CSRC, h)
           for h in ("ptx.cuh", "svp_internal.h", "attn_common.cuh",
                     "fp4.cuh")] + [
    os.path.join(INCLUDE, "svp.h")]

# the Python calls that marshal in C++ (linked to libsvp.so beside it)
CALLS_SRC = os.path.join(CSRC, "calls.cpp")
CALLS_LIB = os.path.join(PKG, "svp_calls.so")

NVCC = os.environ.get("NVCC", "nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
                "-I", INCLUDE, "-I", CSRC]


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, s) for s in SOURCES] + HEADERS
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [NVCC] + FLAGS + list(extra) + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def _calls_tag() -> str:
    """What the module's object code is bound to beside its source: torch's
    C++ headers and library folder, and Python's."""
    import importlib.metadata
    import importlib.util
    import sysconfig
    try:
        where = importlib.util.find_spec("torch").origin
        torch = f"{importlib.metadata.version('torch')} {where}"
    except (AttributeError, importlib.metadata.PackageNotFoundError):
        torch = "none"
    return f"torch {torch}\npython {sysconfig.get_config_var('SOABI')}\n"


def _calls_tag_file() -> str:
    return os.path.join(BUILD_DIR, "svp_calls.tag")


def _calls_stale() -> bool:
    deps = (CALLS_SRC, os.path.join(INCLUDE, "svp.h"))
    if (not os.path.exists(CALLS_LIB) or not os.path.exists(_calls_tag_file()) or
            any(os.path.getmtime(d) > os.path.getmtime(CALLS_LIB) for d in deps)):
        return True
    with open(_calls_tag_file()) as f:
        return f.read() != _calls_tag()


def _compile_calls() -> str:
    """Object file of the marshalling module, against torch's headers."""
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    obj = os.path.join(BUILD_DIR, "calls.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-c",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DSVP_TORCH="{torch.__version__}"',
           "-I", INCLUDE, "-isystem", inc, "-isystem",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem",
           sysconfig.get_paths()["include"], "-isystem",
           os.path.join(cuda, "include"), CALLS_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for calls.cpp:\n{r.stderr}")
    return obj


def _link_calls(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = CALLS_LIB + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libsvp.so", "-L", lib,
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
           "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, CALLS_LIB)


def build(force: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile every CUDA source for sm_103a and link libsvp.so, and the
    Python calls' module beside it (in place)."""
    kernels, calls = force or _stale(), force or _calls_stale()
    if not kernels and not calls:
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls_obj = ex.submit(_compile_calls) if calls else None
        objs = (list(ex.map(lambda s: _compile(s, extra), SOURCES))
                if kernels else None)
        if objs:
            _link(objs)
        if calls_obj:
            try:
                _link_calls(calls_obj.result())
            except Exception as e:
                raise RuntimeError(
                    "svp_calls.so did not build, so the 4-bit cache, gather, "
                    "score and eviction calls, those on selected pages, page "
                    "assignment and log probabilities will raise (libsvp.so is "
                    f"in place): {e}") from e
            with open(_calls_tag_file(), "w") as f:
                f.write(_calls_tag())
    return LIB


def _link(objs) -> None:
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC] + ARCH + ["-shared", "-Xlinker", "-soname=libsvp.so", "-o",
                           tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)


def build_variant(name: str, defines, force: bool = False) -> str:
    """A separately named copy of the library (libsvp_<name>.so beside
    libsvp.so) compiled with extra preprocessor definitions, e.g. the test
    build whose producers stall so that the bounded waits run out."""
    lib = os.path.join(PKG, f"libsvp_{name}.so")
    deps = [os.path.join(CSRC, s) for s in SOURCES] + HEADERS
    if (not force and os.path.exists(lib) and
            all(os.path.getmtime(d) <= os.path.getmtime(lib) for d in deps)):
        return lib
    out_dir = os.path.join(BUILD_DIR, name)
    os.makedirs(out_dir, exist_ok=True)
    extra = [f"-D{d}" for d in defines]

    def one(src):
        obj = os.path.join(out_dir, os.path.splitext(src)[0] + ".o")
        cmd = [NVCC] + FLAGS + extra + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(one, SOURCES))
    tmp = lib + f".tmp{os.getpid()}"
    r = subprocess.run([NVCC] + ARCH + ["-shared", "-o", tmp] + objs,
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    build(force="--force" in sys.argv, ptxas_verbose="-v" in sys.argv)
    print(LIB)
