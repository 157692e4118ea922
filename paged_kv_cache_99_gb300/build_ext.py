"""Builds libpa.so in-tree with nvcc for sm_103a (parallel compiles, no cmake), and the Python
calls over it (csrc/binding.c) with the C compiler."""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import platform
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
SOURCES = ["pa_api.cu", "decode.cu", "chunk_tc.cu", "reshape_and_cache.cu", "selftest.cu", "copy_blocks.cu",
           "rope.cu", "norm_rope.cu",
           "scored.cu", "tree_commit.cu", "evict.cu", "pool.cpp"]
HEADERS = ["pa_device.cuh", "pa_internal.h"]
BUILD_DIR = os.path.join(HERE, "_build", platform.machine())
LIB_PATH = os.path.join(BUILD_DIR, "libpa.so")
BINDING = "binding.c"
TENSOR_INFO = "tensor_info.cpp"
try:
    _TORCH = importlib.metadata.version("torch")
except importlib.metadata.PackageNotFoundError:
    _TORCH = "unknown"
# named by the torch it is built against, whose tensors it reads
BINDING_PATH = os.path.join(BUILD_DIR, f"_binding-{_TORCH}" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(path: str, sources) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    deps = [os.path.join(CSRC, f) for f in sources] + [os.path.join(INCLUDE, "pa.h"), __file__]
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile what is out of date: libpa.so, whose path it returns, and the extension module over
    it.  Without the latter (no C compiler or no Python headers) there is a warning, and the calls
    that go through it raise ImportError; the library and all other calls do not need it."""
    if force or _stale(LIB_PATH, SOURCES + HEADERS):
        _build_lib(verbose)
    if force or _stale(BINDING_PATH, [BINDING, TENSOR_INFO, "tensor_info.h"]):
        try:
            _build_binding()
        except (OSError, RuntimeError) as e:
            if os.path.exists(BINDING_PATH):
                os.remove(BINDING_PATH)        # of an older source: not to be called
            warnings.warn(f"{BINDING} was not built: {e}", RuntimeWarning, stacklevel=2)
    return LIB_PATH


def _build_lib(verbose: bool) -> None:
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    common = ARCH_FLAGS + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                           "-Xcompiler", "-fvisibility=hidden"]
    if verbose:
        common += ["-Xptxas", "-v"]

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *common, "-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        if verbose:
            print(res.stdout + res.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB_PATH + f".{os.getpid()}.tmp"
    cmd = [nvcc, *ARCH_FLAGS, "-shared", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB_PATH)


def _run(cmd, what: str) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"building {what} failed:\n{res.stdout}\n{res.stderr}")


def _build_binding() -> None:
    """The extension module of the calls in csrc/binding.c, beside libpa.so and linked to it, with
    csrc/tensor_info.cpp if torch's headers, its libraries and a C++ compiler are there (else tensors
    are asked through their Python methods)."""
    tmp = BINDING_PATH + f".{os.getpid()}.tmp"
    obj, info = (os.path.join(BUILD_DIR, f"{name}.{os.getpid()}.o") for name in ("binding", "tensor_info"))
    cc = shutil.which("gcc") or shutil.which("cc") or "cc"
    flags = ["-O2", "-fPIC", "-I", INCLUDE, "-I", sysconfig.get_paths()["include"]]
    link = [cc, "-shared", obj, "-o", tmp, "-L", BUILD_DIR, "-l:libpa.so", "-Wl,-rpath,$ORIGIN"]
    try:
        _run([cc, *flags, "-c", os.path.join(CSRC, BINDING), "-o", obj], BINDING)
        try:
            spec = importlib.util.find_spec("torch")
            if spec is None or spec.origin is None:
                raise RuntimeError("torch is not installed")
            torch_dir = os.path.dirname(spec.origin)
            _run([shutil.which("g++") or shutil.which("c++") or "c++", *flags, "-std=c++17",
                  "-I", os.path.join(torch_dir, "include"),
                  "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                  "-c", os.path.join(CSRC, TENSOR_INFO), "-o", info], TENSOR_INFO)
            _run([*link, info, "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10",
                  "-lstdc++"], TENSOR_INFO)
        except (OSError, RuntimeError) as e:
            warnings.warn(f"{TENSOR_INFO} was not built, calls take longer: {e}", RuntimeWarning, stacklevel=2)
            _run(link, BINDING)
        os.replace(tmp, BINDING_PATH)
    finally:
        for path in (obj, info, tmp):
            if os.path.exists(path):
                os.remove(path)


if __name__ == "__main__":
    print(build(force=True, verbose=True))
