"""Build the CUDA library ``libfa_gb300.so`` in-tree for sm_103a.

Each ``csrc/*.cu`` translation unit is compiled in parallel with
``nvcc -gencode arch=compute_103a,code=sm_103a`` and the objects are linked
into one shared library next to this file. ``csrc/fast_calls.cpp`` (the step
calls' way from Python objects to that library) is compiled beside them with
the host compiler against the installed torch and becomes the extension module
``_fast``; the library needs neither, and where the module cannot be built the
calls go through their checks in Python. A rebuild happens only when a source or
header is newer than what was built from it (or ``force=True``), and of the module
when there is none for this Python and this torch.
"""

from __future__ import annotations

import os
import re
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD_DIR = os.path.join(os.path.dirname(HERE), "_build")
LIB_NAME = "libfa_gb300.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
FAST_SRC = os.path.join(CSRC, "fast_calls.cpp")

ARCH = "-gencode=arch=compute_103a,code=sm_103a"
NVCC_FLAGS = [
    ARCH,
    "-O3",
    "-lineinfo",
    "-std=c++17",
    "-Xcompiler=-fPIC",
    "-Xcompiler=-fvisibility=hidden",
    "--expt-relaxed-constexpr",
    "-Xptxas=-v",
]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return cand


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers() -> list[str]:
    return [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]


def _older(built: str, deps: list[str]) -> bool:
    return not os.path.exists(built) or any(os.path.getmtime(f) > os.path.getmtime(built) for f in deps)


def _lib_stale() -> bool:
    deps = sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + _headers()
    return _older(LIB_PATH, deps)


def fast_path() -> str:
    """The extension module's file, named after the Python and the torch whose layouts it was compiled to: one built
    for others is not found, and a new one is built."""
    import torch

    abi = f"{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}.cxx11-{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    return os.path.join(HERE, f"_fast.{re.sub(r'[^A-Za-z0-9._+-]', '_', abi)}.so")


def _fast_sources() -> list[str]:
    return [FAST_SRC, *_headers()]


def _failed_mark() -> tuple[str, str]:
    """A file that says which extension could not be built, and what it says then."""
    return (os.path.join(BUILD_DIR, "fast.failed"),
            f"{fast_path()} {max(os.path.getmtime(f) for f in _fast_sources())}")


def _fast_stale() -> bool:
    path, text = _failed_mark()
    if os.path.exists(path) and open(path).read() == text:
        return False  # once is enough: the calls go without it
    return _older(fast_path(), _fast_sources())


def needs_build() -> bool:
    return _lib_stale() or _fast_stale()


def _run(cmd: list[str], what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r.stderr


def _cuda_include() -> str:
    home = os.environ.get("CUDA_HOME") or os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    return os.path.join(home, "include")


def _compile_fast() -> str:
    """Object file of the extension module, against the headers of the torch that runs."""
    import torch

    root = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD_DIR, "fast_calls.o")
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], _cuda_include()]
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-isystem{i}" for i in inc), "-c",
          FAST_SRC, "-o", obj], "compiling fast_calls.cpp")
    return obj


def _link_fast(obj: str) -> None:
    """Linked against the library beside it and the torch that is installed here."""
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = fast_path() + ".tmp"
    _run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, f"-L{HERE}", f"-l:{LIB_NAME}", f"-L{lib}",
          "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN",
          f"-Wl,-rpath,{lib}"], "linking _fast")
    os.replace(tmp, fast_path())


def _compile_lib(ex: ThreadPoolExecutor, verbose: bool) -> list[str]:
    nvcc = _nvcc()

    def compile_one(src: str) -> tuple[str, str]:
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    results = list(ex.map(compile_one, sources()))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    return [o for o, _ in results]


def _link_lib(objs: list[str]) -> None:
    tmp = LIB_PATH + ".tmp"
    cmd = [_nvcc(), ARCH, "-shared", f"-Xlinker=-soname={LIB_NAME}", "-o", tmp, *objs, "-lcuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        # libcuda is only needed at run time through the runtime's entry-point
        # lookup; link without it where no driver stub is installed
        cmd = cmd[:-1]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link what is stale; returns the library's path. Raises where the library does not
    compile, warns where the extension does not (the calls then go through their checks in Python)."""
    lib_due, fast_due = force or _lib_stale(), force or _fast_stale()
    if not lib_due and not fast_due:
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    mark, text = _failed_mark()
    with ThreadPoolExecutor(max_workers=min(9, os.cpu_count() or 4)) as ex:
        fast = ex.submit(_compile_fast) if fast_due else None
        if lib_due:
            _link_lib(_compile_lib(ex, verbose))
        if fast:
            try:
                _link_fast(fast.result())
                if os.path.exists(mark):
                    os.remove(mark)
            except Exception as e:  # whatever a host without compiler or headers answers
                with open(mark, "w") as f:
                    f.write(text)
                warnings.warn(f"the step calls' extension module was not built, they take their slower way: {e}",
                              RuntimeWarning, stacklevel=2)
    return LIB_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB_PATH)
