"""Build the attention library (libfa.so) in-tree with nvcc for sm_103a.

Each .cu under csrc/ is compiled in parallel to an object under _build/, then
linked into lib/libfa.so.  Beside them the C++ compiler builds lib/fa_torch.so,
which passes torch tensors to the paged-cache entry points.  The C ABI does not
need it: it is skipped where there is no torch for CUDA, and where it cannot be
built that is a warning (and an error of the calls that need it).  Nothing is
installed anywhere else.  What is newer than its sources and headers is not
built again; the binding also says in a file beside it which torch and Python it
was built for.
"""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.util
import json
import os
import runpy
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libfa.so")
BINDING_SOURCE = os.path.join(CSRC, "torch_binding.cpp")
BINDING_PATH = os.path.join(LIB_DIR, "fa_torch.so")
BINDING_STAMP = os.path.join(LIB_DIR, "fa_torch.json")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    exe = shutil.which("nvcc")
    if exe:
        return exe
    for cand in ("/usr/local/cuda/bin/nvcc",):
        if os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) \
        + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _newer(built: str, inputs: list[str]) -> bool:
    return os.path.exists(built) and all(os.path.getmtime(f) <= os.path.getmtime(built) for f in inputs)


def _torch_place() -> str | None:
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec is not None and spec.submodule_search_locations else None


def binding_target() -> list[str] | None:
    """What the binding has to be built for: torch's version, its CUDA and this
    Python's ABI.  None without a torch for CUDA.  (torch is not imported: that
    takes seconds.)"""
    at = _torch_place()
    if at is None:
        return None
    try:
        v = runpy.run_path(os.path.join(at, "version.py"))
    except OSError:
        return None
    if not v.get("cuda"):
        return None
    return [str(v["__version__"]), v["cuda"], str(sysconfig.get_config_var("SOABI"))]


def binding_built_for() -> list[str] | None:
    """What the binding that is there was built for (None: it does not say)."""
    try:
        with open(BINDING_STAMP) as f:
            return json.load(f)
    except (OSError, ValueError):
        return None


def library_up_to_date() -> bool:
    return _newer(LIB_PATH, _inputs())


def binding_up_to_date() -> bool:
    """Whether the binding is there and fits this torch and Python (true where
    there is none to build)."""
    target = binding_target()
    if target is None:
        return True
    inputs = [BINDING_SOURCE, os.path.join(INCLUDE, "fa.h"), os.path.abspath(__file__)]
    return _newer(BINDING_PATH, inputs) and binding_built_for() == target


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def _build_binding(target: list[str]) -> None:
    import torch

    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(at, "include"),
           "-I" + os.path.join(at, "include", "torch", "csrc", "api", "include"),
           "-I" + os.path.join(cuda, "include"), "-I" + INCLUDE, BINDING_SOURCE, "-o", tmp,
           "-L" + os.path.join(at, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)
    with open(BINDING_STAMP, "w") as f:
        json.dump(target, f)


def _build_library(ex: concurrent.futures.Executor, verbose: bool, flags: list[str]) -> None:
    exe = nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [exe, *ARCH, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    objs = list(ex.map(compile_one, sources()))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    r = subprocess.run([exe, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile and link libfa.so, and the binding where there is a torch for it;
    returns libfa.so's path."""
    force = force or bool(extra_flags)
    library = force or not library_up_to_date()
    target = binding_target() if force or not binding_up_to_date() else None
    if not library and target is None:
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(sources()) + 1) as ex:
        binding = ex.submit(_build_binding, target) if target else None
        if library:
            _build_library(ex, verbose, NVCC_FLAGS + list(extra_flags or []))
        if binding is not None:
            try:
                binding.result()
            except Exception as e:                  # noqa: BLE001 (a torch that does not import, g++, headers)
                warnings.warn(f"the torch binding of the paged-cache calls was not built: {e}", RuntimeWarning, stacklevel=2)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
