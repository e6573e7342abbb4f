"""Build the CUDA library in-tree: csrc/*.cu -> _build/libember.so (sm_103a), and
the torch side of the paged-cache operators: csrc/paged_torch.cpp ->
_build/paged_torch<suffix> (a Python extension against the installed torch).

Each translation unit compiles in parallel with nvcc, then one nvcc -shared
link.  The library needs neither torch nor a host C++ compiler beyond nvcc's, so
build() leaves the extension alone; build_ext() (g++ and torch's headers) makes
it when runtime.PagedKV is first used, build_all() both at once.
"""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libember.so")
TORCH_SRC = os.path.join(CSRC, "paged_torch.cpp")
TORCH_EXT = os.path.join(OUT, "paged_torch" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I" + INCLUDE]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    return sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC)
                        if f.endswith((".cuh", ".h"))] + [os.path.join(INCLUDE, "ember.h")]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _torch_id() -> str:
    """The torch that an extension is compiled against: another one may not load it, or load it and differ."""
    import torch
    return f"{torch.__version__} {torch.version.git_version} {os.path.dirname(torch.__file__)}"


def ext_up_to_date() -> bool:
    deps = (TORCH_SRC, os.path.join(INCLUDE, "ember.h"))
    made_for = TORCH_EXT + ".torch"
    if not os.path.exists(TORCH_EXT) or not os.path.exists(made_for):
        return False
    with open(made_for) as f:
        if f.read() != _torch_id():
            return False
    return all(os.path.getmtime(p) <= os.path.getmtime(TORCH_EXT) for p in deps)


def build_ext(force: bool = False) -> str:
    """Compile the torch extension (marshalling only; every kernel is in libember.so)."""
    if not force and ext_up_to_date():
        return TORCH_EXT
    import torch
    from torch.utils import cpp_extension as cpp
    os.makedirs(OUT, exist_ok=True)
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [*cpp.include_paths(), sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    tmp = TORCH_EXT + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *("-I" + i for i in inc), TORCH_SRC,
           "-o", tmp, "-L" + torch_lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("torch extension failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    with contextlib.suppress(FileNotFoundError):
        os.remove(TORCH_EXT + ".torch")      # never beside a binary that it does not speak of
    os.replace(tmp, TORCH_EXT)
    with open(tmp, "w") as f:
        f.write(_torch_id())
    os.replace(tmp, TORCH_EXT + ".torch")
    return TORCH_EXT


def build_all(force: bool = False) -> None:
    """The library and the torch extension, side by side."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        ext = ex.submit(build_ext, force)
        build(force)
        ext.result()


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OUT, exist_ok=True)
    nvcc = _nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(OUT, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
