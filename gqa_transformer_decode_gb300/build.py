"""Build the CUDA library in-tree: csrc/*.cu -> _build/libember.so (sm_103a), and
the torch sides of the operators: csrc/paged_torch.cpp -> _build/paged_torch<suffix>
and csrc/rows_torch.cpp -> _build/rows_torch<suffix> (Python extensions against the
installed torch).

Each translation unit compiles in parallel with nvcc, then one nvcc -shared
link.  The library needs neither torch nor a host C++ compiler beyond nvcc's, so
build() leaves the extensions alone; build_ext() and build_rows_ext() (g++ and
torch's headers) make one when it is first used, build_all() all at once.
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
ROWS_SRC = os.path.join(CSRC, "rows_torch.cpp")
_SUFFIX = sysconfig.get_config_var("EXT_SUFFIX") or ".so"
TORCH_EXT = os.path.join(OUT, "paged_torch" + _SUFFIX)
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


def _ext_up_to_date(src: str, ext: str) -> bool:
    deps = (src, os.path.join(CSRC, "torch_args.h"), os.path.join(INCLUDE, "ember.h"))
    made_for = ext + ".torch"
    if not os.path.exists(ext) or not os.path.exists(made_for):
        return False
    with open(made_for) as f:
        if f.read() != _torch_id():
            return False
    return all(os.path.getmtime(p) <= os.path.getmtime(ext) for p in deps)


def ext_up_to_date() -> bool:
    return _ext_up_to_date(TORCH_SRC, TORCH_EXT)


def build_ext(force: bool = False) -> str:
    """Compile the torch extension of the paged-cache operators (marshalling only; every kernel is in libember.so)."""
    return _build_ext(TORCH_SRC, TORCH_EXT, force)


def build_rows_ext(force: bool = False) -> str:
    """The same for the operators on rows."""
    return _build_ext(ROWS_SRC, os.path.join(OUT, "rows_torch" + _SUFFIX), force)


def _build_ext(src: str, ext: str, force: bool) -> str:
    if not force and _ext_up_to_date(src, ext):
        return ext
    import torch
    from torch.utils import cpp_extension as cpp
    os.makedirs(OUT, exist_ok=True)
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [*cpp.include_paths(), sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    tmp = ext + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *("-I" + i for i in inc), src,
           "-o", tmp, "-L" + torch_lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("torch extension failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    with contextlib.suppress(FileNotFoundError):
        os.remove(ext + ".torch")      # never beside a binary that it does not speak of
    os.replace(tmp, ext)
    with open(tmp, "w") as f:
        f.write(_torch_id())
    os.replace(tmp, ext + ".torch")
    return ext


def build_all(force: bool = False) -> None:
    """The library and the torch extensions, side by side."""
    with cf.ThreadPoolExecutor(max_workers=2) as ex:
        exts = [ex.submit(build_ext, force), ex.submit(build_rows_ext, force)]
        build(force)
        for e in exts:
            e.result()


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
