"""Build libbea.so in-tree with nvcc for sm_103a.

Each CUDA translation unit under ``csrc/`` is compiled in parallel to an
object under ``_build/`` and the objects are linked into ``libbea.so`` next
to this file (CUDA runtime linked statically; the driver API is reached at
run time through the runtime's entry-point query, so loading the library
needs no GPU). Rebuilds only when a source or header is newer than the
library.

``csrc/binding.cpp``, the Python binding of the short calls, is compiled by the
host compiler against torch's headers (in parallel with the CUDA units) and
linked into ``_bind.so``, which finds libbea.so next to itself. The library does
not need it: where it cannot be built, that is said on stderr, libbea.so is there
all the same, and only the calls that go through the binding raise. Beside it
stands what it was built for (torch, Python, flags): one built for another is
neither loaded nor taken for up to date.
"""

from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libbea.so")
BIND_SRC = os.path.join(CSRC, "binding.cpp")
BIND = os.path.join(HERE, "_bind.so")
BINDING_FLAGS = ["-O2", "-std=c++17", "-fPIC"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
              "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(
        os.path.join(ROOT, "include", "*.h"))


def _newer(target: str, files) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(f) <= os.path.getmtime(target) for f in files)


def library_up_to_date() -> bool:
    return _newer(LIB, _sources() + _headers() + [__file__])


def binding_stamp() -> str:
    """What a binding built now is built for: it uses torch's and Python's C++ objects as they lie in memory."""
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}, {' '.join(_host_compiler() + BINDING_FLAGS)}"


def _stamp_path() -> str:
    return BIND + ".stamp"


def built_binding_stamp() -> str | None:
    """What the binding that is there was built for."""
    if not os.path.exists(BIND) or not os.path.exists(_stamp_path()):
        return None
    with open(_stamp_path()) as f:
        return f.read()


def binding_up_to_date() -> bool:
    try:
        return _newer(BIND, [BIND_SRC] + _headers() + [__file__]) and built_binding_stamp() == binding_stamp()
    except ImportError:
        return False


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def _compile(src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _host_compiler() -> list[str]:
    return ["g++"]


def _cuda_home() -> str:
    return os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(nvcc()) or nvcc())))


def _torch_paths() -> tuple[list[str], str]:
    import torch
    root = os.path.dirname(torch.__file__)
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(_cuda_home(), "include")]
    return ["-I" + i for i in include], os.path.join(root, "lib")


def _compile_binding() -> str:
    obj = os.path.join(BUILD, "binding.o")
    include, _ = _torch_paths()
    cmd = [*_host_compiler(), *BINDING_FLAGS, *include, "-c", BIND_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BIND_SRC}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link(cmd: list[str], target: str) -> None:
    """Run a link command that writes `target`.tmp and put the result in place."""
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(target + ".tmp", target)


def _link_binding(obj: str) -> None:
    _link([*_host_compiler(), "-shared", "-o", BIND + ".tmp", obj, "-L" + os.path.dirname(LIB), "-l:" + os.path.basename(LIB),
           "-Wl,-rpath,$ORIGIN", "-L" + _torch_paths()[1], "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
           "-ltorch_python", "-L" + os.path.join(_cuda_home(), "lib64"), "-lcudart"], BIND)
    with open(_stamp_path(), "w") as f:
        f.write(binding_stamp())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libbea.so, and the binding where that can be done; returns the library's path."""
    library, binding = force or not library_up_to_date(), force or not binding_up_to_date()
    if not library and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(_sources()) + 1) as ex:
        bind_obj = ex.submit(_compile_binding) if binding else None
        results = list(ex.map(_compile, _sources())) if library else []
    if library:
        log = "".join(err for _obj, err in results)
        with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
            f.write(log)
        if verbose:
            sys.stderr.write(log)
        _link([nvcc(), *ARCH, "-shared", "-o", LIB + ".tmp", *[o for o, _ in results]], LIB)
    if binding:
        try:
            _link_binding(bind_obj.result())
        except Exception as e:  # no torch, no host compiler, an error of either: the library stands without it
            sys.stderr.write(f"the Python binding of the rotary and paged calls was not built: {e}\n")
            if os.path.exists(BIND):
                os.remove(BIND)  # of other sources
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
