"""Build libpagedattn.so in-tree for sm_103a (nvcc, no cmake).

Each translation unit compiles in its own nvcc process, in parallel, then one
nvcc call links the shared library. The output lands in
``paged_kv_cache_261_gb300/_build/`` (git-ignored). Where torch is installed, g++ builds
the Python module of csrc/binding.cpp beside it, for that torch and that Python; the package works
without it, so failing to build it is a warning. Run as a script
or call ``build_library()``.
"""
from __future__ import annotations

import hashlib
import os
import shutil
import subprocess
import sys
import warnings
from concurrent.futures import ThreadPoolExecutor
from importlib.machinery import EXTENSION_SUFFIXES

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libpagedattn.so")
HEADER = os.path.join(ROOT, "include", "pagedattn.h")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr"]

SOURCES = ["capi.cu", "kv_write.cu", "kv_write_fp8.cu", "decode_simt.cu", "decode_tc.cu", "decode_fp8.cu",
           "prefill_tc.cu", "kv_int4.cu", "decode_int4.cu", "decode_mass.cu", "evict.cu", "decode_noalloc.cu",
           "selftest.cu", "kv_fp8_block.cu", "decode_fp8_block.cu", "step_layout.cu", "rotary.cu", "allocator.cpp"]


BINDING = "binding.cpp"


def _torch_version():
    """The version of the torch that is there, if it has CUDA; torch is not imported for it."""
    import importlib.util
    import runpy
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    try:
        v = runpy.run_path(os.path.join(spec.submodule_search_locations[0], "version.py"))
    except Exception:
        return None
    return v.get("__version__") if v.get("cuda") else None


def binding_path(torch_version: str) -> str:
    """Of this interpreter: its tag is in the name, as an extension module's."""
    return os.path.join(BUILD, f"_pagedattn_binding_{torch_version}{EXTENSION_SUFFIXES[0]}")


def interface() -> str:
    """What the library and its callers have to agree on: a number made of the header, compiled into both."""
    with open(HEADER, "rb") as f:
        return f"-DPA_INTERFACE=0x{hashlib.sha256(f.read()).hexdigest()[:16]}ull"


def _binding_command(obj: str):
    import sysconfig

    import torch
    root = os.path.join(os.path.dirname(torch.__file__), "include")
    nvcc_include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    include = [root, os.path.join(root, "torch", "csrc", "api", "include"), nvcc_include, sysconfig.get_paths()["include"]]
    return ["g++", "-std=c++17", "-O2", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            interface(), *("-I" + d for d in include), "-c", os.path.join(CSRC, BINDING), "-o", obj]


def _link_binding(obj: str, folder: str, to: str) -> None:
    """Links the binding with the library in `folder`; it will look for that beside itself."""
    import torch
    _run(["g++", "-shared", "-o", to, obj, "-L" + folder, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
          "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
          "-ltorch_python"], "linking the binding")


def _run(cmd, what: str):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [HEADER, os.path.abspath(__file__)]
    return [f for f in files if os.path.isfile(f)]


def _stale(target: str) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in _deps())


def _binding_wanted(torch_version: str | None) -> bool:
    """Whether there is a binding to build: none is there, or an old one, and building these sources has not failed."""
    return torch_version is not None and _stale(binding_path(torch_version)) and \
        _stale(binding_path(torch_version) + ".failed")


def _no_binding(torch_version: str, why: Exception) -> None:
    """The package works without its binding, more slowly: a failure to build it is told, and not tried again
    before a source changes."""
    with open(binding_path(torch_version) + ".failed", "w") as f:
        f.write(f"{why}\n")
    warnings.warn("the compiled module of the serving step's calls was not built; they go through ctypes "
                  f"(build.py --force tries again). {why}")


def build_library(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    torch_version = _torch_version()
    lib = force or _stale(LIB)
    binding = torch_version is not None if lib else _binding_wanted(torch_version)
    if not lib and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)

    def object_of(src: str) -> str:
        return os.path.join(BUILD, src + f".{os.getpid()}.o")

    def compile_one(src: str):
        """None, or why the binding did not compile."""
        try:
            cmd = _binding_command(object_of(src)) if src == BINDING else \
                [_nvcc(), *ARCH, *NVCC_FLAGS, interface(), "-c", os.path.join(CSRC, src), "-o", object_of(src)]
            r = _run(cmd, f"compiling {src}")
        except Exception as e:
            if src == BINDING:
                return e
            raise
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return None

    sources = (SOURCES if lib else []) + ([BINDING] if binding else [])
    with ThreadPoolExecutor(max_workers=jobs or len(sources)) as ex:
        why = list(ex.map(compile_one, sources))[-1]
    # Both are linked before either is put in place, and a new library leaves no binding of an old one beside it,
    # for whatever torch or Python that was.
    new = os.path.join(BUILD, f"new.{os.getpid()}")
    os.makedirs(new, exist_ok=True)
    if lib:
        _run([_nvcc(), *ARCH, "-shared", "-o", os.path.join(new, os.path.basename(LIB)), *map(object_of, SOURCES)], "link")
    if binding and why is None:
        try:
            _link_binding(object_of(BINDING), new if lib else BUILD, os.path.join(new, BINDING + ".so"))
        except Exception as e:
            why = e
    if lib:
        for f in os.listdir(BUILD):
            if f.startswith("_pagedattn_binding_"):
                os.remove(os.path.join(BUILD, f))
        os.replace(os.path.join(new, os.path.basename(LIB)), LIB)
    if binding:
        if why is None:
            os.replace(os.path.join(new, BINDING + ".so"), binding_path(torch_version))
        else:
            _no_binding(torch_version, why)
    shutil.rmtree(new)
    for src in sources:
        if os.path.exists(object_of(src)):
            os.remove(object_of(src))
    return LIB


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose=True))
