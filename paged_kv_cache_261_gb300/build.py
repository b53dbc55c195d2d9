"""Build libpagedattn.so in-tree for sm_103a (nvcc, no cmake).

Each translation unit compiles in its own nvcc process, in parallel, then one
nvcc call links the shared library. The output lands in
``paged_kv_cache_261_gb300/_build/`` (git-ignored). Where torch is installed, g++ builds
the Python module of csrc/binding.cpp beside it, for that version of torch. Run as a script
or call ``build_library()``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

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
    try:
        from importlib.metadata import version
        version("torch")
    except Exception:
        return None
    import torch
    return torch.__version__ if torch.version.cuda else None


def binding_path(torch_version: str) -> str:
    return os.path.join(BUILD, f"_pagedattn_binding_{torch_version}.so")


def _binding_command(obj: str):
    import sysconfig

    import torch
    root = os.path.join(os.path.dirname(torch.__file__), "include")
    nvcc_include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    include = [root, os.path.join(root, "torch", "csrc", "api", "include"), nvcc_include, sysconfig.get_paths()["include"]]
    return ["g++", "-std=c++17", "-O2", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *("-I" + d for d in include), "-c", os.path.join(CSRC, BINDING), "-o", obj]


def _link_binding(obj: str, torch_version: str) -> None:
    import torch
    tmp = binding_path(torch_version) + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + BUILD, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
          "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
          "-ltorch_python"], "linking the binding")
    os.replace(tmp, binding_path(torch_version))


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


def build_library(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    torch_version = _torch_version()
    if not force and not _stale(LIB) and (torch_version is None or not _stale(binding_path(torch_version))):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src + f".{os.getpid()}.o")
        cmd = _binding_command(obj) if src == BINDING else \
            [nvcc, *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        r = _run(cmd, f"compiling {src}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    sources = SOURCES + ([BINDING] if torch_version else [])
    with ThreadPoolExecutor(max_workers=jobs or len(sources)) as ex:
        objs = list(ex.map(compile_one, sources))
    tmp = LIB + f".tmp{os.getpid()}"
    _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs[:len(SOURCES)]], "link")
    os.replace(tmp, LIB)
    if torch_version:
        _link_binding(objs[-1], torch_version)
    for o in objs:
        os.remove(o)
    return LIB


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose=True))
