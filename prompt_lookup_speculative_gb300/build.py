"""Compile the CUDA library in-tree for GB300 (sm_103a).

The library is eight translation units, ``csrc/lookup_draft.cu`` (the drafting
step), ``csrc/lookup_loop.cu`` (the decode-loop steps around it),
``csrc/lookup_index.cu`` (the incremental n-gram index),
``csrc/lookup_ctxcache.cu`` (context-cache drafting), ``csrc/lookup_kv_append.cu``,
``csrc/lookup_attention.cu`` and ``csrc/lookup_logits.cu`` (the target model's side
of a verify step) and ``csrc/read_floor.cu``
(a measurement aid: a plain streaming read), built with nvcc into
``_build/liblookup_draft.so`` next to this file.  The drafting step's source is
also compiled with LOOKUP_DRAFT_CHECKED=1 into ``_build/liblookup_draft_checked.so``:
the same entry points with device-side index checks (include/lookup_draft.h).  The CUDA runtime is linked
statically, so the library loads on a machine without a GPU (its calls then
fail with a CUDA error) and needs nothing from the Python environment.

``csrc/target_binding.cpp``, the Python entry of the target's operators, is compiled
with the host compiler against the installed PyTorch's and Python's headers (PyTorch's
version and Python's ABI are part of the file's name) and does not link against the
library.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO_DIR = os.path.dirname(PKG_DIR)
INCLUDE_DIR = os.path.join(REPO_DIR, "include")
SOURCES = [os.path.join(PKG_DIR, "csrc", f)
           for f in ("lookup_draft.cu", "lookup_loop.cu", "lookup_index.cu", "lookup_ctxcache.cu",
                     "lookup_kv_append.cu", "lookup_attention.cu", "lookup_logits.cu", "read_floor.cu")]
HEADERS = [os.path.join(INCLUDE_DIR, f)
           for f in ("lookup_draft.h", "lookup_loop.h", "lookup_index.h", "lookup_ctxcache.h",
                     "lookup_target.h")] + \
          [os.path.join(PKG_DIR, "csrc", "common.cuh")]
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "liblookup_draft.so")
# The checked build of the drafting step (LOOKUP_DRAFT_CHECKED=1; read_floor.cu rides along
# so that it exports everything lookup_draft.h declares): device-side
# index checks that set bits in a check word instead of faulting.
CHECKED_SOURCES = [os.path.join(PKG_DIR, "csrc", f) for f in ("lookup_draft.cu", "read_floor.cu")]
CHECKED_LIB_PATH = os.path.join(BUILD_DIR, "liblookup_draft_checked.so")

BINDING_SOURCE = os.path.join(PKG_DIR, "csrc", "target_binding.cpp")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    found = shutil.which("nvcc")
    if found:
        return found
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def compile_command(out: str, extra: list[str] | None = None, checked: bool = False) -> list[str]:
    """nvcc command line of the library (checked=True: the checked build of the
    drafting step)."""
    sources = CHECKED_SOURCES if checked else SOURCES
    defines = ["-DLOOKUP_DRAFT_CHECKED=1"] if checked else []
    return [nvcc_path(), *ARCH_FLAGS, "-lineinfo", "-O3", "-std=c++17", "--threads", "4",
            "-Xcompiler", "-fPIC,-O2", "-shared", "-cudart", "static",
            "-I", INCLUDE_DIR, *defines, "-o", out, *sources, *(extra or [])]


def _torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec is not None else None


def binding_path() -> str | None:
    """Where the target operators' Python entry is built; None without PyTorch, or with one
    that was built without CUDA."""
    torch_dir = _torch_dir()
    if torch_dir is None or not os.path.exists(os.path.join(torch_dir, "lib", "libc10_cuda.so")):
        return None
    return os.path.join(BUILD_DIR, f"_target-{importlib.metadata.version('torch')}{sysconfig.get_config_var('EXT_SUFFIX')}")


def binding_command(out: str) -> list[str]:
    """Host compiler's command line of the Python entry of the target's operators."""
    torch_dir = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC",
            "-I", sysconfig.get_paths()["include"], "-I", os.path.join(torch_dir, "include"),
            "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
            "-I", os.path.join(cuda, "include"), "-I", INCLUDE_DIR, "-o", out, BINDING_SOURCE,
            "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def up_to_date() -> bool:
    for lib in (LIB_PATH, CHECKED_LIB_PATH, binding_path()):
        if lib is None:
            continue
        if not os.path.exists(lib):
            return False
        t = os.path.getmtime(lib)
        if not all(os.path.getmtime(p) <= t for p in SOURCES + HEADERS + [BINDING_SOURCE, __file__]):
            return False
    return True


def build(force: bool = False, verbose: bool = False) -> str:
    """Build both libraries (regular and checked) and the target operators' Python
    entry, side by side, if one is missing or stale; return the regular library's path.
    The libraries need nothing from Python: they are in place even where the entry's
    compilation fails (which raises all the same)."""
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose else None
    jobs = []
    for lib, checked in ((LIB_PATH, False), (CHECKED_LIB_PATH, True)):
        built = lib + f".tmp{os.getpid()}"
        jobs.append((subprocess.Popen(compile_command(built, extra, checked)), built, lib))
    binding, entry = binding_path(), None
    if binding:
        tmp = binding + f".tmp{os.getpid()}"
        entry = subprocess.Popen(binding_command(tmp))
    failed = [p.args for p, _, _ in jobs if p.wait() != 0]
    entry_failed = entry is not None and entry.wait() != 0
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    for _, built, lib in jobs:
        os.replace(built, lib)
    if entry_failed:
        if os.path.exists(binding):                      # an older one does not fit the new library
            os.remove(binding)
        raise subprocess.CalledProcessError(1, entry.args)
    if binding:
        os.replace(tmp, binding)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
