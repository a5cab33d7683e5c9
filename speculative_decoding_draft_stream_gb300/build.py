"""Builds libnanospec.so in-tree with nvcc for sm_103a (GB300).

Each CUDA translation unit is compiled in its own nvcc process (in parallel),
then the objects are linked into one shared library next to this file.  It is a
C library and needs nvcc alone.  The Python binding of the serving operators
(_serving.so) is compiled beside it where g++, Python's headers and torch are
there; otherwise the library is built without it, and serving.py says so when
it is used.  Each of the two is skipped while it is newer than its sources and
headers, the binding also only while torch and Python are those that it was
built against.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_NAME = "libnanospec.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
BINDING_PATH = os.path.join(PKG_DIR, "_serving.so")
SOURCES = ["ns_api.cu", "ns_state.cu", "ns_topk.cu", "ns_noalloc.cu", "ns_umma.cu", "ns_slots.cu", "ns_step.cu",
           "ns_dense.cu", "ns_pages.cu", "ns_rotate.cu", "ns_logprobs.cu", "ns_paged_attn.cu", "ns_paged_attn8.cu",
           "ns_paged_umma.cu", "ns_paged_umma8.cu", "ns_shared_attn.cu", "ns_shared_attn8.cu",
           "ns_prompt_attn.cu", "ns_ops_api.cu"]
BINDING = "ns_binding.cpp"
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH_FLAGS + [
    "-O3",
    "-lineinfo",
    "-std=c++17",
    "-Xcompiler",
    "-fPIC",
    "-Xcompiler",
    "-fvisibility=hidden",
]


def nvcc_path() -> str:
    cand = shutil.which("nvcc")
    if cand:
        return cand
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    return os.path.join(home, "bin", "nvcc")


def _headers():
    return [os.path.join(ROOT, "include", f) for f in ("nanospec.h", "nanospec_ops.h")] + [os.path.abspath(__file__)]


def _library_inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES]
    return files + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + _headers()


def _newer(path, inputs) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in inputs)


def library_up_to_date() -> bool:
    return _newer(LIB_PATH, _library_inputs())


def binding_tools():
    """What the binding is built with: (torch's folder, Python's headers, a line that names both versions), or the
    reason why it cannot be built."""
    if shutil.which("g++") is None:
        return "no g++"
    include = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")):
        return "no Python.h"
    try:
        import torch
    except ImportError:
        return "no torch"
    folder = os.path.dirname(torch.__file__)
    if not os.path.exists(os.path.join(folder, "include", "ATen", "core", "Tensor.h")):
        return "no headers of torch"
    return folder, include, f"torch {torch.__version__} in {folder}, Python {sys.version}\n"


def _stamp() -> str:
    return os.path.join(BUILD_DIR, "ns_binding.built_against")


def binding_up_to_date() -> bool:
    tools = binding_tools()
    if isinstance(tools, str) or not _newer(BINDING_PATH, [os.path.join(CSRC, BINDING)] + _headers()):
        return False
    try:
        with open(_stamp()) as f:
            return f.read() == tools[2]
    except FileNotFoundError:
        return False


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def _run(cmd, what, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, flush=True)


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile and link the library, and the binding where its tools are there; returns the library's path."""
    library, tools = force or not library_up_to_date(), binding_tools()
    binding = not isinstance(tools, str) and (force or not binding_up_to_date())
    if isinstance(tools, str):
        if os.path.exists(BINDING_PATH):  # of other tools, and perhaps of an older library
            os.remove(BINDING_PATH)
        print(f"{os.path.basename(BINDING_PATH)} is not built: {tools}", file=sys.stderr)
    if not library and not binding:
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = nvcc_path()
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        _run([nvcc, *flags, "-c", os.path.join(CSRC, src), "-o", obj], f"nvcc failed on {src}", verbose)
        return obj

    def compile_binding():
        folder, python, _ = tools
        include = [os.path.join(folder, "include"), os.path.join(folder, "include", "torch", "csrc", "api", "include"),
                   python, os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")]
        obj = os.path.join(BUILD_DIR, "ns_binding.o")
        _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *["-I" + p for p in include], "-c",
              os.path.join(CSRC, BINDING), "-o", obj], f"g++ failed on {BINDING}", verbose)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding_obj = ex.submit(compile_binding) if binding else None
        if library:
            objs = list(ex.map(compile_one, SOURCES))
            tmp = LIB_PATH + ".tmp"
            _run([nvcc, *ARCH_FLAGS, "-shared", "-o", tmp, *objs], "link failed", verbose)
            os.replace(tmp, LIB_PATH)
        if binding:
            obj = binding_obj.result()
            tmp = BINDING_PATH + ".tmp"
            _run(["g++", "-shared", "-o", tmp, obj, "-L" + PKG_DIR, "-l:" + LIB_NAME, "-Wl,-rpath,$ORIGIN",
                  "-L" + os.path.join(tools[0], "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"],
                 f"linking {BINDING_PATH} failed", verbose)
            os.replace(tmp, BINDING_PATH)
            with open(_stamp(), "w") as f:
                f.write(tools[2])
    return LIB_PATH


if __name__ == "__main__":
    extra = sys.argv[1:]
    print(build(force=True, verbose=True, extra_flags=extra))
