"""Builds libnanospec.so in-tree with nvcc for sm_103a (GB300).

Each CUDA translation unit is compiled in its own nvcc process (in parallel),
then the objects are linked into one shared library next to this file, and the
Python binding of the serving operators (_serving.so, compiled beside them
against torch's headers) is linked to it.  The build is skipped when both are
newer than every source and header.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_NAME = "libnanospec.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
BINDING_PATH = os.path.join(PKG_DIR, "_serving.so")
SOURCES = ["ns_api.cu", "ns_state.cu", "ns_topk.cu", "ns_noalloc.cu", "ns_umma.cu", "ns_slots.cu", "ns_step.cu",
           "ns_dense.cu", "ns_pages.cu", "ns_logprobs.cu", "ns_paged_attn.cu", "ns_paged_umma.cu", "ns_prompt_attn.cu",
           "ns_ops_api.cu"]
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


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES + [BINDING]]
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files += [os.path.join(ROOT, "include", f) for f in ("nanospec.h", "nanospec_ops.h")]
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(BINDING_PATH):
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(BINDING_PATH))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile and link the library; returns its path."""
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = nvcc_path()
    flags = NVCC_FLAGS + list(extra_flags or [])

    def run(cmd, what):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        run([nvcc, *flags, "-c", os.path.join(CSRC, src), "-o", obj], f"nvcc failed on {src}")
        return obj

    def compile_binding():
        import sysconfig

        import torch

        torch_dir = os.path.dirname(torch.__file__)
        include = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                   sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")]
        obj = os.path.join(BUILD_DIR, "ns_binding.o")
        run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *["-I" + p for p in include], "-c",
             os.path.join(CSRC, BINDING), "-o", obj], f"g++ failed on {BINDING}")
        return obj, os.path.join(torch_dir, "lib")

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(compile_binding)
        objs = list(ex.map(compile_one, SOURCES))
        binding_obj, torch_lib = binding.result()
    tmp = LIB_PATH + ".tmp"
    run([nvcc, *ARCH_FLAGS, "-shared", "-o", tmp, *objs], "link failed")
    os.replace(tmp, LIB_PATH)
    tmp = BINDING_PATH + ".tmp"
    run(["g++", "-shared", "-o", tmp, binding_obj, "-L" + PKG_DIR, "-l:" + LIB_NAME, "-Wl,-rpath,$ORIGIN",
         "-L" + torch_lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"], f"linking {BINDING_PATH} failed")
    os.replace(tmp, BINDING_PATH)
    return LIB_PATH


if __name__ == "__main__":
    extra = sys.argv[1:]
    print(build(force=True, verbose=True, extra_flags=extra))
