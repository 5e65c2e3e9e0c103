"""Build the in-tree CUDA library ``fusion_b2b_gemm_gb300/_lib/libb2b.so`` and
the modules ``_lib/attn_binding.so`` and ``_lib/ffn_binding.so``
(``binding/attention.cpp``, ``binding/feedforward.cpp``, host code against torch's
headers) that pass tensors to its attention and feed-forward calls.

Every translation unit under ``csrc/`` is compiled for sm_103a only
(``-gencode arch=compute_103a,code=sm_103a``) in parallel, then linked with
the static CUDA runtime.  The driver API is reached at run time through
``cudaGetDriverEntryPointByVersion``, so the library loads on a machine
without a GPU (no ``libcuda`` link dependency).
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libb2b.so")
OBJ_DIR = os.path.join(HERE, "_build")
BINDINGS = {"attn_binding": "attention.cpp", "ffn_binding": "feedforward.cpp"}  # module: source under binding/

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
                     "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    cand = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    p = os.path.join(cand, "bin", "nvcc")
    if os.path.exists(p):
        return p
    found = shutil.which("nvcc")
    if not found:
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libb2b.so")
    return found


def _sources():
    srcs = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))
    headers = sorted(f for f in os.listdir(CSRC) if f.endswith((".cuh", ".h")))
    return srcs, headers


def _digest(srcs, headers) -> str:
    h = hashlib.sha256()
    h.update(" ".join(NVCC_FLAGS).encode())
    for name in srcs + headers:
        with open(os.path.join(CSRC, name), "rb") as f:
            h.update(name.encode())
            h.update(f.read())
    with open(os.path.join(INCLUDE, "b2b.h"), "rb") as f:
        h.update(f.read())
    return h.hexdigest()


def _current(path: str, stamp: str, digest: str) -> bool:
    if not (os.path.exists(path) and os.path.exists(stamp)):
        return False
    with open(stamp) as f:
        return f.read().strip() == digest


def build_binding(force: bool = False) -> list[str] | None:
    """Compile each binding if its source, b2b.h or torch changed; return their paths (None without torch)."""
    torch_spec = importlib.util.find_spec("torch")
    if torch_spec is None:
        return None
    torch_dir = torch_spec.submodule_search_locations[0]
    inc = os.path.join(torch_dir, "include")
    flags = ["-O2", "-std=c++17", "-fPIC", "-shared", "-w", "-I" + INCLUDE, "-I" + inc,
             "-I" + os.path.join(inc, "torch", "csrc", "api", "include"), "-I" + sysconfig.get_paths()["include"]]
    libs = ["-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    os.makedirs(OUT_DIR, exist_ok=True)

    def compile_one(name: str) -> str:
        src, out = os.path.join(HERE, "binding", BINDINGS[name]), os.path.join(OUT_DIR, name + ".so")
        h = hashlib.sha256(" ".join(flags + libs).encode())
        for path in (src, os.path.join(INCLUDE, "b2b.h"), os.path.join(torch_dir, "version.py")):
            with open(path, "rb") as f:
                h.update(f.read())
        stamp = os.path.join(OUT_DIR, name + ".sha256")
        if not force and _current(out, stamp, h.hexdigest()):
            return out
        tmp = out + f".tmp{os.getpid()}"
        r = subprocess.run(["g++"] + flags + [src, "-o", tmp] + libs, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on {src}:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, out)
        with open(stamp, "w") as f:
            f.write(h.hexdigest() + "\n")
        return out

    with cf.ThreadPoolExecutor(len(BINDINGS)) as ex:
        return list(ex.map(compile_one, BINDINGS))


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    """Compile and link libb2b.so and the bindings if any source changed; return the library's path."""
    with cf.ThreadPoolExecutor(1) as ex:
        binding = ex.submit(build_binding, force)
        lib = _build_library(force, verbose, jobs)
        binding.result()
    return lib


def _build_library(force: bool, verbose: bool, jobs: int | None) -> str:
    srcs, headers = _sources()
    digest = _digest(srcs, headers)
    stamp = os.path.join(OUT_DIR, "libb2b.sha256")
    if not force and _current(LIB, stamp, digest):
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    os.makedirs(OBJ_DIR, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(name: str) -> str:
        obj = os.path.join(OBJ_DIR, name.rsplit(".", 1)[0] + ".o")
        cmd = [nvcc] + NVCC_FLAGS + ["-c", os.path.join(CSRC, name), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {name}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    jobs = jobs or max(1, min(len(srcs), os.cpu_count() or 4))
    with cf.ThreadPoolExecutor(jobs) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    with open(stamp, "w") as f:
        f.write(digest + "\n")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
