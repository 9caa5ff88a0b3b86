"""Build libpkv.so, libpkv_prefill.so and the binding's _call.so and _tensor.so
in-tree for sm_103a with nvcc (no cmake, no torch extension).

The translation units compile in parallel.  Both shared libraries are linked
with the static CUDA runtime so they load without extra library paths.  The
prefill kernel (thread-block clusters sharing K/V loads by TMA multicast) sits
in libpkv_prefill.so of its own, so that a process that only decodes never
loads it; that library takes its error reporting from libpkv.so, found next to
it through an $ORIGIN run path.  _call.so and _tensor.so are CPython modules that
convert the arguments of the per-step calls and call libpkv.so: plain numbers and
addresses the one, torch tensors the other, which alone is compiled against
torch's headers and is left out where torch is not installed.
"""
from __future__ import annotations

import hashlib
import importlib.util
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libpkv.so")
PREFILL_LIB_PATH = os.path.join(PKG_DIR, "libpkv_prefill.so")
CALL_PATH = os.path.join(PKG_DIR, "_call.so")
TENSOR_PATH = os.path.join(PKG_DIR, "_tensor.so")

CUDA_SOURCES = ["append.cu", "api.cu", "decode_f16.cu", "decode_bf16.cu", "decode_e4m3.cu", "decode_e5m2.cu",
                "noalloc.cu", "decode_int8.cu", "append_int8.cu", "rope.cu",
                "block_index.cu", "decode_listed.cu", "decode_listed_fp8.cu", "decode_rest.cu", "prefix.cu",
                "decode_window.cu", "decode_window_fp8.cu", "draft.cu", "tree.cu", "tree_16.cu", "tree_fp8.cu",
                "tree_one.cu", "tree_chunk.cu"]
PREFILL_SOURCES = ["prefill.cu"]
CXX_SOURCES = ["pool.cpp"]
CALL_SOURCES = ["pycall.cpp"]
TENSOR_SOURCES = ["pytensor.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpkv.so")


def _torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")
    return None if spec is None else spec.submodule_search_locations[0]


def outputs() -> list[str]:
    """What build() makes."""
    return [LIB_PATH, PREFILL_LIB_PATH, CALL_PATH] + ([TENSOR_PATH] if _torch_dir() else [])


def _torch_version() -> str:
    if _torch_dir() is None:
        return "no torch"
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f.read()


def _source_digest() -> str:
    h = hashlib.sha256()
    for d in (CSRC, INCLUDE):
        for name in sorted(os.listdir(d)):
            if name.endswith((".cu", ".cuh", ".cpp", ".h")):
                with open(os.path.join(d, name), "rb") as f:
                    h.update(name.encode())
                    h.update(f.read())
    h.update(" ".join(ARCH + NVCC_FLAGS + [sysconfig.get_paths()["include"], _torch_version()]).encode())
    return h.hexdigest()


def _run(cmd: list[str]) -> None:
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"build step failed ({res.returncode}): {' '.join(cmd)}\n{res.stdout}")


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link outputs() next to this file; skip when up to date."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    stamp = os.path.join(BUILD_DIR, "libpkv.stamp")
    digest = _source_digest()
    if not force and all(os.path.exists(p) for p in [*outputs(), stamp]):
        with open(stamp) as f:
            if f.read().strip() == digest:
                return LIB_PATH
    nvcc = _nvcc()
    jobs = []
    for src in CUDA_SOURCES + PREFILL_SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        jobs.append([nvcc, *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj])
    torch_dir = _torch_dir()
    modules = [(CALL_SOURCES, [], CALL_PATH, [])]
    if torch_dir:
        modules.append((TENSOR_SOURCES, ["-isystem", os.path.join(torch_dir, "include")], TENSOR_PATH,
                        ["-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]))
    for sources, flags in [(CXX_SOURCES, []), *((m[0], m[1]) for m in modules)]:
        for src in sources:
            obj = os.path.join(BUILD_DIR, src.replace(".cpp", ".o"))
            jobs.append([nvcc, *NVCC_FLAGS, "-I" + sysconfig.get_paths()["include"], *flags, "-x", "c++", "-c",
                         os.path.join(CSRC, src), "-o", obj])
    with ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
        for cmd, _ in zip(jobs, ex.map(_run, jobs)):
            if verbose:
                print(" ".join(cmd))
    objs = [os.path.join(BUILD_DIR, s.rsplit(".", 1)[0] + ".o") for s in CUDA_SOURCES + CXX_SOURCES]
    tmp = LIB_PATH + ".tmp"
    _run([nvcc, *ARCH, "-shared", "-cudart", "static", "-Xlinker", "-soname,libpkv.so", "-o", tmp, *objs])
    os.replace(tmp, LIB_PATH)
    pobjs = [os.path.join(BUILD_DIR, s.rsplit(".", 1)[0] + ".o") for s in PREFILL_SOURCES]
    tmp = PREFILL_LIB_PATH + ".tmp"
    _run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *pobjs, "-L" + PKG_DIR, "-lpkv",
          "-Xlinker", "-rpath,$ORIGIN"])
    os.replace(tmp, PREFILL_LIB_PATH)
    for sources, _, path, libs in modules:
        cobjs = [os.path.join(BUILD_DIR, s.rsplit(".", 1)[0] + ".o") for s in sources]
        tmp = path + ".tmp"
        _run([nvcc, "-shared", "-cudart", "none", "-o", tmp, *cobjs, "-L" + PKG_DIR, "-lpkv", *libs,
              "-Xlinker", "-rpath,$ORIGIN"])
        os.replace(tmp, path)
    with open(stamp, "w") as f:
        f.write(digest)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
