"""Builds the CUDA library libdsa_gb300.so in-tree for sm_103a (GB300), and the native argument
marshalling _marshal.so of the paged caches' and the drafts' calls against the installed torch (g++).  The library
needs nvcc only: without torch the marshalling is left out, which nothing but those Python calls use.

Plain nvcc, no CMake: each translation unit under csrc/ compiles in parallel to an object,
then one shared library is linked.  The CUDA runtime is linked statically, so the library
depends only on the driver.  Usage: ``python -m sparse_attention_indexer_e4m3_gb300.build``.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libdsa_gb300.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
MARSHAL_PATH = os.path.join(HERE, "_marshal.so")
MARSHAL_STAMP = os.path.join(BUILD_DIR, "_marshal.txt")  # what _marshal.so was built against

SOURCES = ["dsa_api.cu", "index_d128.cu", "index_d64.cu", "kres_d128.cu", "kres_d64.cu", "select_kernels.cu", "attn.cu", "attn_bwd.cu", "attn_kv4.cu", "kv4.cu",
           "kv4_api.cu", "paged_attn.cu", "step.cu", "paged_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fvisibility=hidden"]


def nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdsa_gb300.so")
    return cand


def _deps() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "dsa.h"))
    files.append(os.path.abspath(__file__))
    return files


def _newer(path: str, deps: list[str]) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in deps)


def _torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec is not None else None


def lib_up_to_date() -> bool:
    return _newer(LIB_PATH, [f for f in _deps() if os.path.basename(f) != "marshal.cpp"])


def _marshal_stamp(torch_dir: str) -> str:
    """The torch and Python whose C++ interfaces _marshal.so uses."""
    with open(os.path.join(torch_dir, "version.py")) as f:
        version = f.read()
    return f"{sysconfig.get_config_var('SOABI')}\n{torch_dir}\n{version}"


def marshal_up_to_date() -> bool:
    """_marshal.so is newer than its sources and built against this torch and Python (or torch is not there)."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        return True
    if not os.path.exists(MARSHAL_STAMP):
        return False
    with open(MARSHAL_STAMP) as f:
        if f.read() != _marshal_stamp(torch_dir):
            return False
    return _newer(MARSHAL_PATH, [os.path.join(CSRC, "marshal.cpp"), os.path.join(INCLUDE, "dsa.h"), os.path.abspath(__file__)])


def up_to_date() -> bool:
    return lib_up_to_date() and marshal_up_to_date()


def _compile_marshal(cc: str) -> None:
    """g++ of marshal.cpp against the installed torch's headers and libraries; nothing without torch."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        return
    inc, lib = os.path.join(torch_dir, "include"), os.path.join(torch_dir, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include")
    tmp = MARSHAL_PATH + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE,
           "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"), "-I", sysconfig.get_paths()["include"],
           "-I", cuda, os.path.join(CSRC, "marshal.cpp"), "-o", tmp, "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on marshal.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL_PATH)
    with open(MARSHAL_STAMP, "w") as f:
        f.write(_marshal_stamp(torch_dir))


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile (if stale) and return the path of libdsa_gb300.so."""
    make_lib = force or bool(extra_flags) or not lib_up_to_date()
    make_marshal = force or not marshal_up_to_date()
    if not (make_lib or make_marshal):
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *flags, "-I", INCLUDE, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        marshal = ex.submit(_compile_marshal, cc) if make_marshal else None
        objs = list(ex.map(compile_one, SOURCES)) if make_lib else []
        if make_lib:
            tmp = LIB_PATH + f".tmp{os.getpid()}"
            cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
            os.replace(tmp, LIB_PATH)
        if marshal is not None:
            marshal.result()
    return LIB_PATH


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None
    print(build(force=True, verbose=v, extra_flags=extra))
