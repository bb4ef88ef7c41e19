"""Builds libgbattn.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each .cu under csrc/ compiles in its own nvcc process (in parallel); the objects
link into one shared library with the CUDA runtime linked statically, so the
library only needs the NVIDIA driver at run time.  No torch, no cmake.

_binding, an extension module built beside it with the host compiler against the installed torch, is the
quick way from Python into the library (csrc/binding.cpp).  The package works without it,
at the interpreter's pace, so a machine on which it does not build gets a warning.  It is
built again by itself where it is missing or another torch is installed since.
"""

from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgbattn.so")
SOURCES = ["attn_fwd.cu", "paged_decode.cu", "kv_cache.cu", "norm_rope.cu", "kv4_cache.cu", "kv4_decode.cu",
           "tree_attn.cu", "tree_short.cu", "draft_verify.cu", "kv_keep.cu", "api.cu", "api_rope.cu", "api_tree.cu",
           "decode_noalloc.cu"]
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_STAMP = os.path.join(BUILD, "_binding.torch")  # the torch it was built for, what went wrong
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cuda_home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(cuda_home, "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def _flags(verbose_ptxas: bool):
    f = ARCH + ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
                "-Xcompiler", "-fPIC,-fvisibility=hidden,-O2", "-I", INCLUDE, "-I", CSRC]
    if verbose_ptxas:
        f += ["-Xptxas", "-v"]
    return f


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, n) for n in os.listdir(CSRC)] + [os.path.join(INCLUDE, "gbattn.h"),
                                                                   __file__]
    return max(os.path.getmtime(f) for f in files if os.path.isfile(f))


def torch_version() -> str | None:
    """The installed torch's version, without importing it."""
    if "torch" in sys.modules:
        return sys.modules["torch"].__version__
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        return None
    try:
        with open(os.path.join(os.path.dirname(spec.origin), "version.py")) as f:
            return re.search(r"^__version__ = ['\"](.+?)['\"]", f.read(), re.M)[1]
    except (OSError, TypeError):
        return None


def binding_is_current() -> bool:
    """Whether there is nothing to do about _binding: built for the installed torch, failed to
    be (another try would end the same way), or in a tree that cannot be written to."""
    version = torch_version()
    if version is None or not os.access(os.path.dirname(BINDING), os.W_OK):
        return True
    try:
        with open(BINDING_STAMP) as f:
            built_for, _, wrong = f.read().partition("\n")
    except OSError:
        return False
    return built_for == version and (bool(wrong) or os.path.exists(BINDING))


def renew_binding() -> None:
    """Builds _binding and notes what for; a failure is a warning."""
    wrong = build_binding()
    if wrong:
        sys.stderr.write(f"warning: _binding was not built, calls go the slower way:\n{wrong}\n")
    try:
        os.makedirs(BUILD, exist_ok=True)
        with open(BINDING_STAMP, "w") as f:
            f.write(f"{torch_version()}\n{wrong or ''}")
    except OSError:  # a tree that cannot be written to
        pass


def build_binding() -> str | None:
    """Compiles _binding; returns what went wrong, or None."""
    try:
        import torch
    except ImportError as e:
        return str(e)
    root = os.path.dirname(torch.__file__)
    inc, libs = os.path.join(root, "include"), os.path.join(root, "lib")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    tmp = f"{BINDING}.{os.getpid()}.tmp"
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden", "-I", INCLUDE,
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda,
           f'-DBUILT_FOR_TORCH="{torch.__version__}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", BINDING_SOURCE, "-o",
           tmp, "-L", libs, "-lc10", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{libs}"]
    try:
        res = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        return str(e)
    if res.returncode != 0:
        return res.stderr
    os.replace(tmp, BINDING)
    return None


def build(force: bool = False, verbose_ptxas: bool = False, jobs: int | None = None) -> str:
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps_mtime():
        if not binding_is_current():
            renew_binding()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    if os.path.exists(BINDING):
        os.remove(BINDING)  # never older than the library it calls
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc] + _flags(verbose_ptxas) + ["-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, res

    objs = []
    with concurrent.futures.ThreadPoolExecutor(max_workers=jobs or len(SOURCES) + 1) as ex:
        binding = ex.submit(renew_binding)
        for src, obj, res in ex.map(compile_one, SOURCES):
            if res.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
            if verbose_ptxas:
                sys.stderr.write(res.stderr)
            objs.append(obj)
        binding.result()
    tmp = LIB + ".tmp"
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static", "-ldl", "-lpthread",
                                                         "-lrt"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
