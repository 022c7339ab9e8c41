"""Build the C-ABI shared library ``libpka.so`` in-tree for sm_103a.

Every translation unit under ``csrc/`` is compiled in parallel with nvcc
(one ``-gencode arch=compute_103a,code=sm_103a``), then linked into
``paged_kv_attention_32_gb300/_lib/libpka.so``.  The native part of the Python binding
(``binding/binding.cpp``, host code against torch's headers) becomes
``_lib/_pka_binding.so`` beside it.  Object files go to ``_build/`` at the repository root.  Run ``python -m
paged_kv_attention_32_gb300.build`` (or ``__graft_entry__.build()``).
"""

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build", "pka")
LIB_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIB_DIR, "libpka.so")
BINDING_SRC = os.path.join(PKG, "binding", "binding.cpp")
BINDING = os.path.join(LIB_DIR, "_pka_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", CSRC, "-I", INCLUDE]
CUDA_FLAGS = ARCH + ["-lineinfo", "--expt-relaxed-constexpr"]


def _nvcc():
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(home, "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def _sources():
    return sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def _compile(src, verbose):
    obj = os.path.join(BUILD, src + ".o")
    cmd = [_nvcc()] + COMMON + (CUDA_FLAGS if src.endswith(".cu") else ["-x", "cu"] + ARCH)
    if verbose and src.endswith(".cu"):
        cmd += ["-Xptxas", "-v"]
    cmd += ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    return src, obj, r.returncode, r.stdout + r.stderr


def _torch_dir():
    import torch
    return os.path.dirname(torch.__file__)


def _compile_binding():
    torch_dir = _torch_dir()
    include = os.path.join(torch_dir, "include")
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    obj = os.path.join(BUILD, "binding.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-c", BINDING_SRC, "-o", obj]
    for d in (sysconfig.get_paths()["include"], INCLUDE):
        cmd += ["-I", d]
    for d in (include, os.path.join(include, "torch", "csrc", "api", "include"),
              os.path.join(home, "include")):
        cmd += ["-isystem", d]
    r = subprocess.run(cmd, capture_output=True, text=True)
    return obj, r.returncode, r.stdout + r.stderr


def _link_binding(obj):
    lib = os.path.join(_torch_dir(), "lib")
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", LIB_DIR, "-l:libpka.so", "-L", lib,
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-ltorch_cuda", "-lc10_cuda",
           "-Wl,-rpath,$ORIGIN:" + lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link of the binding failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, BINDING)


def build(verbose=False):
    """Compile and link ``libpka.so`` and the native binding; return the library's path.
    Raises on failure."""
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    srcs = _sources()
    objs, errors = [], []
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_compile_binding)
        for src, obj, rc, log in ex.map(lambda s: _compile(s, verbose), srcs):
            if verbose and log.strip():
                print(f"--- {src}\n{log}", file=sys.stderr)
            if rc != 0:
                errors.append(f"--- {src} failed:\n{log}")
            objs.append(obj)
        binding_obj, rc, log = binding.result()
        if rc != 0:
            errors.append(f"--- binding.cpp failed:\n{log}")
    if errors:
        raise RuntimeError("nvcc failed:\n" + "\n".join(errors))
    tmp = LIB + ".tmp"
    cmd = [_nvcc()] + ARCH + ["-shared", "-Xlinker", "-soname=libpka.so", "-o", tmp] + objs + ["-lcudart_static", "-ldl", "-lrt", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB)
    _link_binding(binding_obj)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
