"""Build libfkv.so in-tree with nvcc for sm_103a (GB300), and the Python binding's
argument marshalling (host C++ against torch's headers; one file per Python and
torch, whose versions its name carries).

Each .cu file compiles to an object in parallel, then one shared library is
linked.  No fast-math: the e4m3 quantisation relies on IEEE division.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libfkv.so")
BIND_SOURCE = os.path.join(CSRC, "bind.cpp")
BUILD_DIR = os.path.join(PKG, "_build")
SOURCES = ["fkv_api.cu", "kv_append.cu", "tag_check.cu", "decode_attn.cu", "decode_attn_noalloc.cu", "page_realloc.cu",
           "kv_calibrate.cu", "selftest.cu", "kv_gather.cu", "qk_norm_rope.cu", "step_tables.cu",
           "kv_append_rope.cu", "tree_attn.cu", "tree_attn_small.cu", "tree_attn_wide.cu",
           "tree_commit.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return hs + [os.path.join(ROOT, "include", "fkv.h")]


def bind_path() -> str:
    """The marshalling module for this Python and torch (torch's C++ interface
    changes with its version)."""
    import sys

    import torch
    return os.path.join(PKG, "_fkv_bind.%s-torch-%s.so" % (sys.implementation.cache_tag, torch.__version__))


def _bind_command(out: str):
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [*include_paths(), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
            *[f for d in inc for f in ("-isystem", d)], BIND_SOURCE, "-o", out,
            "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def build(force: bool = False, verbose: bool = False, extra_flags=(), out_lib: str = LIB,
          build_dir: str = BUILD_DIR) -> str:
    """Compile every source (only what changed) and link ``out_lib``."""
    os.makedirs(build_dir, exist_ok=True)
    exe = nvcc()
    hdrs = _headers()
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(build_dir, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s, *hdrs]):
            jobs.append([exe, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", s, "-o", o])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("compiling failed:\n%s\n%s%s" % (" ".join(cmd), r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)

    # any libfkv.so is called through it, a variant's (out_lib) too
    bind, bind_out = None, bind_path()
    if (force and out_lib == LIB) or _stale(bind_out, [BIND_SOURCE, os.path.join(ROOT, "include", "fkv.h")]):
        bind = bind_out + ".tmp%d" % os.getpid()
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        list(ex.map(run, ([_bind_command(bind)] if bind else []) + jobs))
    if bind:
        os.replace(bind, bind_out)
    if force or jobs or _stale(out_lib, objs):
        tmp = out_lib + ".tmp%d" % os.getpid()
        run([exe, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"])
        os.replace(tmp, out_lib)
    return out_lib


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
