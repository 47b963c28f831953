"""Builds libmkv.so (the C-ABI library) in-tree with nvcc for sm_103a, and
_marshal.so, the tensor marshalling of its Python binding, with g++ against the
interpreter's torch.

Each translation unit is compiled in parallel, then the .cu ones are linked
into one shared library next to this file.  The library needs nvcc alone:
without torch it is built all the same, without _marshal.so.  Usage: python -m two_compressed_kv_gb300.build_lib
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmkv.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
SOURCES = ["mkv_api.cu", "k_compress.cu", "k_score.cu", "k_select.cu", "k_attn.cu", "k_checks.cu",
           "k_append.cu", "paged_api.cu", "k_rope.cu", "k_paged_attn_64.cu", "k_paged_attn_128.cu",
           "k_paged_attn_256.cu", "k_paged_join.cu", "k_evict.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
         "--expt-relaxed-constexpr", "-I", os.path.join(HERE, "..", "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _run(cmd):
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError("command failed:\n" + " ".join(cmd) + "\n" + r.stdout)
    return r.stdout


def _marshal_cmd(out: str):
    """Compiles csrc/py_marshal.cpp against this interpreter and its torch."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    inc = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"), cuda,
           os.path.join(HERE, "..", "include")]
    lib = os.path.join(root, "lib")
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
             os.path.join(CSRC, "py_marshal.cpp"), "-o", out]
            + [f for i in inc for f in ("-isystem", i)]
            + ["-L" + lib, "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
               "-ltorch_cuda", "-lc10_cuda"])


def _build_marshal() -> str:
    tmp = os.path.join(BUILD, os.path.basename(MARSHAL))
    _run(_marshal_cmd(tmp))
    return tmp


def build(verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nv = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    jobs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        jobs.append(([nv, "-c", os.path.join(CSRC, src), "-o", obj] + ARCH + FLAGS + extra, obj))
    with cf.ThreadPoolExecutor(max_workers=len(jobs) + 1) as ex:
        marshal = ex.submit(_build_marshal)
        outs = list(ex.map(lambda j: _run(j[0]), jobs))
    if verbose or ptxas_info:
        for (cmd, _), out in zip(jobs, outs):
            print(" ".join(cmd[:3]))
            print(out)
    tmp = LIB + ".tmp"
    _run([nv, "-shared", "-o", tmp] + [o for _, o in jobs] + ARCH + ["-cudart", "static"])
    os.replace(tmp, LIB)
    # The library stands by itself.  A marshalling module that does not go with it is taken away:
    # its argument structs may be another version's.
    try:
        os.replace(marshal.result(), MARSHAL)
    except Exception as e:
        if os.path.exists(MARSHAL):
            os.remove(MARSHAL)
        if not (isinstance(e, ImportError) and e.name == "torch"):
            raise
        print("torch cannot be imported: built without _marshal.so, which mkv_rope and mkv_paged_* "
              "need in Python", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv))
