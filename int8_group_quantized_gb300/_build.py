"""Builds libdgq.so in-tree with nvcc for sm_103a (one -gencode; the translation units
of csrc/ compiled in parallel).  Used by ``__graft_entry__.build()`` and by the binding when the
library is missing or older than its sources."""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import os
import shlex
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libdgq.so")
TENSORS_DIR = PKG  # of the binding's checks on tensors

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
# The quantiser's fp32 steps are bit-exact IEEE operations: no FMA contraction there.
UNITS = {
    "dgq_compress.cu": ["-fmad=false", "-prec-div=true", "-prec-sqrt=true"],
    "dgq_compress_cluster.cu": ["-fmad=false", "-prec-div=true", "-prec-sqrt=true"],
    "dgq_append.cu": ["-fmad=false", "-prec-div=true", "-prec-sqrt=true"],
    "dgq_formats.cu": ["-fmad=false", "-prec-div=true", "-prec-sqrt=true"],
    "dgq_prefill.cu": ["-fmad=false", "-prec-div=true", "-prec-sqrt=true"],
    "dgq_attn.cu": [],
    "dgq_attn_window.cu": [],
    "dgq_block8.cu": ["-fmad=false", "-prec-div=true"],
    "dgq_host.cu": [],
    "dgq_noalloc.cu": [],
    "dgq_pages.cu": [],
    "dgq_prompt.cu": [],
    "dgq_tables.cu": [],
}


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources() -> list[str]:
    return [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC))
            if f.endswith((".cu", ".cuh", ".h"))] + [os.path.join(INCLUDE, "dgq.h")]


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def tensors_path() -> str:
    """The native module of the running torch and Python: it reads tensors where this torch's headers say that their
    fields are, so what was built for another one is another file and never opened.  (ImportError without torch.)"""
    import sysconfig
    import torch
    key = f"{torch.__version__}-{(torch.version.git_version or '')[:12]}-{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    return os.path.join(TENSORS_DIR, f"_tensors-{key}{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_tensors(force: bool = False) -> None:
    """Compiles the binding's native checks on tensors (tensors_path).  The binding has the same checks in Python, and a
    caller of the C ABI needs neither: a machine without torch, its headers or a C++ compiler (CXX, or g++) is
    told and goes without.  A source that did not compile is not tried again before it changes."""
    import sysconfig
    made_of = [os.path.join(CSRC, "dgq_tensors.cpp"), os.path.join(INCLUDE, "dgq.h")]
    try:
        import torch
        path = tensors_path()
        failed = os.path.join(OUT_DIR, os.path.basename(path) + ".failed")
        newest = max(os.path.getmtime(f) for f in made_of)
        if not force and any(os.path.exists(f) and os.path.getmtime(f) >= newest for f in (path, failed)):
            return
        with contextlib.suppress(FileNotFoundError):
            os.remove(path)  # (of an earlier source)
        root = os.path.dirname(torch.__file__)
        inc, lib = os.path.join(root, "include"), os.path.join(root, "lib")
        tmp = path + f".{os.getpid()}.tmp"
        res = subprocess.run(
            [*shlex.split(os.environ.get("CXX") or "g++"), "-std=c++17", "-O2", "-fPIC", "-shared",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
             "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
             "-I", sysconfig.get_paths()["include"], "-I", INCLUDE, made_of[0], "-o", tmp, "-L", lib, "-ltorch_python", "-ltorch",
             "-ltorch_cpu", "-lc10", "-ldl", f"-Wl,-rpath,{lib}"], capture_output=True, text=True)
        if res.returncode == 0:
            os.replace(tmp, path)
            return
        why = res.stderr[-2000:]
        os.makedirs(OUT_DIR, exist_ok=True)
        with open(failed, "w") as f:
            f.write(why)
    except (ImportError, OSError) as e:  # no torch, no compiler
        why = str(e)
    print(f"the native checks on tensors are not built and run in Python:\n{why}", file=sys.stderr)


def build(force: bool = False, verbose: bool = False) -> str:
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        job = ex.submit(build_tensors, force)
        lib = build_lib(force, verbose)
        job.result()
    return lib


def build_lib(force: bool = False, verbose: bool = False) -> str:
    if not force and not stale():
        return LIB
    nvcc = _nvcc()
    os.makedirs(OUT_DIR, exist_ok=True)

    def compile_unit(name: str) -> str:
        obj = os.path.join(OUT_DIR, name.replace(".cu", ".o"))
        cmd = [nvcc, *COMMON, *ARCH, *UNITS[name], "-c", os.path.join(CSRC, name), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {name}:\n{res.stderr}")
        if verbose and res.stderr:
            print(res.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(UNITS)) as ex:
        objs = list(ex.map(compile_unit, UNITS))
    tmp = LIB + f".{os.getpid()}.tmp"
    subprocess.check_call([nvcc, *ARCH, "-shared", "-cudart", "shared", *objs, "-o", tmp])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
