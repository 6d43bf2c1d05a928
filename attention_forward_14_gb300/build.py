"""Build libattn_fwd.so (sm_103a) in-tree with nvcc, its checked variant, and
the Python entry of the operators around the attention (``_marshal_ext.so``,
C++ against torch's headers).

Each translation unit under csrc/ is compiled in parallel, then linked into
``attention_forward_14_gb300/libattn_fwd.so``, which does not wait for the
Python entry: without a C++ compiler, torch's headers or Python's the library
is built all the same, and the operators that need the entry say so when they
are called.  The checked variant,
``libattn_fwd_checked.so``, compiles every translation unit again with
ATTN_CHECKED=1 (every computed copy coordinate, output offset, decoded unit
and on-chip address of the forward and backward kernels is compared with
its bounds; a violation is recorded in the status word and the CTA winds
down).  Usage:
``python -m attention_forward_14_gb300.build [--force] [-v]``.
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libattn_fwd.so")
LIB_CHECKED = os.path.join(HERE, "libattn_fwd_checked.so")
MARSHAL = os.path.join(HERE, "_marshal_ext.so")
MARSHAL_STAMP = "marshal.stamp"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["attn_fwd_api.cu", "inst_d64.cu", "inst_d128_noncausal.cu", "inst_d128_causal.cu", "inst_fp8.cu",
           "attn_bwd_inst.cu", "attn_bwd_inst_varlen.cu", "qk_norm_rope.cu", "kv_append.cu", "attn_kv8.cu",
           "attn_kv8_wide.cu"]
# the translation units compiled again, checked (all of them: forward and backward)
CHECKED_SOURCES = SOURCES


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(ROOT, "include", "attn_fwd.h"))
    files.append(os.path.abspath(__file__))
    return files


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _cxx() -> str:
    return os.environ.get("CXX", "g++")


def _torch_dir() -> str | None:
    from importlib.util import find_spec
    spec = find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _marshal_built_for() -> str:
    """What the Python entry is compiled for, besides its sources: an entry
    built for another torch or Python must not be loaded."""
    from importlib.metadata import PackageNotFoundError, version
    try:
        torch_version = version("torch")
    except PackageNotFoundError:
        torch_version = "none"
    return f"torch {torch_version}, python {sysconfig.get_config_var('SOABI')} in {sys.prefix}, {_cxx()}"


def _marshal_stale() -> bool:
    deps = [os.path.join(CSRC, "marshal.cpp"), os.path.join(ROOT, "include", "attn_fwd.h"), os.path.abspath(__file__)]
    if _stale(MARSHAL, deps):
        return True
    try:
        with open(os.path.join(BUILD, MARSHAL_STAMP)) as f:
            return f.read() != _marshal_built_for()
    except OSError:
        return True


def _marshal_lacks() -> str | None:
    """What the Python entry cannot be compiled without and is not here."""
    if shutil.which(_cxx()) is None:
        return f"no C++ compiler ({_cxx()})"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "no Python headers"
    torch_dir = _torch_dir()
    if torch_dir is None or not os.path.exists(os.path.join(torch_dir, "include", "torch", "csrc", "Exceptions.h")):
        return "no torch headers"
    return None


def _compile_marshal() -> str:
    """The object file of csrc/marshal.cpp (host code)."""
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    obj = os.path.join(BUILD, "marshal.o")
    cmd = [_cxx(), "-std=c++17", "-O2", "-fPIC", "-c", os.path.join(CSRC, "marshal.cpp"), "-o", obj,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for d in (inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"], cuda,
              os.path.join(ROOT, "include")):
        cmd += ["-I", d]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"marshal.cpp failed to compile:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_marshal(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = [_cxx(), "-shared", "-o", tmp, obj, "-L", lib, "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"_marshal_ext.so failed to link:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)
    with open(os.path.join(BUILD, MARSHAL_STAMP), "w") as f:
        f.write(_marshal_built_for())


def build(force: bool = False, verbose: bool = False, checked: bool = True) -> str:
    """Build the library (and, with ``checked``, its checked variant) when a
    source is newer than it; returns the library's path."""
    deps = _deps()
    want = [(LIB, False)] + ([(LIB_CHECKED, True)] if checked else [])
    todo = [(lib, chk) for lib, chk in want if force or _stale(lib, deps)]
    marshal = force or _marshal_stale()
    if marshal:
        lacks = _marshal_lacks()
        if lacks:
            marshal = False
            if os.path.exists(MARSHAL):
                os.remove(MARSHAL)  # of other sources, or for another torch
            sys.stderr.write(f"{lacks}: {os.path.basename(MARSHAL)} is not built, and the operators that it enters raise\n")
    if not todo and not marshal:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    if verbose:
        flags += ["-Xptxas", "-v"]

    def obj_path(src, chk):
        return os.path.join(BUILD, os.path.splitext(src)[0] + ("_checked.o" if chk else ".o"))

    def compile_one(job):
        src, chk = job
        obj = obj_path(src, chk)
        cmd = [cc, *flags, *(["-DATTN_CHECKED=1"] if chk else []), "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}{' (checked)' if chk else ''}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    jobs = [(src, False) for src in SOURCES] if todo else []
    jobs += [(src, True) for src in CHECKED_SOURCES if any(chk for _, chk in todo)]
    with ThreadPoolExecutor(max_workers=len(jobs) + 1) as ex:
        host = ex.submit(_compile_marshal) if marshal else None
        list(ex.map(compile_one, jobs))
    for lib, chk in todo:
        objs = [obj_path(src, chk and src in CHECKED_SOURCES) for src in SOURCES]
        tmp = lib + f".tmp{os.getpid()}"
        r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib)
    if host:  # the library is there whatever becomes of it
        _link_marshal(host.result())
    return LIB


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    main()
