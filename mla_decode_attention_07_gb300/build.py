"""In-tree build of libmla.so for sm_103a (nvcc, no cmake).

Each .cu under csrc/ is compiled to an object in parallel, then linked into
``_build/libmla.so`` next to this file; csrc/binding.c (the marshalling of some
calls from Python, CPython C API) becomes ``_build/_binding<suffix>``, with the
running Python's own suffix for extension modules, so that another Python builds
its own; without Python's headers it is left out, and those calls say so.
``python -m mla_decode_attention_07_gb300.build [--verbose]``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libmla.so")
BINDING = "_binding" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so")
SOURCES = ["mla_api.cu", "mla_decode_sm103.cu", "mla_decode_narrow_sm103.cu", "mla_noalloc.cu",
           "gemm_sm103.cu", "attention_sm103.cu", "rope_append_sm103.cu",
           "mla_decode_fp8_sm103.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags(verbose: bool):
    f = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
                "--expt-relaxed-constexpr"]
    if verbose:
        f += ["-Xptxas", "-v"]
    return f


def _deps_mtime() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "mla.h")]
    return max(os.path.getmtime(p) for p in paths)


def python_includes() -> list[str] | None:
    """Where Python's headers are, or None."""
    dirs = [sysconfig.get_paths()["include"], sysconfig.get_paths()["platinclude"]]
    return dirs if any(os.path.exists(os.path.join(d, "Python.h")) for d in dirs) else None


def build(force: bool = False, verbose: bool = False) -> str:
    binding = os.path.join(OUT_DIR, BINDING)
    headers = python_includes()
    made = [LIB, binding] if headers else [LIB]
    if (not force and all(os.path.exists(p) for p in made)
            and min(os.path.getmtime(p) for p in made) >= _deps_mtime()):
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    cc = nvcc()
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
        objs.append(obj)
        cmd = [cc, *_flags(verbose), "-c", os.path.join(CSRC, src), "-o", obj]
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                            text=True)))
    tmp_binding = binding + f".tmp{os.getpid()}"
    if headers:
        cmd = [os.environ.get("CC", "gcc"), "-O2", "-Wall", "-shared", "-fPIC", "-I", INCLUDE,
               *(x for d in headers for x in ("-I", d)), os.path.join(CSRC, "binding.c"), "-o",
               tmp_binding]
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                            text=True)))
    else:
        sys.stderr.write("Python's headers are missing: built without csrc/binding.c\n")
    failed = []
    for cmd, p in procs:
        out, _ = p.communicate()
        if out and (verbose or p.returncode):
            sys.stderr.write(out)
        if p.returncode:
            failed.append(" ".join(cmd))
    if failed:
        raise RuntimeError("compiling failed:\n" + "\n".join(failed))
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs])
    if headers:
        os.replace(tmp_binding, binding)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="--verbose" in sys.argv))
