"""Builds libbakron.so in-tree with nvcc for sm_103a (GB300).

The translation units under csrc/ compile in parallel to objects in
_build/, then link into kronecker_hessian_gptq_gb300/libbakron.so.  A build
is skipped when the library is newer than every source and header.  Beside it
_marshal.so (csrc/marshal.cpp, g++, against torch's own headers) is the Python
module that makes the calls for which ctypes is too slow.  It fits one version
of torch and of Python, which _marshal.tag names; the library needs neither,
and is built without it where there is no torch.
"""

from __future__ import annotations

import glob
import importlib.util
import os
import runpy
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libbakron.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_TAG = os.path.join(PKG, "_marshal.tag")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libbakron.so")


def sources() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(out: str, inputs: list) -> bool:
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(f) <= t for f in inputs)


def _library_up_to_date() -> bool:
    return _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                  + [os.path.join(INCLUDE, "bakron.h"), os.path.abspath(__file__)])


def _torch_folder():
    """Where torch is, which is not imported for it; None: nowhere."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None


def marshal_tag(torch_version) -> str:
    """What _marshal.so fits: one version of torch, whose headers it holds code of, and of Python."""
    return f"torch {torch_version}, Python {sysconfig.get_config_var('SOABI')}"


def _marshal_up_to_date(tag: str) -> bool:
    if not _newer(MARSHAL, [os.path.join(CSRC, "marshal.cpp"), os.path.join(INCLUDE, "bakron.h"), os.path.abspath(__file__)]):
        return False
    return marshal_fits(tag)


def marshal_fits(tag: str) -> bool:
    """Whether there is a _marshal.so, for this tag."""
    if not os.path.exists(MARSHAL) or not os.path.exists(MARSHAL_TAG):
        return False
    with open(MARSHAL_TAG) as f:
        return f.read() == tag


def up_to_date() -> bool:
    torch = _torch_folder()
    return _library_up_to_date() and (torch is None or _marshal_up_to_date(_tag_of(torch)))


def _tag_of(torch: str) -> str:
    return marshal_tag(runpy.run_path(os.path.join(torch, "version.py"))["__version__"])


def _marshal_command(torch: str, out: str) -> list:
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    return [cxx, "-O1", "-std=c++17", "-shared", "-fPIC", os.path.join(CSRC, "marshal.cpp"), "-o", out, "-I", INCLUDE,
            "-I", os.path.join(torch, "include"), "-I", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
            "-I", sysconfig.get_paths()["include"], "-I", os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
            "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-ldl"]


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile and link what is not up to date; returns the library's path."""
    torch = _torch_folder()
    library = force or not _library_up_to_date()
    module = torch is not None and (force or not _marshal_up_to_date(_tag_of(torch)))
    procs = []

    def start(what, cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((what, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))

    objs = []
    if library:
        nvcc = _nvcc()
        os.makedirs(BUILD, exist_ok=True)
        flags = NVCC_FLAGS + ARCH + ["-I", INCLUDE, "-I", CSRC] + list(extra_flags or [])
        for src in sources():
            obj = os.path.join(BUILD, os.path.basename(src) + ".o")
            objs.append(obj)
            start(src, [nvcc, "-c", src, "-o", obj] + flags)
    if module:
        start(MARSHAL, _marshal_command(torch, MARSHAL + ".tmp"))
    failed = []
    for what, p in procs:
        out, _ = p.communicate()
        if out and (verbose or p.returncode):
            sys.stdout.write(out)
        if p.returncode:
            failed.append(what)
    if library and set(failed) <= {MARSHAL}:
        tmp = LIB + ".tmp"
        subprocess.run([nvcc, "-shared", "-o", tmp] + objs + ARCH + ["-Xcompiler", "-fPIC"], check=True)
        os.replace(tmp, LIB)
    if module and MARSHAL not in failed:
        os.replace(MARSHAL + ".tmp", MARSHAL)
        with open(MARSHAL_TAG, "w") as f:
            f.write(_tag_of(torch))
    if failed:
        raise RuntimeError(f"compilation failed for {failed}")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
