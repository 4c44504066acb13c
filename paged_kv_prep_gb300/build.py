"""Build the CUDA library ``libpkv.so`` in-tree with nvcc for sm_103a, and the
binding's C++ part ``_marshal.so`` against it and torch's libraries.

Each translation unit is compiled in its own nvcc process (in parallel), then
linked into one shared library with the CUDA runtime linked statically.  The
ptxas resource report of every kernel is kept in ``_build/ptxas.log``.  The library
needs nvcc alone; where torch is not installed ``_marshal.so``, which only calls on
torch's tensors use, is left out.
"""
from __future__ import annotations

import contextlib
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIBRARY = os.path.join(HERE, "libpkv.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
MARSHAL_ABI = os.path.join(BUILD, "marshal.abi")       # what _marshal.so was built for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libpkv.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(
        os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def torch_path():
    """Where torch is installed, None where it is not."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None


def abi(torch_version) -> str:
    """What ``_marshal.so`` goes by: torch's inlined layouts, Python's and its API."""
    return f"torch {torch_version}, {sysconfig.get_config_var('SOABI')}"


def marshal_abi() -> str:
    """What the ``_marshal.so`` that is there was built for ("" where that is not known)."""
    try:
        with open(MARSHAL_ABI) as f:
            return f.read()
    except OSError:
        return ""


def _torch_version(torch):
    """torch.__version__, without importing it."""
    with open(os.path.join(torch, "version.py")) as f:
        return re.search(r"^__version__\s*=\s*['\"]([^'\"]*)", f.read(), re.M).group(1)


def up_to_date() -> bool:
    torch = torch_path()
    if torch and marshal_abi() != abi(_torch_version(torch)):
        return False
    built = [LIBRARY] + ([MARSHAL] if torch else [])
    if not all(map(os.path.exists, built)):
        return False
    t = min(map(os.path.getmtime, built))
    return all(os.path.getmtime(p) <= t for p in _inputs())


def marshal_commands(nvcc, torch):
    """The compiler's and the linker's command for ``_marshal.so``."""
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    include = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(torch, "include"),
               os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")]
    obj = os.path.join(BUILD, "pkv_marshal.o")
    compile_it = [cxx, "-c", os.path.join(CSRC, "pkv_marshal.cpp"), "-o", obj, "-O2", "-std=c++17", "-fPIC"]
    for path in include:
        compile_it += ["-isystem" if path is not INCLUDE else "-I", path]
    link = [cxx, "-shared", "-o", MARSHAL + ".tmp", obj, "-L", HERE, "-l:" + os.path.basename(LIBRARY), "-L",
            os.path.join(torch, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    return compile_it, link


def _begin_marshal(nvcc):
    """Starts on ``_marshal.so`` beside the library: (its link command, the compiler's command, its process or why there
    is none); None where torch is not installed."""
    torch = torch_path()
    if not torch:
        return None
    compile_it, link = marshal_commands(nvcc, torch)
    try:
        return link, compile_it, subprocess.Popen(compile_it, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    except OSError as e:
        return link, compile_it, e


def _compiled(process):
    """Waits for the compiler: why it failed, or None."""
    if isinstance(process, OSError):
        return str(process)
    out, _ = process.communicate()
    return out.decode(errors="replace") if process.returncode else None


def _link_marshal(link, compile_it, error):
    """Links ``_marshal.so`` against the library; what fails here leaves the library built."""
    cmd = compile_it
    if error is None:
        r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        cmd, error = link, r.stdout.decode(errors="replace") if r.returncode else None
    if error is not None:
        raise RuntimeError(f"libpkv.so is built, _marshal.so is not (it needs g++ and torch's headers):\n{' '.join(cmd)}\n{error}")
    with contextlib.suppress(FileNotFoundError):
        os.remove(MARSHAL_ABI)                         # a build that ends here is none
    os.replace(MARSHAL + ".tmp", MARSHAL)
    with open(MARSHAL_ABI, "w") as f:
        f.write(abi(_torch_version(torch_path())))


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIBRARY
    nvcc = nvcc_path()
    os.makedirs(BUILD, exist_ok=True)
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                     "-I", INCLUDE, "-I", CSRC, "-Xptxas", "-v", "--expt-relaxed-constexpr"]
    marshal = _begin_marshal(nvcc)
    procs = []
    objs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
        objs.append(obj)
        cmd = [nvcc, "-c", src, "-o", obj] + common
        procs.append((src, cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                 stderr=subprocess.STDOUT)))
    log = []
    failed = []
    for src, cmd, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        log.append(f"== {os.path.basename(src)}\n{text}")
        if p.returncode != 0:
            failed.append((src, " ".join(cmd), text))
    if marshal:
        marshal = *marshal[:2], _compiled(marshal[2])
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        f.write("\n".join(log))
    if failed:
        msg = "\n".join(f"{s}:\n{c}\n{t}" for s, c, t in failed)
        raise RuntimeError(f"the compiler failed:\n{msg}")
    tmp = LIBRARY + ".tmp"
    link = [nvcc, "-shared", "-o", tmp] + objs + ARCH + ["-Xcompiler", "-fPIC"]
    r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(tmp, LIBRARY)
    if marshal:
        _link_marshal(*marshal)
    if verbose:
        print("\n".join(log))
    return LIBRARY


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
