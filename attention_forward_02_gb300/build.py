"""Build the sm_103a CUDA library in-tree (attention_forward_02_gb300/_build/).

Seven translation units (forward, backward, decoding, the 8-bit and the 4-bit paged
cache, page tables, rotary positions), one -gencode
(compute_103a -> sm_103a), static cudart, no link against libcuda (the TMA
encoder is fetched through the runtime's driver entry-point query).  The same
units are compiled a second time with FA_BOUNDS_CHECK into the checked
build (libfa_gb300_checked.so, device-side address checks; a test build).  All
of them compile in parallel, and beside them, with g++, the small CPython module
that shortens the host's way to the entry points around the caches (fa_cache_py.cpp).
"""
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libfa_gb300.so"
LIB = os.path.join(OUT_DIR, LIB_NAME)
# The same sources with the device-side address checks compiled in
# (FA_BOUNDS_CHECK; see include/fa.h): a test build, never the product path.
LIB_CHECKED = os.path.join(OUT_DIR, "libfa_gb300_checked.so")
SOURCES = [os.path.join(CSRC, f) for f in ("fa_fwd.cu", "fa_bwd.cu", "fa_decode.cu", "fa_cache.cu", "fa_cache4.cu",
                                             "fa_pages.cu", "fa_rope.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in ("fa_fwd_kernel.cuh", "fa1_fwd_kernel.cuh",
                                                  "fa_bwd_kernel.cuh", "fa_decode_kernel.cuh", "fa_decode_tc_kernel.cuh",
                                                  "fa_cache_kernel.cuh", "fa_cache_decode_kernel.cuh",
                                                  "fa_cache4_kernel.cuh", "fa_cache4_run.cuh", "fa_cache4_running.cuh",
                                                  "fa_cache4_decode_kernel.cuh", "fa_cache4_short_kernel.cuh",
                                                  "fa_cache4_tc_kernel.cuh",
                                                  "fa_pages_kernel.cuh", "fa_rope_kernel.cuh",
                                                  "fa_cache_host.h", "fa_common.cuh",
                                                  "fa_host.h", "sm100_ptx.cuh")] + [
    os.path.join(INCLUDE, "fa.h")]
BINDING_NAME = "_fa_cache_py"
BINDING_SOURCE = os.path.join(CSRC, "fa_cache_py.cpp")
BINDING = os.path.join(OUT_DIR, BINDING_NAME + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put the CUDA 13 toolkit on PATH)")


def _flags():
    return [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
            "-Xcompiler", "-fvisibility=hidden", "-I" + INCLUDE, "-I" + CSRC]


def compile_commands(out, verbose_ptxas=False, checked=False):
    """One nvcc -c per translation unit, then the link of the shared library."""
    objs, compiles = [], []
    for src in SOURCES:
        obj = out + "." + os.path.splitext(os.path.basename(src))[0] + ".o"
        cmd = [nvcc_path(), *_flags(), *(["-DFA_BOUNDS_CHECK"] if checked else []), "-c", "-o", obj, src]
        if verbose_ptxas:
            cmd.insert(1, "-Xptxas=-v")
        objs.append(obj)
        compiles.append(cmd)
    link = [nvcc_path(), *ARCH, "-shared", "-o", out, *objs]
    return compiles, link, objs


def _stale(lib):
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in DEPS)


def binding_command(out):
    """g++ against the installed torch's headers and libraries."""
    import torch
    root = os.path.dirname(torch.__file__)
    include, lib = os.path.join(root, "include"), os.path.join(root, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
            '-DFA_TORCH_VERSION="%s"' % torch.__version__,
            "-isystem" + include, "-isystem" + os.path.join(include, "torch", "csrc", "api", "include"),
            "-isystem" + cuda, "-I" + sysconfig.get_paths()["include"], "-I" + INCLUDE, BINDING_SOURCE,
            "-o", out, "-L" + lib, "-lc10", "-ltorch_cpu", "-ltorch_python", "-lc10_cuda", "-Wl,-rpath," + lib]


def build_binding(force=False):
    """Compile the CPython module if its source is newer or torch another one; returns its path, or None
    where it cannot be built (the cache's functions then take their longer way through ctypes).  An older
    module does not outlive a failed compilation: it may speak to another ABI."""
    os.makedirs(OUT_DIR, exist_ok=True)
    sources = [BINDING_SOURCE, os.path.join(INCLUDE, "fa.h")]
    note = BINDING + ".torch"  # the torch it was built against
    try:
        import torch
        version = str(torch.__version__)
        if not force and os.path.exists(BINDING) and all(
                os.path.getmtime(p) <= os.path.getmtime(BINDING) for p in sources):
            with open(note) as f:
                if f.read() == version:
                    return BINDING
    except FileNotFoundError:  # a module that does not say
        pass
    except ImportError as e:
        return _no_binding(note, e)
    tmp = BINDING + ".tmp%d" % os.getpid()
    try:
        subprocess.run(binding_command(tmp), check=True)
    except (ImportError, AttributeError, OSError, subprocess.CalledProcessError) as e:
        return _no_binding(note, e)
    os.replace(tmp, BINDING)
    with open(tmp, "w") as f:
        f.write(version)
    os.replace(tmp, note)
    return BINDING


def _no_binding(note, why):
    print("the cache's CPython module was not built: %s" % why, file=sys.stderr)
    for path in (note, BINDING):
        if os.path.exists(path):
            os.remove(path)
    return None


def build_library(force=False, verbose_ptxas=False, checked=True):
    """Compile the library (and, with checked=True, its checked build) if a
    source is newer than it; return the product library's path.  All
    translation units compile in parallel."""
    os.makedirs(OUT_DIR, exist_ok=True)
    jobs = [(LIB, False)] + ([(LIB_CHECKED, True)] if checked else [])
    jobs = [(lib, chk) for lib, chk in jobs if force or _stale(lib)]
    if not jobs:
        build_binding(force)
        return LIB
    plans = []
    for lib, chk in jobs:
        tmp = lib + ".tmp%d" % os.getpid()
        plans.append((lib, tmp) + compile_commands(tmp, verbose_ptxas and not chk, chk))
    compiles = [c for _, _, cs, _, _ in plans for c in cs]
    with ThreadPoolExecutor(len(compiles) + 1) as ex:
        binding = ex.submit(build_binding, force)
        for f in [ex.submit(subprocess.run, c, check=True) for c in compiles]:
            f.result()
        binding.result()
    for lib, tmp, _, link, objs in plans:
        subprocess.run(link, check=True)
        for o in objs:
            os.remove(o)
        os.replace(tmp, lib)
    return LIB


if __name__ == "__main__":
    print(build_library(force=True, verbose_ptxas=True))
