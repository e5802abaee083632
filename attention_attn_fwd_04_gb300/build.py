"""Build the CUDA library ``libattn_gb300.so`` in-tree for sm_103a.

Each ``csrc/*.cu`` file is compiled in parallel with nvcc
(``-gencode arch=compute_103a,code=sm_103a``) and the objects are linked into
one shared library next to this file.  ``csrc/generation_binding.cpp`` becomes
the CPython module ``_generation`` beside it (host code against PyTorch's and
Python's headers, linked to the library).  Rebuilds only what changed, the
module also for another PyTorch or Python than it was compiled against.

    python -m attention_attn_fwd_04_gb300.build [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libattn_gb300.so")
BINDING_SRC = os.path.join(CSRC, "generation_binding.cpp")
BINDING = os.path.join(HERE, "_generation" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_OBJ = os.path.join(OBJDIR, "generation_binding.o")
BINDING_STAMP = os.path.join(OBJDIR, "generation_binding.txt")  # what BINDING was made with

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
              "--expt-relaxed-constexpr", "-I", CSRC, "-I", INCLUDE]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build")


def _headers():
    return (glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, obj: str, verbose: bool) -> str:
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
    return r.stderr


def _binding_command(obj: str):
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-DTORCH_API_INCLUDE_EXTENSION_H",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch.compiled_with_cxx11_abi()),
            "-I", INCLUDE, "-isystem", inc,
            "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
            "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda,
            "-c", BINDING_SRC, "-o", obj]


def _binding_made_with() -> str:
    """What the module depends on beside the repository's files: it holds
    inlined accessors of one PyTorch's tensors and one Python's objects."""
    import torch
    return "\n".join([torch.__version__, sysconfig.get_config_var("SOABI"),
                      *_binding_command(BINDING_OBJ)])


def _binding_stale(hdrs) -> bool:
    if _stale(BINDING_OBJ, [BINDING_SRC, *hdrs]) or not os.path.exists(BINDING_STAMP):
        return True
    with open(BINDING_STAMP) as f:
        return f.read() != _binding_made_with()


def _compile_binding(obj: str) -> str:
    r = subprocess.run(_binding_command(obj), capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s\n%s" % (BINDING_SRC, r.stdout, r.stderr))
    return r.stderr


def _link_binding(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp%d" % os.getpid()
    r = subprocess.run(["g++", "-shared", "-o", tmp, obj, "-L", HERE, "-lattn_gb300", "-L", libs,
                        "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
                        "-Wl,-rpath,$ORIGIN"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, BINDING)
    # an untagged module, as earlier builds made it, would pass for any Python's
    untagged = os.path.join(HERE, "_generation.so")
    if os.path.exists(untagged):
        os.remove(untagged)
    with open(BINDING_STAMP, "w") as f:
        f.write(_binding_made_with())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every kernel source and link the shared library; returns its path."""
    os.makedirs(OBJDIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdrs = _headers()
    jobs = []
    for src in srcs:
        obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
        if force or _stale(obj, [src, *hdrs]):
            jobs.append((src, obj))
    bind = force or _binding_stale(hdrs)
    if jobs or bind:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs) + 1, os.cpu_count() or 4)) as ex:
            futs = {ex.submit(_compile, s, o, verbose): s for s, o in jobs}
            if bind:
                futs[ex.submit(_compile_binding, BINDING_OBJ)] = BINDING_SRC
            for f in cf.as_completed(futs):
                log = f.result()
                if verbose and log:
                    sys.stderr.write(log)
    objs = [os.path.join(OBJDIR, os.path.basename(s)[:-3] + ".o") for s in srcs]
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        cmd = [_nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
        os.replace(tmp, LIB)
    if bind or _stale(BINDING, [BINDING_OBJ]):
        _link_binding(BINDING_OBJ)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose))
