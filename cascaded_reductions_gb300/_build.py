"""Builds librf.so (the CUDA kernels and the C ABI) in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` file compiles to an object in parallel; the objects link
into ``cascaded_reductions_gb300/librf.so``.  A rebuild happens only when a
source or header is newer than the library.  ``csrc/calls.cpp``, the quick way
from Python into some of its calls, is compiled against the installed torch
beside it.
"""

import concurrent.futures
import glob
import hashlib
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "librf.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-v,-warn-spills", "-I", INCLUDE, "-I", CSRC] + ARCH


def calls_path():
    """Where the Python calls' extension for the installed torch lies (its file name carries the
    interpreter's tag and a hash of torch's version), and torch's folder; (None, None) without
    torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None, None
    torch = list(spec.submodule_search_locations)[0]
    with open(os.path.join(torch, "version.py"), "rb") as f:
        tag = hashlib.sha256(f.read()).hexdigest()[:12]
    return os.path.join(HERE, f"_rf_calls_{sys.implementation.cache_tag}_{tag}.so"), torch


def build_calls(force=False):
    """Compile csrc/calls.cpp with the host compiler against the installed torch.  The package
    does without it (the same calls, marshalled in Python), so a failure is told and not raised."""
    path, torch = calls_path()
    src = os.path.join(CSRC, "calls.cpp")
    if path is None or (not force and not _stale(path, [src] + _headers())):
        return path
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [INCLUDE, os.path.join(torch, "include"),
           os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = f"{path}.{os.getpid()}.tmp"       # of this process: builds may run side by side
    cmd = [os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-fPIC", "-shared", src, "-o", tmp]
    cmd += [f"-I{i}" for i in inc]
    cmd += ["-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode == 0:
            os.replace(tmp, path)
            return path
        err = f"status {r.returncode} {r.stderr[-2000:]}"
    except OSError as e:
        err = str(e)
    print(f"calls.cpp not built, the Python calls marshal in Python: {err}")
    for p in (tmp, path):                   # what is there is of an older rf.h
        if os.path.exists(p):
            os.remove(p)
    return None


def _nvcc():
    for cand in (os.environ.get("CUDA_HOME", ""), "/usr/local/cuda"):
        p = os.path.join(cand, "bin", "nvcc") if cand else ""
        if p and os.path.exists(p):
            return p
    p = shutil.which("nvcc")
    if p is None:
        raise RuntimeError("nvcc not found: set CUDA_HOME or put nvcc on PATH")
    return p


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _log(obj):
    """Where the compiler's report on an object's kernels is kept."""
    return obj[:-2] + ".ptxas"


def _compile(nvcc, src, obj, extra):
    cmd = [nvcc, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stderr}")
    with open(_log(obj), "w") as f:
        f.write(r.stderr)
    return r.stderr


def registers(log):
    """Registers per thread of each kernel that a compiler's report names, by mangled name."""
    used, name = {}, None
    for line in log.splitlines():
        m = re.search(r"Compiling entry function '(\w+)'", line)
        name = m.group(1) if m else name
        m = re.search(r"Used (\d+) registers", line)
        if m and name:
            used[name], name = int(m.group(1)), None
    return used


def pair_registers():
    """What every attention kernel on CTA pairs has to be compiled to: they divide the registers of
    exactly so many per thread between their warpgroups, and refuse to be launched with others."""
    with open(os.path.join(CSRC, "attn_pair.cuh")) as f:
        return int(re.search(r"constexpr int REGS = (\d+)", f.read()).group(1))


def divided_registers():
    """The same of all kernels that divide their registers, by a part of their names."""
    pair = pair_registers()
    with open(os.path.join(CSRC, "paged_decode.cu")) as f:
        teams = int(re.search(r"constexpr int REGS = (\d+)", f.read()).group(1))
    return {"attn_pair_kernel": pair, "paged_pair_kernel": pair, "paged_decode_kernel": teams}


def _report_pairs(log):
    for name, n in registers(log).items():
        for part, want in divided_registers().items():
            if part in name and n != want:
                print(f"WARNING: {name} has {n} registers per thread instead of {want}: the calls that run on "
                      "it will return RF_ERR_UNSUPPORTED", file=sys.stderr)


def build(force=False, verbose=False, extra_flags=(), lib=None, objdir=None):
    """Compile every CUDA source and link librf.so; returns the library path.

    ``lib`` / ``objdir`` build a variant elsewhere (e.g. the bounds-checked
    debug library, ``extra_flags=["-DRF_CHECK_BOUNDS"]``) without touching
    the default one."""
    lib = lib or LIB
    objdir = objdir or OBJDIR
    srcs = _sources()
    hdrs = _headers()
    if not force and not _stale(lib, srcs + hdrs):
        if lib == LIB:
            build_calls()
        return lib
    nvcc = _nvcc()
    os.makedirs(objdir, exist_ok=True)
    objs = [os.path.join(objdir, os.path.basename(s)[:-3] + ".o") for s in srcs]
    jobs = []
    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 4))) as ex:
        calls = ex.submit(build_calls, force) if lib == LIB else None
        for s, o in zip(srcs, objs):
            if force or _stale(o, [s] + hdrs) or not os.path.exists(_log(o)):
                jobs.append(ex.submit(_compile, nvcc, s, o, list(extra_flags)))
        logs = [j.result() for j in jobs]
        for lg in logs:
            _report_pairs(lg)
        if calls is not None:
            calls.result()
    if verbose:
        for lg in logs:
            if lg:
                print(lg)
    tmp = lib + ".tmp"
    cmd = [nvcc, "-shared", *ARCH, "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of {os.path.basename(lib)} failed:\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


def build_checked(force=False):
    """The bounds-checked debug variant: _build_checked/librf_checked.so."""
    d = os.path.join(HERE, "_build_checked")
    return build(force=force, extra_flags=["-DRF_CHECK_BOUNDS"],
                 lib=os.path.join(d, "librf_checked.so"), objdir=d)


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
