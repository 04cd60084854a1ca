"""Build step of the CUDA libraries: nvcc, sm_100a, in-tree libsdm.so (the SDM C
ABI of include/sdm.h) and libsdm_probe.so (the benchmark's random-row probe), and of
_sequence.so (g++, the sequence operators' host side, linked to libsdm.so)."""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
SO = os.path.join(HERE, "libsdm.so")
PROBE_SRC = os.path.join(HERE, "probe", "probe_rows.cu")
PROBE_SO = os.path.join(HERE, "libsdm_probe.so")
BINDING_SRC = os.path.join(HERE, "binding", "sequence.cpp")
BINDING_SO = os.path.join(HERE, "_sequence.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
         "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(SO):
        return True
    t = os.path.getmtime(SO)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [
        os.path.join(HERE, "..", "include", "sdm.h"), os.path.abspath(__file__)]
    return any(os.path.getmtime(f) > t for f in deps)


def build_probe(force: bool = False) -> str:
    """Compile probe/probe_rows.cu into libsdm_probe.so (skipped when up to date)."""
    deps = [PROBE_SRC, os.path.join(HERE, "probe", "probe_rows.h"), os.path.abspath(__file__)]
    if (not force and os.path.exists(PROBE_SO)
            and all(os.path.getmtime(f) <= os.path.getmtime(PROBE_SO) for f in deps)):
        return PROBE_SO
    tmp = PROBE_SO + ".tmp%d" % os.getpid()
    subprocess.check_call([NVCC] + FLAGS + ["-shared", "-o", tmp, PROBE_SRC, "-lcudart"])
    os.replace(tmp, PROBE_SO)
    return PROBE_SO


def build_binding(force: bool = False) -> str:
    """Compile binding/sequence.cpp into _sequence.so (skipped when up to date)."""
    deps = [BINDING_SRC, os.path.join(HERE, "..", "include", "sdm.h"), os.path.abspath(__file__)]
    if (not force and os.path.exists(BINDING_SO)
            and all(os.path.getmtime(f) <= os.path.getmtime(BINDING_SO) for f in deps)):
        return BINDING_SO
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(NVCC)))
    tmp = BINDING_SO + ".tmp%d" % os.getpid()
    subprocess.check_call(
        [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
         "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)]
        + ["-I" + d for d in (os.path.join(HERE, "..", "include"), inc,
                              os.path.join(inc, "torch", "csrc", "api", "include"),
                              sysconfig.get_paths()["include"], os.path.join(cuda, "include"))]
        + [BINDING_SRC, "-o", tmp, "-L" + HERE, "-lsdm", "-L" + lib, "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_python", "-ltorch", "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, BINDING_SO)
    return BINDING_SO


def build(force: bool = False, verbose: bool = False, out: str = None, defines=()) -> str:
    """Compile csrc/*.cu into libsdm.so (skipped when up to date), the probe library
    and the sequence operators' host side.  `out` and `defines` (e.g.
    "SDM_RECUR_THREADS=512") build a variant of libsdm.so elsewhere."""
    if out is None:
        build_probe(force)
    so = out or SO
    if out is None and not defines and not force and not _stale():
        build_binding()
        return SO
    objdir = os.path.join(os.path.dirname(so) if out else HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    procs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src)[:-3] + ".o")
        cmd = [NVCC] + FLAGS + ["-D" + d for d in defines] + ["-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    failed = False
    for src, pr in procs:
        out, _ = pr.communicate()
        if pr.returncode != 0 or verbose:
            sys.stderr.write(out.decode(errors="replace"))
        if pr.returncode != 0:
            failed = True
    if failed:
        raise RuntimeError("nvcc failed")
    tmp = so + ".tmp%d" % os.getpid()
    subprocess.check_call([NVCC, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-o", tmp]
                          + objs + ["-lcudart"])
    os.replace(tmp, so)
    if so == SO:
        build_binding(force)
    return so


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(SO)
