"""Builds libsdpa.so in-tree with nvcc for sm_103a, and the paged helpers'
CPython extension _bind with the host compiler.

Each CUDA translation unit is compiled in parallel, then linked into one
shared library with the CUDA runtime linked statically.  The extension is
built against the installed torch.  The library does not depend on it: without
a torch for CUDA the library alone is built, and an extension that does not
compile is reported, and left out.  Its name holds the interpreter's tag, and
it is built again when the torch that it was built against changes.
Usage:
    python -m transformer_scaled_dot_02_gb300.build [--force]
"""
from __future__ import annotations

import concurrent.futures as cf
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
BUILD_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libsdpa.so")
BIND = os.path.join(HERE, "_bind" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
BIND_SOURCE = os.path.join(CSRC, "bind.cpp")
SOURCES = ["api.cu", "sdpa_tc.cu", "sdpa_one_tile.cu", "sdpa_bwd.cu", "sdpa_f32.cu", "gemm_tc.cu",
           "decode.cu", "mha_noalloc.cu", "sdpa_bwd_wide.cu", "paged.cu"]
HEADERS = ["kernels.h", "ptx.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libsdpa")


def _flags() -> list[str]:
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                   "-I", CSRC, "--expt-relaxed-constexpr"]


def _torch_dir() -> str | None:
    """The folder of an installed torch for CUDA."""
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        return None
    torch = os.path.dirname(spec.origin)
    return torch if os.path.exists(os.path.join(torch, "lib", "libc10_cuda.so")) else None


def _torch_version(torch: str) -> str:
    """What torch.__version__ will be."""
    with open(os.path.join(torch, "version.py")) as f:
        found = re.search(r"""^__version__\s*=\s*['"]([^'"]+)""", f.read(), re.M)
    if found is None:
        raise RuntimeError("no version in %s" % os.path.join(torch, "version.py"))
    return found.group(1)


def _fits(torch: str) -> str:
    """What an extension built now fits: this interpreter, this torch."""
    return "%s\n%s\n%s\n" % (os.path.basename(BIND), torch, _torch_version(torch))


def _bind_stamp() -> str:
    return os.path.join(BUILD_DIR, os.path.basename(BIND) + ".fits")


def _bind_stale(torch: str) -> bool:
    if _stale(BIND, [BIND_SOURCE, os.path.join(INCLUDE, "sdpa.h"), __file__]):
        return True
    try:
        with open(_bind_stamp()) as f:
            return f.read() != _fits(torch)
    except (RuntimeError, OSError):
        return True


def _bind_command(nvcc: str, torch: str, out: str) -> list[str]:
    """Compiles and links the extension against the torch in this folder."""
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE,
            '-DSDPA_TORCH_VERSION="%s"' % _torch_version(torch),
            "-isystem", os.path.join(torch, "include"), "-isystem", cuda, "-I", sysconfig.get_paths()["include"],
            BIND_SOURCE, "-o", out, "-L", os.path.join(torch, "lib"),
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    headers = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(INCLUDE, "sdpa.h")]
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers + [__file__]):
            jobs.append([nvcc] + _flags() + ["-c", s, "-o", o])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("%s failed:\n%s\n%s%s" % (os.path.basename(cmd[0]), " ".join(cmd), r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)

    # the extension compiles beside the library's sources, and fails by itself
    bind_tmp = os.path.join(BUILD_DIR, os.path.basename(BIND) + ".tmp%d" % os.getpid())
    torch = _torch_dir()
    bind = torch and (force or _bind_stale(torch))
    with cf.ThreadPoolExecutor(max_workers=len(jobs) + 1) as ex:
        binding = ex.submit(lambda: run(_bind_command(nvcc, torch, bind_tmp))) if bind else None
        list(ex.map(run, jobs))
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        run([nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs)
        os.replace(tmp, LIB)
    if binding is not None:
        try:
            binding.result()
            os.replace(bind_tmp, BIND)
            with open(_bind_stamp(), "w") as f:
                f.write(_fits(torch))
        except (RuntimeError, OSError) as e:
            # (one of older sources must not be taken for it)
            if os.path.exists(BIND):
                os.remove(BIND)
            sys.stderr.write("the paged helpers' extension was not built: %s\n" % e)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
